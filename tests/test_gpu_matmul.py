"""fp8z_matmul against the sum of its definition in 64 bits.

Bound, from the formula: a block's S is four tensor core steps of 32 products that
cut off where FP32 ends, each by at most two units of the largest partial sum (4 * 2 *
2^-22 = 32 * 2^-24 of the sum of absolute values); its factor is rounded at most three
times and added up with one rounding a block, so that FP32 results are off by at most
(kb + 35) * 2^-24 * sum |a b| scaled, and 16-bit results by half a step of their type
beside it.  An out that is added to is rounded once more."""
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, *shape):
    """Finite E4M3 codes of all sizes, zeros of both signs among them."""
    q = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.int32)
    return torch.where((q & 127) == 127, q - 1, q).to(torch.uint8)


def scales(g, *shape):
    return torch.exp(2.0 * torch.randn(shape, generator=g, device="cuda"))


def strided(t, pad, lead=0):
    """t in a buffer of longer rows that starts `lead` elements late; what is around it is 0x7F bytes (NaN codes)."""
    rows, cols = t.shape
    raw = torch.full(((lead + rows * (cols + pad)) * t.element_size(),), 0x7F, dtype=torch.uint8, device="cuda").view(t.dtype)
    v = raw[lead:].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def values(q):
    return q.view(torch.float8_e4m3fn).double()


def spread(s, k):
    return s.double().repeat_interleave(128, -1)[..., :k]


def definition(a, sa, b, sb, per_block):
    """The product and the sum of absolute values, in 64 bits."""
    k = a.shape[1]
    x = values(a.contiguous()) * spread(sa, k)
    rows = sb.repeat_interleave(128, 0)[:b.shape[0]] if per_block else sb
    w = values(b.contiguous()) * spread(rows, k)
    return x @ w.t(), x.abs() @ w.abs().t()


def check(out, want, size, k, before=None):
    eps = 0.0 if out.dtype == F32 else torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps
    if before is not None:
        want = want + before.double()
        size = size + before.double().abs()
    kb = -(-k // 128)
    bound = (kb + 35) * 2.0 ** -24 * size + eps * want.abs() * (1 + 1e-3) + tiny
    if before is not None:
        bound = bound + 2.0 ** -24 * want.abs()
    bad = ~((out.double() - want).abs() <= bound)
    if out.dtype == F16:
        bad &= want.abs() < 65504.0
    assert not bad.any(), (out[bad][:4], want[bad][:4], bad.nonzero()[:4], int(bad.sum()))


def product(m, n, k, per_block=True, dtype=BF16, accumulate=False, seed=0, pad=0, lead=0, out_pad=0, out_lead=0, small=1.0):
    g = gen(seed)
    kb = -(-k // 128)
    a, b = codes(g, m, k), codes(g, n, k)
    sa, sb = scales(g, m, kb) * small / (448.0 * max(k, 1) ** 0.5), scales(g, -(-n // 128) if per_block else n, kb) / 448.0
    if pad or lead:
        a, b, sa, sb = strided(a, pad, lead), strided(b, pad, lead), strided(sa, 1, 1), strided(sb, 1, 1)
    start = torch.randn(m, n, generator=g, device="cuda").to(dtype) if accumulate else torch.full((m, n), 7.0, dtype=dtype, device="cuda")
    out = strided(start, out_pad, out_lead)
    ws = torch.empty(fp8z.fp8z_matmul_workspace(a, b, out), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_matmul(a, sa, b, sb, out, accumulate=accumulate, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    want, size = definition(a, sa, b, sb, per_block)
    check(out, want, size, k, start if accumulate else None)
    if out_pad or out_lead:
        base = torch.as_strided(out, (m, n + out_pad), (n + out_pad, 1)).contiguous()
        assert (base[:, n:].contiguous().view(torch.uint8) == 0x7F).all(), "written behind a row"
    return out


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 130, 129), (8, 576, 7168), (15, 100, 100), (16, 300, 640), (17, 200, 384),
          (33, 257, 1000), (64, 1000, 256), (65, 129, 2048), (100, 300, 1000), (129, 129, 127), (200, 18432, 384),
          (255, 1000, 576), (511, 3000, 130), (1003, 2001, 576), (2048, 2304, 256), (2049, 4100, 640), (5, 70000, 128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_blocks(m, n, k):
    for i, dtype in enumerate((BF16, F32, F16)):
        product(m, n, k, dtype=dtype, seed=i)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (100, 128, 128), (128, 200, 8192), (300, 129, 1000), (576, 1000, 640),
                                   (2000, 2304, 384), (2304, 4000, 1029)])
def test_rows(m, n, k):
    for i, (dtype, acc) in enumerate(((F32, True), (F32, False), (BF16, False))):
        product(m, n, k, per_block=False, dtype=dtype, accumulate=acc, seed=i)


@pytest.mark.parametrize("m,n,k", [(3, 200, 200), (70, 300, 1000), (1000, 2000, 500), (2500, 2500, 129)])
@pytest.mark.parametrize("pad,lead,out_pad,out_lead", [(16, 16, 8, 8), (1, 0, 0, 0), (3, 5, 1, 3), (0, 1, 4, 4)])
def test_strides(m, n, k, pad, lead, out_pad, out_lead):
    product(m, n, k, dtype=BF16, pad=pad, lead=lead, out_pad=out_pad, out_lead=out_lead)
    product(m, n, k, dtype=F32, accumulate=True, pad=pad, lead=lead, out_pad=out_pad, out_lead=out_lead)
    product(m, n, k, per_block=False, dtype=F32, pad=pad, lead=lead, out_pad=out_pad, out_lead=out_lead)


def bank(e, m, n, k, cuts, dtype=BF16, wide=False, accumulate=False, seed=0):
    """Rows cuts[i] .. cuts[i + 1] of a against weight i."""
    g = gen(seed)
    kb, nb = -(-k // 128), -(-n // 128)
    a, b = codes(g, m, k), codes(g, e, n, k)
    sa, sb = scales(g, m, kb) / (448.0 * k ** 0.5), scales(g, e, nb, kb) / 448.0
    offsets = torch.tensor(cuts, dtype=torch.int64 if wide else torch.int32, device="cuda")
    out = torch.full((m, n), 7.0, dtype=dtype, device="cuda")
    ws = torch.empty(fp8z.fp8z_matmul_workspace(a, b, out, offsets), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_matmul(a, sa, b, sb, out, offsets=offsets, accumulate=accumulate, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for i in range(e):
        r = slice(cuts[i], cuts[i + 1])
        if cuts[i] < cuts[i + 1]:
            want, size = definition(a[r], sa[r], b[i], sb[i], True)
            check(out[r], want, size, k, torch.full_like(out[r], 7.0) if accumulate else None)
    assert (out[:cuts[0]] == 7.0).all() and (out[cuts[-1]:] == 7.0).all(), "rows of no group"


@pytest.mark.parametrize("e,m,n,k,cuts", [
    (1, 5, 128, 128, [0, 5]), (4, 10, 200, 384, [0, 3, 3, 9, 10]), (3, 40, 129, 200, [5, 5, 20, 33]),
    (8, 300, 256, 256, [0, 0, 1, 17, 150, 151, 299, 299, 300]), (4, 2000, 1024, 256, [0, 1300, 1300, 1999, 2000]),
    (2, 3000, 2304, 128, [100, 700, 2950]), (256, 512, 128, 128, [min(512, 3 * i) for i in range(257)]),
    (5, 50, 64, 77, [0, 0, 0, 0, 0, 0])])
def test_groups_of_rows(e, m, n, k, cuts):
    bank(e, m, n, k, cuts)
    bank(e, m, n, k, cuts, dtype=F32, wide=True, accumulate=True, seed=1)


def gradients(e, m, n, cuts, dtype=F32, accumulate=False, seed=0):
    """Columns cuts[i] .. cuts[i + 1] of a and b give gradient i."""
    g = gen(seed)
    k = cuts[-1] + (0 if cuts[-1] % 128 else 128)
    kb = -(-k // 128)
    a, b = codes(g, m, k), codes(g, n, k)
    sa, sb = scales(g, m, kb) / (448.0 * k ** 0.5), scales(g, n, kb) / 448.0
    offsets = torch.tensor(cuts, dtype=torch.int64, device="cuda")
    start = torch.randn(e, m, n, generator=g, device="cuda").to(dtype)
    out = start.clone()
    ws = torch.empty(fp8z.fp8z_matmul_workspace(a, b, out, offsets), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_matmul(a, sa, b, sb, out, offsets=offsets, accumulate=accumulate, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for i in range(e):
        c0, c1 = cuts[i], cuts[i + 1]
        s = slice(c0 // 128, -(-c1 // 128))
        want, size = definition(a[:, c0:c1], sa[:, s], b[:, c0:c1], sb[:, s], False)
        check(out[i], want, size, max(c1 - c0, 1), start[i] if accumulate else None)


@pytest.mark.parametrize("e,m,n,cuts", [(1, 100, 200, [0, 128]), (3, 130, 257, [0, 384, 384, 640]),
                                        (4, 512, 768, [128, 256, 1024, 1024, 1100]), (2, 33, 1000, [0, 0, 0]),
                                        (5, 300, 129, [0, 128, 128, 128, 512, 1280])])
def test_groups_of_columns(e, m, n, cuts):
    for i, (dtype, acc) in enumerate(((F32, False), (F32, True), (BF16, False))):
        gradients(e, m, n, cuts, dtype, acc, i)
