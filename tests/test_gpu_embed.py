"""Embedding lookup and its gradient against plain forms.

Lookup: one FP32 product and one rounding, as the plain form does: equal bits.
Gradient: a sum of L terms in FP32 in any order of additions is within L * 2^-24
of the sum of the terms' absolute values; the scale, the addition to the old
gradient and the result's own rounding (2^-8 BF16, 2^-11 FP16 and its subnormal
spacing) come on top."""
import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
ROUND = {F32: U, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 0.0, BF16: 0.0, F16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    fp8z.lib()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(n, h, dtype, seed, pad=0, std=1.0):
    """[n, h] with a row stride of h + pad elements."""
    t = torch.randn(n, h + pad, generator=_gen(seed), device="cuda").mul_(std).to(dtype)
    return t[:, :h]


@pytest.mark.parametrize("tokens,vocab,hidden", [(0, 5, 8), (1, 1, 1), (3, 100, 7), (8, 1000, 128), (257, 50, 576),
                                                 (33, 999, 8200), (5, 17, 9001)])
@pytest.mark.parametrize("src", [F32, BF16, F16])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_lookup(tokens, vocab, hidden, src, pad):
    table = _rows(vocab, hidden, src, 1, pad)
    for wide in (torch.int64, torch.int32):
        ids = torch.randint(0, vocab, (tokens,), generator=_gen(2), device="cuda").to(wide)
        for dst in (F32, BF16, F16):
            for scale in (1.0, 11.3137085):
                out = torch.full((tokens, hidden + pad), 7.0, dtype=dst, device="cuda")
                fp8z.fp8z_embedding(ids, table, out[:, :hidden], scale=scale)
                want = (table[ids.long()].float() * torch.tensor(scale, device="cuda")).to(dst)
                assert torch.equal(out[:, :hidden], want)
                assert bool((out[:, hidden:] == 7.0).all())          # nothing written past the rows


def test_lookup_ids_out_of_range():
    table = _rows(10, 16, BF16, 1)
    ids = torch.tensor([0, 9, 10, -1, 2 ** 40, 3], device="cuda")
    out = torch.full((6, 16), 5.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_embedding(ids, table, out, dev_status=st)
    assert st.item() == fp8z.FP8Z_EINVAL
    assert not out[2:5].any() and torch.equal(out[[0, 1, 5]], table[[0, 9, 3]].float())


def _ids(kind, n, v, seed):
    g = _gen(seed)
    if kind == "uniform":
        return torch.randint(0, v, (n,), generator=g, device="cuda")
    if kind == "one":
        return torch.full((n,), v - 1, device="cuda")
    if kind == "two":
        return torch.randint(0, 2, (n,), generator=g, device="cuda") * (v - 1)
    u = torch.rand(n, generator=g, device="cuda")
    return (float(v) ** u).long().clamp_(1, v) - 1


def _grad64(ids, d, v, scale, padding, base):
    keep = (ids >= 0) & (ids < v) & (ids != padding)
    i, x = ids[keep].long(), d.double()[keep] * scale
    total = torch.zeros(v, d.shape[1], dtype=torch.float64, device="cuda").index_add_(0, i, x)
    size = torch.zeros_like(total).index_add_(0, i, x.abs())
    count = torch.zeros(v, dtype=torch.float64, device="cuda").index_add_(0, i, torch.ones_like(i, dtype=torch.float64))
    if base is not None:
        total += base.double()
    return total, size, count


def _check_grad(ids, d, table, before, scale, padding, accumulate):
    base = before if accumulate else None
    want, size, count = _grad64(ids, d, table.shape[0], scale, padding, base)
    bound = (count[:, None] + 3) * U * size + want.abs() * (2 * U + ROUND[table.dtype]) + TINY[table.dtype]
    assert bool(((table.double() - want).abs() <= bound).all())
    if accumulate:
        assert torch.equal(table[count == 0], before[count == 0])


@pytest.mark.parametrize("tokens,vocab,hidden", [(0, 9, 8), (1, 1, 1), (1, 300, 24), (7, 5, 9), (100, 1000, 576), (2048, 33, 64),
                                                 (2049, 3000, 40), (5000, 1200, 72), (9001, 70000, 16), (20000, 50, 24),
                                                 (40000, 700, 40)])
@pytest.mark.parametrize("kind", ["uniform", "one", "two", "zipf"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad(tokens, vocab, hidden, kind, accumulate):
    ids = _ids(kind, tokens, vocab, 5)
    for src, dst, pad in ((BF16, F32, 0), (F16, F16, 8), (F32, BF16, 3)):
        d = _rows(tokens, hidden, src, 6, pad)
        full = torch.randn(vocab, hidden + pad, generator=_gen(8), device="cuda").to(dst)
        table, before = full[:, :hidden], full.clone()
        ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(tokens, vocab, hidden), dtype=torch.uint8, device="cuda")
        ws.fill_(255)
        fp8z.fp8z_embedding_grad(ids, d, table, ws, scale=0.5, padding_idx=0, accumulate=accumulate)
        _check_grad(ids, d, table, before[:, :hidden], 0.5, 0, accumulate)
        assert torch.equal(full[:, hidden:], before[:, hidden:])
        first = table.clone()
        full.copy_(before)
        fp8z.fp8z_embedding_grad(ids.int(), d, table, ws, scale=0.5, padding_idx=0, accumulate=accumulate)
        assert torch.equal(first, table)                     # the same bits every time


def test_grad_ids_out_of_range_and_no_padding():
    v, h = 40, 16
    ids = torch.tensor([0, 3, -1, 40, 3, 39, 2 ** 35, 0], device="cuda")
    d = _rows(8, h, BF16, 1)
    table = torch.full((v, h), 9.0, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(8, v, h), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_embedding_grad(ids, d, table, ws, dev_status=st)
    assert st.item() == fp8z.FP8Z_EINVAL
    _check_grad(ids, d, table, None, 1.0, -1, False)


def test_grad_against_differences():
    """d/dT of sum(out * r) by central differences of the lookup itself: the
    lookup is linear, so a step of 2^-6 on values that FP32 holds exactly leaves
    only the rounding of two sums of tokens * hidden products."""
    n, v, h = 30, 6, 8
    ids = _ids("uniform", n, v, 1)
    table = (torch.randint(-8, 8, (v, h), generator=_gen(2), device="cuda") / 8.0).float()
    r = (torch.randint(-8, 8, (n, h), generator=_gen(3), device="cuda") / 8.0).float()
    grad = torch.empty(v, h, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(n, v, h), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_embedding_grad(ids, r, grad, ws, scale=3.0)
    out, step = torch.empty(n, h, device="cuda"), 2.0 ** -6
    for i, j in ((0, 0), (3, 5), (5, 7)):
        f = []
        for sign in (1.0, -1.0):
            t = table.clone()
            t[i, j] += sign * step
            fp8z.fp8z_embedding(ids, t, out, scale=3.0)
            f.append(float((out.double() * r.double()).sum()))
        assert (f[0] - f[1]) / (2 * step) == pytest.approx(grad[i, j].item(), abs=1e-9)


def test_without_padding_every_bad_id_is_reported():
    ids, d = torch.tensor([-1, 2], device="cuda"), _rows(2, 8, BF16, 1)
    table, st = torch.zeros(4, 8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(2, 4, 8), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_embedding_grad(ids, d, table, ws, dev_status=st)
    assert st.item() == fp8z.FP8Z_EINVAL and torch.equal(table[2], d[1].float()) and not table[[0, 1, 3]].any()


def test_grad_does_not_read_padding():
    """What the gradient holds at padding tokens, NaN included, does not matter."""
    ids = torch.tensor([3, 0, 5, 0, 3], device="cuda")
    d = _rows(5, 40, BF16, 1)
    d[1], d[3] = float("nan"), float("inf")
    table = torch.full((8, 40), 2.0, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(5, 8, 40), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_embedding_grad(ids, d, table, ws, padding_idx=0)
    assert torch.equal(table[3], d[0].float() + d[4].float()) and torch.equal(table[5], d[2].float())
    assert not table[[0, 1, 2, 4, 6, 7]].any()


def test_offsets_past_32_bits():
    v, h = 300001, 7168                      # 2.15e9 elements
    table = torch.zeros(v, h, dtype=BF16, device="cuda")
    table[-3:] = _rows(3, h, BF16, 2)
    ids = torch.tensor([v - 1, 0, v - 3, v - 2, v - 1], device="cuda")
    out = torch.empty(5, h, dtype=BF16, device="cuda")
    fp8z.fp8z_embedding(ids, table, out)
    assert torch.equal(out, table[ids])
    del table
    grad = torch.full((v, h), 3.0, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(5, v, h), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_embedding_grad(ids, out, grad, ws)
    assert torch.equal(grad[v - 1], out[0].float() + out[4].float()) and torch.equal(grad[v - 3], out[2].float())
    assert not grad[1:v - 3].any()


@pytest.mark.parametrize("tokens", [300, 5000])
def test_graph_replay(tokens):
    v, h = 900, 64
    ids, d = _ids("zipf", tokens, v, 1), _rows(tokens, h, BF16, 2)
    grad, out = torch.empty(v, h, device="cuda"), torch.empty(tokens, h, dtype=BF16, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(tokens, v, h), dtype=torch.uint8, device="cuda")
    table = _rows(v, h, BF16, 3)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fp8z.fp8z_embedding(ids, table, out)
            fp8z.fp8z_embedding_grad(ids, d, grad, ws)
    ids.copy_(_ids("uniform", tokens, v, 7))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, table[ids])
    _check_grad(ids, d, grad, None, 1.0, -1, False)


def test_grad_on_another_stream():
    s = torch.cuda.Stream()
    ids = _ids("zipf", 3000, 500, 4)
    d = _rows(3000, 64, BF16, 5)
    table = torch.empty(500, 64, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(3000, 500, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    fp8z.fp8z_embedding_grad(ids, d, table, ws, stream=s)
    s.synchronize()
    _check_grad(ids, d, table, None, 1.0, -1, False)


def test_refusals():
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    table, out = torch.zeros(9, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(4, 9, 8), dtype=torch.uint8, device="cuda")
    for bad in (dict(ids=ids[:3]), dict(ids=ids.float()), dict(table=table.t()), dict(out=out[:, :7]),
                dict(out=out.double()), dict(table=table.cpu())):
        with pytest.raises(ValueError):
            fp8z.fp8z_embedding(**{**dict(ids=ids, table=table, out=out), **bad})
        b = {{"ids": "ids", "table": "d_table", "out": "d_out"}[k]: v for k, v in bad.items()}
        with pytest.raises(ValueError):
            fp8z.fp8z_embedding_grad(**{**dict(ids=ids, d_table=table, d_out=out, workspace=ws), **b})
    with pytest.raises(fp8z.Fp8zError) as e:
        fp8z.fp8z_embedding_grad(ids, out, table, ws[:16])
    assert e.value.status == fp8z.FP8Z_ENOSPACE
    with pytest.raises(fp8z.Fp8zError):
        fp8z.fp8z_embedding(ids, table, out, scale=float("nan"))
