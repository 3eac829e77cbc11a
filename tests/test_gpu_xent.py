"""Softmax cross entropy of a vocabulary projection and its gradient against the
definition in 64 bits.

Bounds.  A logit is a sum of hidden products that are exact in FP32, added in
steps of 16 that may each cut off 2^-22 of the sum of the absolute products:
dl = (hidden / 16 + 2) * 2^-22 * sum |x w|.  The exponent's rounding adds
2^-23 (|l| + |lse|), each exponential 2^-22, the sum of exponentials over 256
columns, the tiles and eight partial rows (256 / 32 * 2 + tiles / 8 + 48) * 2^-24.
With d the bound on the exponent, p is within p * (d + 2^-22) of its value; P is
rounded by u (2^-8 BF16, 2^-11 FP16 with its subnormal spacing, kept times 2^12),
or u^2 where it is split in two; the products add their cut-off sums, and the
result rounds once."""
import math

import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
UNIT = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 0.0, BF16: 0.0, F16: 2.0 ** -25}
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    fp8z.lib()


def _inputs(n, h, v, dtype, seed=0, pad=0, ignored=0.2, std=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, h + pad, generator=g, device="cuda").to(dtype)[:, :h]
    w = (torch.randn(v, h + pad, generator=g, device="cuda") * (std or 2.0 / math.sqrt(h))).to(dtype)[:, :h]
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[torch.rand(n, generator=g, device="cuda") < ignored] = IGNORE
    return x, w, t


def _define(x, w, t, v):
    """64-bit logits, lse, loss, kept, and the bound d on the exponent's error."""
    xd, wd = x.double(), w.double()
    l = xd @ wd.t()
    lse = torch.logsumexp(l, 1)
    keep = (t >= 0) & (t < v)
    at = t.clamp(0, v - 1).long()
    loss = torch.where(keep, lse - l.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    h, tiles = x.shape[1], -(-v // 256)
    size = (xd.abs() @ wd.abs().t()).amax(1)
    top = l.abs().amax(1)
    dl = (h / 16 + 2) * 2.0 ** -22 * size
    dlse = dl + 2.0 ** -22 + 2.0 ** -23 * top + (16 + tiles / 8 + 48) * 2.0 ** -24 + 2.0 ** -24 * lse.abs()
    return l, lse, loss, keep, at, dl, dlse, dl + dlse + 2.0 ** -23 * (top + lse.abs())


def _check_loss(x, w, t, loss, total, lse_got, reduction):
    l, lse, want, keep, at, dl, dlse, d = _define(x, w, t, w.shape[0])
    bound = (dl + dlse + 2.0 ** -24 * want.abs()) * keep
    assert bool(((loss.double() - want).abs() <= bound).all())
    assert bool(((lse_got.double() - lse).abs() <= dlse + 2.0 ** -24 * lse.abs()).all())
    by = max(1, int(keep.sum())) if reduction == "mean" else 1
    assert abs(total[0].item() - float(want.sum()) / by) <= float(bound.sum()) / by + 2.0 ** -23 * abs(float(want.sum())) / by
    assert total[1].item() == int(keep.sum())


def _check_grad(x, w, t, dx, dw, dw_before, reduction, scale):
    l, lse, _, keep, at, _, _, d = _define(x, w, t, w.shape[0])
    by = max(1, int(keep.sum())) if reduction == "mean" else 1
    a = scale / by
    xd, wd = x.double(), w.double()
    p = torch.exp(l - lse[:, None])
    P = p.scatter_add(1, at[:, None], torch.full_like(lse, -1.0)[:, None]) * keep[:, None]
    e = (p * (torch.expm1(d)[:, None] + 2.0 ** -22) + 2.0 ** -24) * keep[:, None]      # on P, before it is rounded
    u = UNIT[x.dtype]
    sub = 2.0 ** -25 / 4096 if x.dtype == F16 else 0.0
    n, v = P.shape

    def bound(mat, other, ulp, terms):
        err = mat.abs() * (ulp + (terms / 16 + 66) * 2.0 ** -22) + e * (1 + ulp) + sub
        return abs(a) * (err @ other.abs())

    want = a * (P @ wd)
    tol = bound(P, wd, u, v) + want.abs() * (UNIT[dx.dtype] + 2.0 ** -22) + TINY[dx.dtype]
    assert bool(((dx.double() - want).abs() <= tol).all())
    split = dw.dtype == F32
    want = a * (P.t() @ xd)
    err = P.abs() * ((u * u if split else u) + (n * (2 if split else 1) / 16 + 66) * 2.0 ** -22) + e * (1 + u) + sub
    tol = abs(a) * (err.t() @ xd.abs())
    if dw_before is not None:
        want = want + dw_before.double()
    tol += want.abs() * (UNIT[dw.dtype] + 2.0 ** -22) + TINY[dw.dtype]
    assert bool(((dw.double() - want).abs() <= tol).all())


def _buffers(n, h, v, dtype, dw_dtype, pad=0):
    loss = torch.full((n,), math.nan, device="cuda")
    lse = torch.full((n,), math.nan, device="cuda")
    total = torch.full((2,), math.nan, device="cuda")
    dx = torch.full((n, h + pad), 7.0, dtype=dtype, device="cuda")
    dw = torch.full((v, h + pad), 0.5, dtype=dw_dtype, device="cuda")
    return loss, lse, total, dx, dw


def _workspace(size):
    return torch.full((size,), 255, dtype=torch.uint8, device="cuda")      # NaN wherever it is read unwritten


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


SHAPES = [(3000, 136, 700), (40, 72, 20000), (1, 8, 1), (1, 64, 256), (7, 100, 1000), (5, 7, 33), (128, 64, 256), (129, 72, 257), (300, 576, 5000),
          (513, 2048, 3001), (64, 40, 70000), (1000, 136, 999), (2, 4104, 515)]


@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_loss(n, h, v, dtype, pad):
    x, w, t = _inputs(n, h, v, dtype, seed=n, pad=pad)
    for reduction, tt in (("mean", t), ("sum", t.int())):
        loss, lse, total, _, _ = _buffers(n, h, v, dtype, F32)
        ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w))
        st = _status()
        fp8z.fp8z_linear_xent(x, w, tt, loss, total, ws, ignore_index=IGNORE, reduction=reduction, lse=lse, dev_status=st)
        assert st.item() == 0                                              # no wait ran out
        _check_loss(x, w, t, loss, total, lse, reduction)


@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("pad,piece,accumulate", [(0, 0, False), (3, 256, True), (8, 600, False)])
def test_gradient(n, h, v, dtype, wide, pad, piece, accumulate):
    x, w, t = _inputs(n, h, v, dtype, seed=n + 1, pad=pad)
    dw_dtype, scale = (F32 if wide else dtype), (1.0 if dtype == BF16 else 64.0)
    loss, lse, total, dx, dw = _buffers(n, h, v, dtype, dw_dtype, pad)
    before = dw[:, :h].clone() if accumulate else None
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw[:, :h], piece_words=piece))
    reduction, st = "sum" if pad else "mean", _status()

    def call():
        fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx[:, :h], dw[:, :h], ws, ignore_index=IGNORE, dev_status=st,
                                   reduction=reduction, grad_scale=scale, accumulate_dw=accumulate, lse=lse)
    call()
    assert st.item() == 0                                                  # no wait ran out
    _check_loss(x, w, t, loss, total, lse, reduction)
    _check_grad(x, w, t, dx[:, :h], dw[:, :h], before, reduction, scale)
    assert bool((dx[:, h:] == 7.0).all()) and bool((dw[:, h:] == 0.5).all())
    first = dx.clone(), dw.clone()
    dw.fill_(0.5)
    call()
    assert torch.equal(first[0], dx) and torch.equal(first[1], dw)          # the same bits every time


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_nothing_kept_and_no_tokens(dtype):
    for n in (0, 37):
        x, w, t = _inputs(n, 64, 300, dtype, ignored=2.0)
        loss, lse, total, dx, dw = _buffers(n, 64, 300, dtype, F32)
        ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
        fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, ignore_index=IGNORE)
        assert total.tolist() == [0.0, 0.0] and not loss.any() and not dx.any() and not dw.any()
        dw.fill_(0.5)
        fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, ignore_index=IGNORE, accumulate_dw=True)
        assert bool((dw == 0.5).all())


def test_targets_out_of_range():
    x, w, t = _inputs(9, 32, 50, BF16, ignored=0.0)
    t[2], t[5], t[7] = 50, -7, 2 ** 33
    loss, lse, total, dx, dw = _buffers(9, 32, 50, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse, dev_status=st)
    assert st.item() == fp8z.FP8Z_EINVAL
    _check_loss(x, w, t, loss, total, lse, "mean")
    _check_grad(x, w, t, dx, dw, None, "mean", 1.0)


def test_extreme_logits_and_bad_rows():
    """Logits of several hundred (a plain sum of exponentials would overflow), and
    one token with an infinity: its own loss and gradient row are lost, no other."""
    x, w, t = _inputs(140, 64, 900, BF16, ignored=0.1, std=10.0)
    loss, lse, total, dx, dw = _buffers(140, 64, 900, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse)
    _check_loss(x, w, t, loss, total, lse, "mean")
    _check_grad(x, w, t, dx, dw, None, "mean", 1.0)
    good = loss.clone(), dx.clone()
    t[3] = 5
    x[3, 7] = math.inf
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum")
    rest = torch.arange(140, device="cuda") != 3
    assert math.isnan(loss[3].item()) and torch.equal(loss[rest], good[0][rest])
    assert bool(dx[rest].isfinite().all()) and bool(dx[3].isnan().any())


def test_what_ignored_tokens_hold_does_not_matter():
    """NaN and infinities in the x of ignored tokens, and in a padded row's unused
    end, leave every result of the others as it is."""
    x, w, t = _inputs(150, 72, 700, BF16, pad=8)
    loss, lse, total, dx, dw = _buffers(150, 72, 700, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws)
    want = [a.clone() for a in (loss, total, dx, dw)]
    x[t == IGNORE] = math.nan
    x[int((t == IGNORE).nonzero()[0]), 3] = math.inf
    x._base[:, 72:] = math.nan
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws)
    assert all(torch.equal(a, b) for a, b in zip((loss, total, dx, dw), want))


def test_graph_replay_and_small_pieces_agree():
    """A captured call replayed on new inputs gives what the eager call gives, and
    the pieces of the vocabulary do not change dw (dx adds them in another order)."""
    x, w, t = _inputs(70, 128, 3000, BF16)
    loss, lse, total, dx, dw = _buffers(70, 128, 3000, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse)
    x2, _, t2 = _inputs(70, 128, 3000, BF16, seed=9)
    x.copy_(x2)
    t.copy_(t2)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    got = [a.clone() for a in (loss, total, dx, dw, lse)]
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse)
    assert all(torch.equal(a, b) for a, b in zip(got, (loss, total, dx, dw, lse)))
    small = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw, piece_words=512))
    assert small.numel() < ws.numel()
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, small, lse=lse)
    assert torch.equal(dw, got[3]) and torch.equal(loss, got[0])


def test_offsets_past_32_bits():
    """A vocabulary projection of more than 2^31 elements: the last words' logits
    and gradients are where they belong.  A logit is within 450 * 2^-22 * 7168 / 40
    = 0.02 (the bound of this file's first lines), a probability within twice that
    in relative terms: 0.05 tells a right row from any other."""
    n, h, v = 3, 7168, 300001
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.zeros(v, h, dtype=BF16, device="cuda")
    w[-5:] = (torch.randn(5, h, generator=g, device="cuda") / 40).to(BF16)
    x = torch.randn(n, h, generator=g, device="cuda").to(BF16)
    t = torch.tensor([v - 1, v - 3, 7], device="cuda")
    loss, lse, total, dx, dw = _buffers(n, h, v, BF16, F32)
    ws = torch.empty(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse)
    l = torch.zeros(n, v, dtype=torch.float64, device="cuda")
    l[:, -5:] = x.double() @ w[-5:].double().t()
    want = torch.logsumexp(l, 1) - l.gather(1, t[:, None])[:, 0]
    # 448 steps of at most 2^-22 of a sum of absolute products under 7168 / 40
    assert bool(((loss.double() - want).abs() <= 450 * 2.0 ** -22 * 7168 / 40).all())
    p = torch.softmax(l, 1)
    p.scatter_add_(1, t[:, None], torch.full((n, 1), -1.0, dtype=torch.float64, device="cuda"))
    for i in (0, 7, v - 5, v - 3, v - 1):
        ref = p[:, i] @ x.double() / n
        size = p[:, i].abs() @ x.double().abs() / n
        assert bool(((dw[i].double() - ref).abs() <= size * (2.0 ** -16 + 0.05) + 1e-12).all())
        assert float((dw[i].double() - ref).norm() / (ref.norm() + 1e-30)) < 0.05


def test_gradient_against_differences():
    """Central differences of the loss itself.  |w| <= 1/4 and a step of 2^-4: the
    third derivative leaves (2^-4)^2 / 6 * (2 * 0.25)^3 < 1e-4, the loss's own
    error (under 4e-6) divided by the step's 2^-3 another 4e-5; dx rounds by 2^-8,
    and P by 2^-8 against sum |P| |w| <= 0.5."""
    n, h, v = 6, 16, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randint(-16, 17, (n, h), generator=g, device="cuda") / 16.0).to(BF16)
    w = (torch.randint(-16, 17, (v, h), generator=g, device="cuda") / 64.0).to(BF16)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    loss, lse, total, dx, dw = _buffers(n, h, v, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum")
    for i, j in ((0, 0), (2, 7), (5, 15)):
        f = []
        for sign in (1, -1):
            y = x.clone()
            y[i, j] += sign * 2.0 ** -4
            fp8z.fp8z_linear_xent(y, w, t, loss, total, ws, reduction="sum")
            f.append(loss.double()[i].item())
        slope = (f[0] - f[1]) / 2.0 ** -3
        assert abs(slope - dx[i, j].item()) <= 1.4e-4 + 2.0 ** -8 * (abs(slope) + 0.5)
    for i, j in ((int(t[0]), 3), (11, 9)):
        f = []
        for sign in (1, -1):
            y = w.clone()
            y[i, j] += sign * 2.0 ** -6
            fp8z.fp8z_linear_xent(x, y, t, loss, total, ws, reduction="sum")
            f.append(loss.double().sum().item())
        slope = (f[0] - f[1]) / 2.0 ** -5
        # six losses' errors over 2^-5; third derivative of each at most |2x|^3 = 8
        assert abs(slope - dw[i, j].item()) <= 6 * (4e-6 * 32 + 2.0 ** -12 / 6 * 8)


def test_another_stream():
    x, w, t = _inputs(200, 128, 2000, BF16)
    loss, lse, total, dx, dw = _buffers(200, 128, 2000, BF16, BF16)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse, stream=s)
    s.synchronize()
    _check_loss(x, w, t, loss, total, lse, "mean")
    _check_grad(x, w, t, dx, dw, None, "mean", 1.0)


def test_refusals():
    x, w, t = _inputs(8, 32, 100, BF16)
    loss, lse, total, dx, dw = _buffers(8, 32, 100, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    ok = dict(x=x, w=w, targets=t, loss=loss, total=total, dx=dx, dw=dw, workspace=ws)
    fp8z.fp8z_linear_xent_grad(**ok)
    for bad in (dict(x=x.float()), dict(w=w.half()), dict(w=w[:, :31]), dict(targets=t[:7]), dict(targets=t.float()),
                dict(loss=loss[:7]), dict(total=total[:1]), dict(dx=dx[:7]), dict(dx=dx.float()), dict(dw=dw.half()),
                dict(dw=dw[:99]), dict(reduction="none"), dict(x=x.cpu()), dict(w=torch.zeros(32, 100, device="cuda").to(BF16).t())):
        with pytest.raises(ValueError):
            fp8z.fp8z_linear_xent_grad(**{**ok, **bad})
    with pytest.raises(fp8z.Fp8zError) as e:
        fp8z.fp8z_linear_xent_grad(**{**ok, "workspace": ws[:4096]})
    assert e.value.status == fp8z.FP8Z_ENOSPACE
    with pytest.raises(fp8z.Fp8zError):
        fp8z.fp8z_linear_xent_grad(**ok, grad_scale=math.inf)


def test_waits_that_run_out():
    """The products' own bounded waits, cut to 1 ns: a launch reports the timeout,
    lets its copies and products finish and returns, and the next call with the
    limit restored is right."""
    x, w, t = _inputs(600, 1024, 20000, BF16)
    loss, lse, total, dx, dw = _buffers(600, 1024, 20000, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_set_wait_limit_ns(1)
    try:
        for _ in range(5):
            st.zero_()
            fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, dev_status=st)
            torch.cuda.synchronize()
            if st.item() != 0:
                break
    finally:
        fp8z.fp8z_set_wait_limit_ns(0)
    assert st.item() == fp8z.FP8Z_ETIMEOUT
    st.zero_()
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, lse=lse, dev_status=st)
    assert st.item() == 0
    _check_loss(x, w, t, loss, total, lse, "mean")
    _check_grad(x, w, t, dx, dw, None, "mean", 1.0)


@pytest.mark.parametrize("ld,start", [(40, 0), (40, 3), (44, 1), (42, 4), (41, 5), (47, 7)])
@pytest.mark.parametrize("n,h,v", [(1, 33, 5), (9, 40, 1025), (32, 34, 3001), (3, 1, 9), (17, 7, 300)])
def test_rows_of_w_between_16_byte_boundaries(ld, start, n, h, v):
    """w starts anywhere and steps by anything; what lies before, between and behind its rows is NaN."""
    x, dense, t = _inputs(n, h, v, BF16, seed=ld + start, pad=1)
    flat = torch.full((start + v * ld + 16,), math.nan, dtype=BF16, device="cuda")
    w = flat[start:start + v * ld].view(v, ld)[:, :h]
    w.copy_(dense)
    loss, lse, total, _, _ = _buffers(n, h, v, BF16, F32)
    ws = _workspace(fp8z.fp8z_linear_xent_workspace(x, w))
    st = _status()
    fp8z.fp8z_linear_xent(x, w, t, loss, total, ws, ignore_index=IGNORE, lse=lse, dev_status=st)
    assert st.item() == 0
    _check_loss(x, w, t, loss, total, lse, "mean")


@pytest.mark.parametrize("n", [1, 8, 16, 32, 40, 300])
@pytest.mark.parametrize("h", [1536, 28672, 28679])
def test_long_sums_are_rounded_not_cut_off(n, h):
    """Products of one sign: a sum that the tensor cores cut off at every 16 of K is short
    by up to 2^-23 of itself a step (a quarter of that on average, 5e-5 at 1792 steps).
    No more than 24 blocks of 64, 96 steps, are added up that way; the sums of these are
    rounded, h / 1024 times at most by 2^-24 (in steps of 256 for a few tokens)."""
    g = torch.Generator(device="cuda").manual_seed(h + n)
    x = (torch.rand(n, h, generator=g, device="cuda") + 0.5).to(BF16)
    w = ((torch.rand(300, h, generator=g, device="cuda") + 0.5) * (20.0 / h)).to(BF16)
    t = torch.randint(0, 300, (n,), generator=g, device="cuda")
    loss, lse, total, _, _ = _buffers(n, h, 300, BF16, F32)
    st = _status()
    fp8z.fp8z_linear_xent(x, w, t, loss, total, _workspace(fp8z.fp8z_linear_xent_workspace(x, w)), lse=lse, dev_status=st)
    assert st.item() == 0
    l = x.double() @ w.double().t()
    want = torch.logsumexp(l, 1)
    off = (96 * 2.0 ** -23 + (h / 256 + 2) * 2.0 ** -24) * l.amax(1)
    rest = 2.0 ** -22 + 2.0 ** -23 * l.amax(1) + 64 * 2.0 ** -24 + 2.0 ** -23 * want
    assert bool(((lse.double() - want).abs() <= off + rest).all())
    assert bool(((loss.double() - (want - l.gather(1, t[:, None])[:, 0])).abs() <= 2 * off + rest).all())
