"""Global gradient norm and clipping against the definition in 64 bits.

Bounds, with u = 2^-24 (FP32): a square carries u, sixteen of them added in
FP32 at most 16u more, the FP64 sum nothing; the root halves that and rounds
once: the norm is within (17/2 + 1) u < 10u.  The factor adds the roundings of
norm + eps, the quotient and the product with grad_scale (3u), the scaled
element one more, and its type's own rounding (2^-8 BF16, 2^-11 FP16; FP16
also its subnormal spacing)."""
import math

import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    fp8z.lib()


@pytest.fixture
def ws():
    return torch.zeros(fp8z.fp8z_grad_norm_workspace(), dtype=torch.uint8, device="cuda")


def _tensors(sizes, dtypes, seed=0, std=1e-3, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + offset, generator=g, device="cuda").mul_(std).to(dtypes[i % len(dtypes)])
        out.append(t[offset:])
    return out


def _norm64(ts, scale=1.0):
    return abs(scale) * math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def _check(srcs, dsts, before, max_norm, scale, norm):
    want = _norm64(before, scale)
    coef = min(1.0, max_norm / (want + 1e-6))
    got, c = norm.tolist()
    assert abs(got - want) <= 10 * U * want + 1e-45
    assert abs(c - coef) <= 13 * U * coef
    for b, d in zip(before, dsts):
        ref = b.double() * scale * coef
        bound = ref.abs() * (15 * U + ROUND[d.dtype]) + TINY[d.dtype]
        assert bool(((d.double() - ref).abs() <= bound).all())


F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SIZES = [[1], [7, 1, 0, 130], [4096], [4095, 4097, 1], [0, 0, 5, 0], [100000, 3, 12345, 0, 65536, 8191],
         [1500000, 4096 * 7, 11]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtypes", [[F32], [BF16], [F16], [F32, BF16, F16]])
@pytest.mark.parametrize("offset", [0, 1])
def test_clip_into_other_tensors(ws, sizes, dtypes, offset):
    srcs = _tensors(sizes, dtypes, offset=offset)
    for dd in (F32, BF16, F16):
        dsts = [torch.empty(t.numel() + offset, dtype=dd, device="cuda")[offset:] for t in srcs]
        tl = fp8z.fp8z_encode_tensor_list(srcs, dsts)
        norm = torch.full((2,), -1.0, device="cuda")
        for max_norm, scale in ((0.5 * _norm64(srcs) + 1e-9, 1.0), (1e6, 0.25), (0.01, -4.0)):
            fp8z.fp8z_grad_clip(tl, max_norm, norm, ws, grad_scale=scale)
            _check(srcs, dsts, srcs, max_norm, scale, norm)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_clip_in_place(ws, sizes, dtype):
    ts = _tensors(sizes, [dtype], seed=3, std=0.1)
    before = [t.clone() for t in ts]
    tl = fp8z.fp8z_encode_tensor_list(ts)
    norm = torch.zeros(2, device="cuda")
    big = _norm64(before) * 2 + 1
    fp8z.fp8z_grad_clip(tl, big, norm, ws)                       # nothing to clip: nothing written
    assert all(torch.equal(a, b) for a, b in zip(ts, before)) and norm[1].item() == 1.0
    fp8z.fp8z_grad_clip(tl, 0.05, norm, ws)
    _check(ts, ts, before, 0.05, 1.0, norm)


def test_norm_alone_empty_and_repeated(ws):
    norm = torch.full((2,), -1.0, device="cuda")
    fp8z.fp8z_grad_norm(fp8z.fp8z_encode_tensor_list([]), norm, ws)
    assert norm.tolist() == [0.0, 1.0]
    ts = _tensors([300001, 17, 4096], [F32, BF16])
    tl = fp8z.fp8z_encode_tensor_list(ts)
    seen = set()
    for _ in range(5):
        fp8z.fp8z_grad_norm(tl, norm, ws, grad_scale=-2.0)
        seen.add(norm[0].item())
    assert len(seen) == 1 and abs(seen.pop() - _norm64(ts, 2.0)) <= 10 * U * _norm64(ts, 2.0)
    zeros = [torch.zeros(1000, device="cuda")]
    fp8z.fp8z_grad_clip(fp8z.fp8z_encode_tensor_list(zeros), 1.0, norm, ws)
    assert norm.tolist() == [0.0, 1.0] and not zeros[0].any()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinite_and_nan_gradients(ws, bad):
    ts = _tensors([5000, 10], [F32])
    ts[0][4321] = bad
    norm = torch.zeros(2, device="cuda")
    fp8z.fp8z_grad_clip(fp8z.fp8z_encode_tensor_list(ts), 1.0, norm, ws)
    if math.isnan(bad):
        assert math.isnan(norm[0].item()) and all(bool(t.isnan().all()) for t in ts)
    else:
        assert norm.tolist() == [math.inf, 0.0]
        assert not ts[1].any() and int(ts[0].isnan().sum()) == 1
    ts = _tensors([50], [F32])
    keep = ts[0].clone()
    fp8z.fp8z_grad_clip(fp8z.fp8z_encode_tensor_list(ts), math.inf, norm, ws)
    assert norm[1].item() == 1.0 and torch.equal(ts[0], keep)


def test_large_and_tiny_values(ws):
    """Squares near both ends of FP32: 1e18^2 is finite, 1e-18^2 is normal."""
    for v in (1e18, 1e-18):
        t = torch.full((70000,), v, device="cuda")
        norm = torch.zeros(2, device="cuda")
        fp8z.fp8z_grad_norm(fp8z.fp8z_encode_tensor_list([t]), norm, ws)
        want = float(t[0].double()) * math.sqrt(70000)
        assert abs(norm[0].item() - want) <= 10 * U * want


def test_other_stream_and_many_tensors(ws):
    s = torch.cuda.Stream()
    ts = _tensors([1 + (i * 37) % 9000 for i in range(700)], [F32, BF16], seed=9)
    dsts = [torch.empty(t.numel(), device="cuda") for t in ts]
    tl = fp8z.fp8z_encode_tensor_list(ts, dsts)
    norm = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        fp8z.fp8z_grad_clip(tl, 0.5, norm, ws)
    s.synchronize()
    _check(ts, dsts, ts, 0.5, 1.0, norm)


def test_more_than_2_31_elements(ws):
    n = 2 ** 31 + 4097
    t = torch.full((n,), 0.5, dtype=F16, device="cuda")
    t[-1] = 2.0
    norm = torch.zeros(2, device="cuda")
    fp8z.fp8z_grad_clip(fp8z.fp8z_encode_tensor_list([t]), 0.25 * math.sqrt(n), norm, ws)
    want = math.sqrt(0.25 * (n - 1) + 4.0)
    assert abs(norm[0].item() - want) <= 10 * U * want
    assert t[-1].item() == 1.0 and t[n // 2].item() == 0.25 and t[0].item() == 0.25


def test_graph_replay(ws):
    ts = _tensors([5000, 77, 20000], [F32, BF16], seed=1)
    dsts = [torch.empty(t.numel(), device="cuda") for t in ts]
    tl, norm = fp8z.fp8z_encode_tensor_list(ts, dsts), torch.zeros(2, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fp8z.fp8z_grad_clip(tl, 0.1, norm, ws)
    for k in (1.0, 3.0):
        for t in ts:
            t.mul_(k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _check(ts, dsts, ts, 0.1, 1.0, norm)


def test_refusals(ws):
    t = torch.zeros(64, device="cuda")
    norm = torch.zeros(2, device="cuda")
    with pytest.raises(ValueError):
        fp8z.fp8z_encode_tensor_list([t], [torch.zeros(63, device="cuda")])
    with pytest.raises(ValueError):
        fp8z.fp8z_encode_tensor_list([t.double()])
    with pytest.raises(ValueError):
        fp8z.fp8z_encode_tensor_list([t.view(8, 8).t()])
    with pytest.raises(ValueError):
        fp8z.fp8z_encode_tensor_list([t.cpu()])
    tl = fp8z.fp8z_encode_tensor_list([t])
    with pytest.raises(ValueError):
        fp8z.fp8z_grad_clip(tl, 1.0, norm[:1], ws)
    with pytest.raises(ValueError):
        fp8z.fp8z_grad_clip(tl, 1.0, norm, ws[:100])
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan)):
        with pytest.raises(fp8z.Fp8zError):
            fp8z.fp8z_grad_clip(tl, norm=norm, workspace=ws, **kw)
    with pytest.raises(fp8z.Fp8zError):
        fp8z.fp8z_grad_clip(tl, 1.0, norm, ws, grad_scale=math.inf)
