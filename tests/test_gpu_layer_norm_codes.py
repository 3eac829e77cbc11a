"""The codes that the norm of many rows writes are fp8z_quantize_rowwise's of its FP32 y, bit for bit.

Rows of +-1 in equal numbers with eps = 0 have mean 0 and rstd 1 exactly, so that y is the weight
with the row's signs: a test chooses the largest magnitude of every tile of 128 and the quotients beside it."""
import numpy as np
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

pytestmark = pytest.mark.gpu

f = np.float32
COLS, TILES = 8192, 64


def many_rows(odd):
    """More rows than two for every SM: the norm takes them through its queue."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count + 96 + odd


def compare(x, w, b, eps, pow2):
    rows, cols = x.shape
    y, q, s = torch.empty_like(x), torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, cols // 128, device="cuda")
    fp8z.fp8z_layer_norm(x, w, b, y, None, None, eps=eps, q=q, q_scale=s, pow2=pow2)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    fp8z.fp8z_quantize_rowwise(y, pow2, q2, s2)
    bad = (s != s2).nonzero()
    assert not len(bad), (len(bad), bad[0], s[tuple(bad[0])].item(), s2[tuple(bad[0])].item())
    bad = (q != q2).nonzero()
    assert not len(bad), (len(bad), bad[0], y[tuple(bad[0])].item(), s[bad[0][0], bad[0][1] // 128].item(), q[tuple(bad[0])].item(),
                          q2[tuple(bad[0])].item())
    return y, q, s


def signs(rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.ones(rows, COLS, device="cuda")
    order = torch.rand(rows, COLS, generator=g, device="cuda").argsort(1)
    return x.scatter_(1, order[:, :COLS // 2], -1.0)


def tile(rng, top, pow2):
    """128 numbers up to `top`: a spread of sizes, and quotients at and beside the middles between codes."""
    s = f(top) / f(448)
    if pow2:
        s = f(2.0 ** np.ceil(np.log2(float(s))))
    t = (f(top) * np.exp2(-rng.random(128) * 24).astype(f)).astype(f)
    mids = (rng.integers(16, 32, 96) / 16.0 * np.exp2(rng.integers(-10, 8, 96))).astype(f)
    near = (mids * s).astype(f)
    for _ in range(2):
        step = rng.integers(-1, 2, 96)
        near = np.where(step == 0, near, np.nextafter(near, np.where(step > 0, f(np.inf), f(0)))).astype(f)
    t[:96] = np.minimum(near, f(top))
    t[127] = top
    return rng.permutation(t)


def edge_tops():
    """448 * 2^j and its neighbours; the ends of the range whose quotients are corrected products, 2^-50 and 2^100;
    the smallest normal scale's; the smallest and largest numbers."""
    tops = []
    for j in (-140, -136, -135, -134, -133, -126, -59, -58, -20, -9, -1, 0, 1, 9, 60, 91, 92, 110, 118, 119):
        t = f(np.ldexp(448.0, j))
        tops += [np.nextafter(t, f(0)), t, np.nextafter(t, f(np.inf))]
    for t in (f(2.0 ** -50), f(2.0 ** 100), f(2.0 ** -126)):
        tops += [np.nextafter(t, f(0)), t, np.nextafter(t, f(np.inf))]
    return np.array([t for t in tops if t > 0] + [f(1e-45), np.finfo(f).max], f)


@pytest.mark.parametrize("pow2", [False, True])
def test_tiles_at_the_edges(pow2):
    rng = np.random.default_rng(1)
    tops = edge_tops()
    for i in range(0, len(tops), TILES):
        part = np.resize(tops[i:i + TILES], TILES)
        with np.errstate(over="ignore", under="ignore", invalid="ignore"):
            w = np.stack([tile(rng, t, pow2) for t in part])
        w[part == 0] = 0
        w = torch.from_numpy(np.nan_to_num(w, nan=0.0, posinf=0.0).reshape(-1)).cuda()
        x = signs(many_rows(i % 2), i)
        y, q, s = compare(x, w, None, 0.0, pow2)
        assert torch.equal(y, x * w)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_quotients_beside_the_middles(pow2, seed):
    rng = np.random.default_rng(seed)
    w = np.stack([tile(rng, f(rng.random() + 1) * f(np.exp2(rng.integers(-40, 90))), pow2) for _ in range(TILES)])
    compare(signs(many_rows(seed % 2), seed), torch.from_numpy(w.reshape(-1)).cuda(), None, 0.0, pow2)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows_odd,cols", [(0, 640), (1, 1280), (1, 7168), (396, 2048)])
def test_rows_of_all_sizes(rows_odd, cols, pow2):
    g = torch.Generator(device="cuda").manual_seed(cols)
    rows = many_rows(rows_odd)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(4 * torch.randn(rows, 1, generator=g, device="cuda"))
    w, b = (torch.randn(cols, generator=g, device="cuda") * torch.exp(6 * torch.randn(cols, generator=g, device="cuda")) for _ in range(2))
    w[128:256] = b[128:256] = 0.0
    w[384:512] *= 1e-30
    b[384:512] *= 1e-30
    y, q, s = compare(x, w, b, 1e-5, pow2)
    assert (s[:, 1] == 1.0).all() and (q[:, 128:256] & 127 == 0).all()
