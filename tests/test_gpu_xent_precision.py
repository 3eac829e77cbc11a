"""What the cross entropy keeps of small losses and probabilities, against 64 bits.

The inputs have two columns for each token t, so that every logit is one that FP32
holds exactly: x[t] is A_t and g, w[v] 1 and -k, hence l[t][v] = A_t - g k[t][v], and
the largest logit is A_t.  With exact logits the error is the softmax's own and does
not grow with A: l - max is exact; its product with log2(e) (within 2^-26) is within
1.25 * 2^-24 of itself, so that an exponential of -G is within r = 2^-22 + 1.25 G 2^-24
of itself, three times that after a partial sum's and a row's rescaling.  The sum s >= 1
of the exponentials collects one 2^-24 for each addition on a term's way: 16 of a chain,
2 to join chains, 4 segments, 8 + 1 tiles of a thread, 5 of a warp: under 40.  logf is
within an ulp."""
import math

import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
UNIT = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
V = 1000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    fp8z.lib()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _exact_logits(n, kind, dtype, odd, top):
    """(x, w, targets, A, g k as float64 [n, V]) with rows of 2 n (+ 1) columns."""
    gen = _gen(n)
    h = 2 * n + (1 if odd else 0)
    a = ((torch.rand(n, generator=gen, device="cuda") * 1.98 - 0.99) * top).to(dtype)
    t = torch.randint(0, V, (n,), generator=gen, device="cuda")
    if kind == "confident":          # the target is above all other words by g
        g = torch.tensor([6.0, 17.0, 40.0], device="cuda")[torch.arange(n, device="cuda") % 3]
        k = torch.ones(n, V, device="cuda")
        k.scatter_(1, t[:, None], 0.0)
    else:                            # the largest logit anywhere, the target anywhere
        g = torch.full((n,), 2.5, device="cuda")
        k = torch.randint(1, 65, (n, V), generator=gen, device="cuda") / 8.0
        k.scatter_(1, torch.randint(0, V, (n, 1), generator=gen, device="cuda"), 0.0)
    x = torch.zeros(n, h, dtype=dtype, device="cuda")
    w = torch.zeros(V, h, dtype=dtype, device="cuda")
    i = torch.arange(n, device="cuda")
    x[i, 2 * i], x[i, 2 * i + 1] = a, g.to(dtype)
    w[:, 0:2 * n:2] = 1.0
    w[:, 1:2 * n:2] = -k.t().to(dtype)
    return x, w, t, a.double(), g.double()[:, None] * k.double()


@pytest.mark.parametrize("n", [3, 20, 40])
@pytest.mark.parametrize("kind", ["confident", "spread"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("odd,piece", [(False, 0), (True, 0), (False, 256)])
@pytest.mark.parametrize("top", [1.0, 4000.0])
def test_small_losses_of_large_logits(n, kind, dtype, odd, piece, top):
    x, w, t, a, gk = _exact_logits(n, kind, dtype, odd, top)
    e = torch.exp(-gk)
    s = e.sum(1)
    own = gk.gather(1, t[:, None])[:, 0]
    tail = s - 1.0
    # log1p keeps a loss of 1e-15
    want = torch.log1p(torch.where(own == 0.0, (e.scatter(1, t[:, None], 0.0)).sum(1), tail)) + own
    r = 3 * (2.0 ** -22 + 1.25 * float(gk.max()) * 2.0 ** -24)
    ds = 40 * 2.0 ** -24 * s + r * tail                     # on s
    bound = ds / s + 2.0 ** -22 * want
    loss, lse, total = (torch.full((k,), math.nan, device="cuda") for k in (n, n, 2))
    ws = torch.full((fp8z.fp8z_linear_xent_workspace(x, w),), 255, dtype=torch.uint8, device="cuda")
    fp8z.fp8z_linear_xent(x, w, t, loss, total, ws, lse=lse, reduction="sum")
    assert bool((loss >= 0).all())
    assert bool(((loss.double() - want).abs() <= bound).all())
    assert bool(((lse.double() - (a + torch.log(s))).abs() <= ds / s + 2.0 ** -22 * torch.log(s) + 2.0 ** -24 * (a.abs() + 8)).all())

    dx = torch.empty_like(x)
    dw = torch.full((V, x.shape[1]), math.nan, device="cuda")
    ws = torch.full((fp8z.fp8z_linear_xent_workspace(x, w, dw=dw, piece_words=piece),), 255, dtype=torch.uint8, device="cuda")
    first = loss.clone()
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum")
    if x.shape[1] % 8 == 0:          # else the loss of few tokens reads w where it is, in another order
        assert torch.equal(first, loss)
    assert bool((loss >= 0).all()) and bool(((loss.double() - want).abs() <= bound).all())
    # dw[v][2 t] = A_t P[t][v]: one product, so P itself is seen
    p = e / s[:, None]
    at_target = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
    P = torch.where(at_target.bool() & (own == 0.0)[:, None], -((s - e.gather(1, t[:, None])[:, 0]) / s)[:, None].expand_as(p), p - at_target)
    got = dw[:, 0:2 * n:2].t().double() / torch.where(a == 0.0, torch.ones_like(a), a)[:, None]
    err = p * (ds / s + r)[:, None] + 2.0 ** -23 * at_target               # and 1 subtracted
    # P leaves in two parts of dtype (FP16 counts in 2^-36 at the least), the product and dw round
    tol = err + P.abs() * (UNIT[dtype] ** 2 + 2.0 ** -22) + (2.0 ** -37 if dtype == F16 else 0.0)
    ok = (got - P).abs() <= tol
    assert bool(ok[a != 0.0].all())


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_dx_of_a_large_vocabulary(n, dtype):
    """x = 0: every logit is 0 and P = 2^-22, exact in both types.  w lies between 0.5 and
    1.5, so that dx = mean(w) - w_y adds up to 1 before the target's row of ones, the last,
    takes nearly all of it away: what was cut off on the way stays.  At most 64 blocks of 64
    words, 256 steps, are added up in tensor memory, each cutting off 2^-23 of the sum; 16 sums
    in registers, 64 parts and the last steps round by 2^-24.  P of the target is 1 less 2^-22."""
    v, h = 1 << 22, 64
    w = torch.empty(v, h, dtype=dtype, device="cuda").uniform_(0.5, 1.5, generator=_gen(1))
    w[-1] = 1.0
    x = torch.zeros(n, h, dtype=dtype, device="cuda")
    t = torch.full((n,), v - 1, device="cuda")
    loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum")
    want = w.double().mean(0) - 1.0
    tol = 256 * 2.0 ** -23 + (16 + 64 + 8) * 2.0 ** -24 + 2.0 ** -22 + want.abs() * UNIT[dtype] + 2.0 ** -25
    assert bool(((dx.double() - want).abs() <= tol).all())


def test_16_bit_dw_of_many_tokens():
    """w = 0: P = 2^-8 for every word that is not a target, and its row of dw is the sum of
    x, between 0.5 and 1.5, over 2^18 tokens, times 2^-8.  The roundings to FP16 (2^-11 at the
    most, 2^-12 in the mean square) have no sign, and over 512 columns their mean is within
    6 * 2^-12 / sqrt(512); what sums cut off has one: 256 steps of 2^-23, and 64 sums that round."""
    n, h, v = 1 << 18, 512, 256
    x = torch.empty(n, h, dtype=F16, device="cuda").uniform_(0.5, 1.5, generator=_gen(2))
    w = torch.zeros(v, h, dtype=F16, device="cuda")
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum")
    want = x.double().sum(0) / 256
    off = (dw[1:].double() - want) / want
    assert bool((off.abs() <= 2.0 ** -11 + 256 * 2.0 ** -23 + 64 * 2.0 ** -24).all())
    assert abs(float(off.mean())) <= 6 * 2.0 ** -12 / math.sqrt(h) + 256 * 2.0 ** -23 + 64 * 2.0 ** -24


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("piece", [0, 256])
def test_small_probabilities_in_fp16(n, piece):
    """Words 14 to 24 below the largest logit: probabilities of 2^-20 to 2^-35.  An FP32 dw
    gets them in two FP16 parts, 22 bits, of which those of 2^-39 count: half of that is lost.
    The exponential and the sum are as in the bounds above."""
    x, w, t, a, _ = _exact_logits(n, "spread", F16, False, 4000.0)
    k = torch.randint(46, 77, (n, V), generator=_gen(n), device="cuda") / 8.0
    k.scatter_(1, t[:, None], 0.0)
    w[:, 1:2 * n:2] = -k.t().to(F16)
    gk = 2.5 * k.double()
    e = torch.exp(-gk)
    s = e.sum(1)
    loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(V, x.shape[1], device="cuda")
    ws = torch.empty(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw, piece_words=piece), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum")
    p = (e / s[:, None]).scatter(1, t[:, None], 0.0)
    got = (dw[:, 0:2 * n:2].t().double() / a[:, None]).scatter(1, t[:, None], 0.0)
    r = 3 * (2.0 ** -22 + 1.25 * 24.0 * 2.0 ** -24)
    tol = p * (r + (40 + 2) * 2.0 ** -24 + 2 * 2.0 ** -22) + 2.0 ** -40
    assert bool(((got - p).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [4096, 65536 + 197])
def test_fp32_dw_is_added_up_in_short_sums(n, dtype):
    """As above with an FP32 dw: 8 blocks of K, 32 steps for each of P's two parts, may cut
    off 2^-23 of their sum, and every sum rounds once when it is added, as dw does at the end.
    One sum of all tokens would cut off 4096 steps of the larger case, 5e-4 at the most."""
    h, v = 136, 256
    x = torch.empty(n, h, dtype=dtype, device="cuda").uniform_(0.5, 1.5, generator=_gen(3))
    w = torch.zeros(v, h, dtype=dtype, device="cuda")
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(v, h, device="cuda")
    ws = torch.empty(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum")
    want = x.double().sum(0) / 256
    sums = -(-n // 512)
    bound = 64 * 2.0 ** -23 + (sums + 1) * 2.0 ** -24
    assert bool(((dw[1:].double() - want).abs() <= bound * want).all())
    # the target's row: 255 / 256 in two parts of dtype, taken away
    want = -x.double().sum(0) * (255 / 256)
    assert bool(((dw[0].double() - want).abs() <= (bound + UNIT[dtype] ** 2) * want.abs()).all())


def test_more_tokens_than_2_to_23():
    """An FP32 dw over 131074 blocks of K, in sums of 8.  w = 0, every target word 0: P is 2^-8,
    or 2^-8 - 1, and x whole numbers of -2 to 2, so that every sum is one that FP32 holds: equal."""
    n, h, v = (1 << 23) + 130, 64, 256
    x = torch.randint(-2, 3, (n, h), generator=_gen(5), device="cuda", dtype=torch.int8).to(BF16)
    w = torch.zeros(v, h, dtype=BF16, device="cuda")
    t = torch.zeros(n, dtype=torch.int32, device="cuda")
    loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(v, h, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(fp8z.fp8z_linear_xent_workspace(x, w, dw=dw), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, reduction="sum", dev_status=status)
    assert status.item() == 0 and not dx.any() and total[1].item() == n
    s = torch.stack([part.double().sum(0) for part in x.split(1 << 20)]).sum(0)
    assert torch.equal(dw[1:].double(), (s / 256).expand(v - 1, h))
    assert torch.equal(dw[0].double(), s / 256 - s)
