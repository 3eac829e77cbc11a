"""fp8z_layer_norm and its gradient against their formulas in 64 bits.

Bounds.  u = 2^-24 is FP32's half step.  A sum of n numbers whose longest chain of additions
is c is off by at most c u times the sum of absolute values: a thread adds at most 32
columns (cols / 1024 in rows past the registers), the joins are 10 more.
  mean: e_m = (c + 1) u mean|x|;  d = x - mean: e_d = e_m + u |d|
  var:  mean(2 |d| e_d) + (c + 2) u var;  rstd: half of that relative to var + eps, and 4 u
  y:    |w| rstd (e_d + |d| e_rstd) + 4 u (|y| + |b|), and half a step of y's type
  dx:   rstd u (6 |g| + (c + 8) (mean|g| + |xh| mean|g xh|)), and half a step
  dw:   a chain of rows / 152 + 1 rows in a block, 38 + 8 parts, 8 warps: (that + 60) u sum|dy xh|
A q code is the nearest E4M3 value of y / s in FP32, and s off by 2 u: half a step of E4M3
(2^-4 of the value, 2^-10 for subnormals), and what y is off."""
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, shape, dtype, std=1.0, off=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + off).to(dtype)


def embed(t, pad, lead):
    """t in longer rows that start late; the rest is NaN."""
    rows, cols = t.shape
    raw = torch.full((lead + rows * (cols + pad),), float("nan"), dtype=t.dtype, device="cuda")
    v = raw[lead:].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def half_step(t, dtype):
    return 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2 * t.abs() * 1.01 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def chain(cols):
    return (32 if cols <= 32768 else cols // 1024 + 1) + 12


def run_forward(rows, cols, dtype, pdtype, weight=True, bias=True, y=True, q=False, pow2=False, pad=0, lead=0, eps=1e-5, seed=0,
                x=None):
    g = gen(seed)
    if x is None:
        x = rand(g, (rows, cols), dtype) * torch.exp(rand(g, (cols,), F32)).to(dtype) + rand(g, (rows, 1), dtype, 3.0)
    if pad or lead:
        x = embed(x, pad, lead)
    w = rand(g, (cols,), pdtype, 0.3, 1.0) if weight else None
    b = rand(g, (cols,), pdtype, 0.3) if bias else None
    out = embed(torch.zeros(rows, cols, dtype=dtype, device="cuda"), pad, lead) if y else None
    mean, rstd = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    codes = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda") if q else None
    scale = torch.zeros(rows, cols // 128, device="cuda") if q else None
    fp8z.fp8z_layer_norm(x, w, b, out, mean, rstd, eps=eps, q=codes, q_scale=scale, pow2=pow2)
    torch.cuda.synchronize()
    d64 = x.double()
    m64 = d64.mean(1, keepdim=True)
    d = d64 - m64
    var = d.square().mean(1, keepdim=True)
    r64 = 1.0 / (var + eps).sqrt()
    w64 = w.double() if weight else torch.ones(cols, dtype=torch.float64, device="cuda")
    b64 = b.double() if bias else torch.zeros(cols, dtype=torch.float64, device="cuda")
    want = d * r64 * w64 + b64
    c = chain(cols)
    e_m = (c + 1) * U * d64.abs().mean(1, keepdim=True)
    e_d = e_m + U * d.abs()
    e_r = ((2 * d.abs() * e_d).mean(1, keepdim=True) + (c + 2) * U * var) / (2 * (var + eps)) + 4 * U
    e_y = w64.abs() * r64 * (e_d + d.abs() * e_r) + 4 * U * (want.abs() + b64.abs())
    assert ((mean.double() - m64[:, 0]).abs() <= e_m[:, 0] + U * m64[:, 0].abs()).all()
    assert ((rstd.double() - r64[:, 0]).abs() <= (e_r * r64)[:, 0]).all()
    if y:
        bad = ~((out.double() - want).abs() <= e_y + half_step(want, dtype))
        assert not bad.any(), (out[bad][:4], want[bad][:4], bad.nonzero()[:4])
        if pad:
            around = torch.as_strided(out, (rows, cols + pad), (cols + pad, 1))[:-1, cols:]
            assert around.isnan().all(), "written behind a row"
    if q:
        s = scale.double()
        top = want.view(rows, -1, 128).abs().amax(-1)
        slack = e_y.view(rows, -1, 128).amax(-1)
        if pow2:
            assert (torch.frexp(scale).mantissa == 0.5).all()
            assert (s * 448.0 >= top - slack).all() and (s * 224.0 < top + slack).all()
        else:
            assert ((s - top / 448.0).abs() <= slack / 448.0 + 2 * U * s).all()
        got = codes.view(torch.float8_e4m3fn).double().view(rows, -1, 128) * s.unsqueeze(-1)
        t = want.view(rows, -1, 128)
        step = torch.maximum(t.abs() * 2.0 ** -4, s.unsqueeze(-1) * 2.0 ** -10)
        assert ((got - t).abs() <= step * (1 + 1e-5) + e_y.view(rows, -1, 128) * 1.1).all()
    return x, w, b, out, mean, rstd, codes, scale


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 256), (9, 255), (2, 1000), (33, 1024), (5, 1025), (400, 2001),
                                       (8, 4097), (700, 4096), (8, 7168), (310, 7168), (310, 7167), (4, 8193), (306, 12000),
                                       (700, 513), (701, 2001), (650, 8176), (650, 8177), (641, 4099), (2, 32768), (3, 32769), (2, 70001)])
def test_forward(rows, cols):
    for i, (dt, pt) in enumerate(((BF16, F32), (F16, F16), (F32, F32), (BF16, BF16))):
        run_forward(rows, cols, dt, pt, weight=i != 2 or cols % 2 == 0, bias=i % 2 == 0, seed=i)


@pytest.mark.parametrize("pad,lead", [(8, 8), (1, 0), (3, 5), (0, 1)])
@pytest.mark.parametrize("rows,cols", [(5, 200), (3, 1000), (400, 4104), (4, 9000), (700, 1003)])
def test_forward_strides(rows, cols, pad, lead):
    run_forward(rows, cols, BF16, F32, pad=pad, lead=lead)
    run_forward(rows, cols, F32, F32, pad=pad, lead=lead)


@pytest.mark.parametrize("rows,cols", [(1, 128), (40, 256), (3, 896), (7, 1152), (320, 2048), (6, 7168), (320, 7168), (2, 16384),
                                       (2, 33024)])
@pytest.mark.parametrize("pow2", [False, True])
def test_forward_codes(rows, cols, pow2):
    for i, (dt, pt) in enumerate(((BF16, F32), (F16, F16), (F32, F32))):
        run_forward(rows, cols, dt, pt, q=True, y=i == 1, pow2=pow2, seed=i)


@pytest.mark.parametrize("pow2", [False, True])
def test_codes_are_the_quantizer_s(pow2):
    """q of an FP32 norm is what fp8z_quantize_rowwise makes of y, bit for bit; tiles of zeros among them."""
    g = gen(3)
    rows, cols = 300, 1280
    x = rand(g, (rows, cols), F32)
    w = rand(g, (cols,), F32)
    w[128:256] = 0.0
    w[300] = 0.0
    w[640:768] *= 1e-30
    y, q, s = torch.empty_like(x), torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, cols // 128, device="cuda")
    fp8z.fp8z_layer_norm(x, w, None, y, None, None, q=q, q_scale=s, pow2=pow2)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    fp8z.fp8z_quantize_rowwise(y, pow2, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert (s[:, 1] == 1.0).all() and (q[:, 128:256] & 127 == 0).all()


def test_constant_rows_and_offsets():
    x = torch.full((4, 1000), 3.0, device="cuda")
    x[1] = 1e4
    x[2] = 0.0
    x[3] = torch.arange(1000, device="cuda") * 1e-3 + 1000.0
    run_forward(4, 1000, F32, F32, x=x)
    y = torch.empty_like(x)
    fp8z.fp8z_layer_norm(x, None, None, y, None, None)
    assert (y[:3] == 0.0).all()
    x[0, 5], x[1, 7] = float("nan"), float("inf")
    fp8z.fp8z_layer_norm(x, None, None, y, None, None)
    assert y[0].isnan().all() and y[1].isnan().any() and y[2:].isfinite().all()


def run_gradient(rows, cols, dtype, pdtype, weight=True, bias=True, accumulate=False, pad=0, lead=0, seed=0, dx=True):
    g = gen(seed)
    x, dy = rand(g, (rows, cols), dtype, 1.0, 0.5), rand(g, (rows, cols), dtype, 0.01)
    w = rand(g, (cols,), pdtype, 0.3, 1.0) if weight else None
    d = x.double()
    mean = d.mean(1).float()
    rstd = (1.0 / ((d - mean.double()[:, None]).square().mean(1) + 1e-5).sqrt()).float()
    out = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    if pad or lead:
        x, dy, out = embed(x, pad, lead), embed(dy, pad, lead), embed(out, pad, lead)
    dw, db = rand(g, (cols,), pdtype, 0.1), rand(g, (cols,), pdtype, 0.1)
    dw0, db0 = dw.double(), db.double()
    ws = torch.full((fp8z.fp8z_layer_norm_grad_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    fp8z.fp8z_layer_norm_grad(dy, x, w, mean, rstd, out if dx else None, dw if weight else None, db if bias else None, ws,
                              accumulate=accumulate)
    torch.cuda.synchronize()
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    gd = dy.double() * (w.double() if weight else 1.0)
    r = rstd.double()[:, None]
    if rows:
        want = r * (gd - gd.mean(1, keepdim=True) - xh * (gd * xh).mean(1, keepdim=True))
        bound = r * U * (6 * gd.abs() + (chain(cols) + 8) * (gd.abs().mean(1, keepdim=True) + xh.abs() * (gd * xh).abs().mean(1, keepdim=True)))
        if dx:
            bad = ~((out.double() - want).abs() <= bound + half_step(want, dtype))
            assert not bad.any(), (out[bad][:4], want[bad][:4], bad.nonzero()[:4])
    if pad and rows > 1:
        assert torch.as_strided(out, (rows, cols + pad), (cols + pad, 1))[:-1, cols:].isnan().all(), "written behind a row"
    c = rows // 152 + 61
    for got, start, terms, there in ((dw, dw0, dy.double() * xh, weight), (db, db0, dy.double(), bias)):
        base = start if accumulate or not there else torch.zeros_like(start)
        if not there:
            assert torch.equal(got.double(), start)
            continue
        want = base + terms.sum(0)
        bound = (c + 3) * U * terms.abs().sum(0) + 2 * U * want.abs()
        bad = ~((got.double() - want).abs() <= bound + half_step(want, pdtype))
        assert not bad.any(), (got[bad][:4], want[bad][:4], bad.nonzero()[:4])


@pytest.mark.parametrize("rows,cols", [(0, 64), (1, 1), (3, 7), (100, 256), (9, 512), (2600, 500), (5, 513), (1021, 2001), (700, 2048),
                                       (8, 4097), (700, 4096), (310, 7168), (310, 7167), (4, 8193), (306, 12000), (2, 32768),
                                       (3, 32769), (160, 40000),
                                       (4001, 513), (3700, 2001), (3650, 8175), (4100, 519), (4100, 1000)])
def test_gradient(rows, cols):
    for i, (dt, pt) in enumerate(((BF16, F32), (F16, F16), (F32, F32), (BF16, BF16))):
        run_gradient(rows, cols, dt, pt, weight=i != 2 or cols % 2 == 0, bias=i % 2 == 0, accumulate=i in (0, 3), seed=i, dx=i != 3)


@pytest.mark.parametrize("pad,lead", [(8, 8), (1, 0), (3, 5), (0, 1)])
@pytest.mark.parametrize("rows,cols", [(5, 200), (3, 1000), (400, 4104), (4, 9000), (3700, 1003)])
def test_gradient_strides(rows, cols, pad, lead):
    run_gradient(rows, cols, BF16, F32, pad=pad, lead=lead)
    run_gradient(rows, cols, F32, F32, pad=pad, lead=lead, accumulate=True)


def test_gradient_against_differences():
    """The sum of c * y over one row, stepped along each column: central differences in FP32 inputs,
    64-bit sums.  A step of 2^-6 leaves a truncation of h^2 / 6 times the third derivative (under 30 here)
    and FP32 noise of 40 u sum|c y| / h."""
    g = gen(9)
    cols, h = 48, 2.0 ** -6
    x, w, b, c = (rand(g, (cols,), F32) for _ in range(4))
    rows = torch.cat([x + s * h * torch.eye(cols, device="cuda") for s in (1.0, -1.0)])
    y = torch.empty_like(rows)
    fp8z.fp8z_layer_norm(rows, w, b, y, None, None)
    loss = (y.double() * c.double()).sum(1)
    diff = (loss[:cols] - loss[cols:]) / ((rows[:cols] - rows[cols:]).double().sum(1))
    one = x[None].contiguous()
    mean, rstd, yy, dx = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(one), torch.empty_like(one)
    fp8z.fp8z_layer_norm(one, w, b, yy, mean, rstd)
    ws = torch.empty(fp8z.fp8z_layer_norm_grad_workspace(1, cols), dtype=torch.uint8, device="cuda")
    fp8z.fp8z_layer_norm_grad(c[None].contiguous(), one, w, mean, rstd, dx, None, None, ws)
    noise = 40 * U * (yy.double() * c.double()).abs().sum() / h
    assert ((dx[0].double() - diff).abs() <= h * h * 5 + noise).all()


def test_same_bits_every_time():
    g = gen(4)
    rows, cols = 2999, 1536
    x, dy, w = rand(g, (rows, cols), BF16), rand(g, (rows, cols), BF16), rand(g, (cols,), F32)
    mean, rstd = x.float().mean(1), 1.0 / x.float().std(1)
    first = None
    for _ in range(4):
        dw, db, dx = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty_like(x)
        ws = torch.empty(fp8z.fp8z_layer_norm_grad_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        fp8z.fp8z_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, ws)
        got = [t.clone() for t in (dw, db, dx)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


@pytest.mark.parametrize("rows,cols", [(3, 1024), (700, 1024), (701, 2001), (2, 40000)])
def test_squares_that_overflow(rows, cols):
    """Values of 1e25: their squares are infinite in FP32, rstd is 0 and y the bias, whichever way the rows go."""
    g = gen(9)
    x = (torch.randn(rows, cols, generator=g, device="cuda").sign() * 1e25).to(BF16)
    b = rand(g, (cols,), F32)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    fp8z.fp8z_layer_norm(x, None, b, y, mean, rstd)
    assert (rstd == 0).all() and torch.equal(y, b.to(BF16).expand(rows, cols))
