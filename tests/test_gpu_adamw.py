"""fp8z_adamw.  FP32 moments: bit for bit, operation by operation in FP32 on the host, and the
oracle's step.  8-bit moments: the same but that a root and a quotient may be off by one unit.
Against the host's FP32 step from the same state, u = 2^-24:
  m' the same; r = sqrt(v') by 2 u of itself;
  the update by 12 u of itself (r, two of d, the quotient, the product), p by that and 2 u;
  scales by what their largest element is off and 4 u, and a code by what moves a value across the middle
  between two codes: one step, for few.
Both against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
f = np.float32


def scalars(hp):
    b1, b2, lr, wd = (hp.given[k] for k in ("beta1", "beta2", "lr", "weight_decay"))       # not rounded to 32 bits
    c1, c2 = 1.0 - b1 ** hp.step, 1.0 - b2 ** hp.step
    return dict(b1=f(b1), b2=f(b2), omb1=f(1 - b1), omb2=f(1 - b2), eps=f(hp.eps), size=f(lr / c1), rs=f(1 / np.sqrt(c2)),
                decay=f(1 - lr * wd), lr_wd=f(lr * wd), post=hp.decay_mode == fp8z.FP8Z_DECAY_POST)


def value(codes):
    return torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).float().numpy()


def encode(x):
    return torch.from_numpy(x.copy()).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def tiles(x):
    return np.pad(x, (0, -x.size % 128)).reshape(-1, 128)


def quantize(x, keep):
    t = tiles(x)
    top = np.fmax.reduce(np.abs(t), axis=1, initial=0)           # a NaN is never the largest
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        s = np.where(top == 0, f(1), np.minimum(f(448) * (f(1) / top), np.finfo(f).max)).astype(f)
        q = encode(t * s[:, None])
        if keep:
            q = np.where((t > 0) & (q == 0), np.uint8(1), q)
        return q.reshape(-1)[:x.size], (f(1) / s).astype(f)


def host_step(t, hp, factor):
    """t: dict of numpy arrays p, g (float32), m, v, and for 8 bits m_scale, v_scale."""
    c = scalars(hp)
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        g = t["g"] * f(factor)
        if "m_scale" in t:
            m = value(t["m"]) * np.repeat(t["m_scale"], 128)[:g.size]
            v = value(t["v"]) * np.repeat(t["v_scale"], 128)[:g.size]
            v = v * v
        else:
            m, v = t["m"], t["v"]
        m = c["b1"] * m + c["omb1"] * g
        v = c["b2"] * v + c["omb2"] * (g * g)
        r = np.sqrt(v)
        su = c["size"] * (m / (r * c["rs"] + c["eps"]))
        if c["post"]:
            p = t["p"] - su
            p = p - c["lr_wd"] * p
        else:
            p = t["p"] * c["decay"] - su
    out = {"p": p}
    if "m_scale" in t:
        out["m"], out["m_scale"] = quantize(m, False)
        out["v"], out["v_scale"] = quantize(r, True)
    else:
        out["m"], out["v"] = m, v
    return out


def make(n, gtype, bits, copy, seed, wide=False, lead=0):
    rng = np.random.default_rng(seed)
    spread = np.exp(rng.normal(size=n) * (6 if wide else 1))
    t = {"p": (rng.normal(size=n) * 0.02).astype(f), "g": (rng.normal(size=n) * 1e-3 * spread).astype(f)}
    g16 = torch.from_numpy(t["g"]).to(gtype)
    t["g"] = g16.float().numpy()
    m, v = (rng.normal(size=n) * 2e-4 * spread).astype(f), (rng.random(n) * 4e-7 * spread ** 2).astype(f)
    if n > 600:
        m[128:256] = v[128:256] = 0.0
        m[300], v[300] = 0.0, 0.0
    if bits == 8:
        t["m"], t["m_scale"] = quantize(m, False)
        t["v"], t["v_scale"] = quantize(np.sqrt(v), True)
    else:
        t["m"], t["v"] = m, v

    def dev(x, at=lead):
        x = torch.as_tensor(x)
        raw = torch.full((x.numel() + at + 5,), 77, dtype=x.dtype, device="cuda")
        raw[at:at + x.numel()] = x.cuda()
        return raw[at:at + x.numel()]
    d = {k: dev(x) for k, x in t.items() if k != "g"}
    d["g"] = dev(g16)
    d["copy"] = dev(torch.zeros(n, dtype=copy)) if copy else None
    return t, d


def lists(ds, **kw):
    return fp8z.fp8z_encode_adamw_list([d["p"] for d in ds], [d["g"] for d in ds], [d["m"] for d in ds], [d["v"] for d in ds],
                                       copies=[d["copy"] for d in ds], exp_avg_scales=[d.get("m_scale") for d in ds],
                                       exp_avg_sq_scales=[d.get("v_scale") for d in ds], **kw)


def bits_of(x):
    """Bit patterns, all NaN alike (of a half-precision gradient that overflowed, and of what it reaches)."""
    x = x if isinstance(x, np.ndarray) else x.cpu().numpy()
    if x.dtype == f:
        return np.where(np.isnan(x), np.uint32(0x7FC00000), x.view(np.uint32))
    return np.where((x & 127) == 127, np.uint8(127), x)


def compare(ds, want):
    for i, (d, w) in enumerate(zip(ds, want)):
        for k, x in w.items():
            assert np.array_equal(bits_of(d[k]), bits_of(x)), (i, k, np.flatnonzero(bits_of(d[k]) != bits_of(x))[:5])
        if d["copy"] is not None:
            assert torch.equal(torch.nan_to_num(d["copy"]), torch.nan_to_num(d["p"].to(d["copy"].dtype)))


def around(ds):
    for d in ds:
        for t in d.values():
            if t is not None:
                whole = torch.as_strided(t, (t.storage_offset() + t.numel() + 5,), (1,), 0)
                assert (whole[t.storage_offset() + t.numel():] == 77).all() and (whole[:t.storage_offset()] == 77).all()


def close(d, w, before, hp, factor):
    """One step with 8-bit moments from the state `before`: d (device) against w (host_step)."""
    got = {k: d[k].cpu().numpy() for k in ("p", "m", "v", "m_scale", "v_scale")}
    u, c, n = 2.0 ** -24, scalars(hp), before["p"].size
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        g = np.abs(before["g"].astype(np.float64)) * factor
        m = np.abs(value(before["m"]).astype(np.float64)) * np.repeat(before["m_scale"], 128)[:n]
        v = (value(before["v"]).astype(np.float64) * np.repeat(before["v_scale"], 128)[:n]) ** 2
        em = 2 * u * (float(c["b1"]) * m + float(c["omb1"]) * g)
        r = np.sqrt(float(c["b2"]) * v + float(c["omb2"]) * g * g)
        upd = float(c["size"]) * em / (2 * u) / (r * float(c["rs"]) + float(c["eps"]))
        p = w["p"].astype(np.float64)
        off = np.abs(got["p"].astype(np.float64) - p) <= 14 * u * upd + 2 * u * (np.abs(p) + np.abs(before["p"]))
        assert (off | (np.isnan(got["p"]) & np.isnan(w["p"])) | (got["p"] == w["p"])).all(), np.flatnonzero(~off)[:5]
        for k, e in (("m", 0.0 * tiles(em).max(1)), ("v", 2 * u * tiles(r).max(1) / 448.0)):
            a, b = got[k + "_scale"].astype(np.float64), w[k + "_scale"].astype(np.float64)
            finite = np.isfinite(b) & np.isfinite(e)         # of a run with an infinity or NaN nothing is asked
            assert np.isfinite(a[finite]).all(), k
            assert (np.abs(a - b)[finite] <= (e + 4 * u * b)[finite]).all(), k
            keep = np.repeat(finite, 128)[:n]
            x, y = value(got[k]).astype(np.float64)[keep], value(w[k]).astype(np.float64)[keep]
            apart = ~((x == y) | (np.isnan(x) & np.isnan(y)))
            step = np.maximum(np.abs(x), np.abs(y)) * 2.0 ** -3 * 1.001
            assert (np.abs(x - y)[apart] <= np.maximum(step[apart], 2.0 ** -9)).all(), k
            # a value crosses a middle, 2^-4 of its size away from the next, by 2^-20 of it: 1 in 2^16, by far
            assert apart.sum() <= 3 + apart.size / 2.0 ** 14, (k, int(apart.sum()), apart.size)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("gtype,copy,factor,step,post", [(F32, None, None, 1, 0), (BF16, BF16, 0.37, 11, 1), (F16, F16, 0.125, 1000, 0)])
@pytest.mark.parametrize("lead", [0, 1, 4])
def test_bits(bits, gtype, copy, factor, step, post, lead):
    """Tensors of every kind of length in one list, aligned and not, dense and spread over many binades."""
    sizes = [0, 1, 3, 127, 128, 129, 1000, 8191, 8192, 8193, 40000, 131072 + 5]
    pairs = [make(n, gtype, bits, copy, 10 * i + step, wide=i % 2 == 1, lead=lead) for i, n in enumerate(sizes)]
    hp = fp8z.hparams(lr=3e-4, step=step, decay_mode=post)
    ds = [d for _, d in pairs]
    table = lists(ds)
    fac = None if factor is None else torch.full((1,), factor, device="cuda")
    state = [t for t, _ in pairs]
    for _ in range(3):
        fp8z.fp8z_adamw(table, hp, grad_factor=fac)
        torch.cuda.synchronize()
        want = [host_step(t, hp, 1.0 if factor is None else factor) for t in state]
        if bits == 32:
            compare(ds, want)
        else:
            for d, w, t in zip(ds, want, state):
                if t["p"].size:
                    close(d, w, t, hp, 1.0 if factor is None else factor)
        # the next step starts from what the device holds
        state = [dict({k: d[k].cpu().numpy() for k in w}, g=t["g"]) for d, w, t in zip(ds, want, state)]
    for d in ds:
        if d["copy"] is not None:
            assert torch.equal(torch.nan_to_num(d["copy"]), torch.nan_to_num(d["p"].to(d["copy"].dtype)))
    around(ds)


def test_mixed_list():
    kinds = [(F32, 32, None), (BF16, 8, F16), (F16, 32, BF16), (F32, 8, None)]
    pairs = [make(3000 + 7 * i, g, b, c, i, lead=i) for i, (g, b, c) in enumerate(kinds)]
    hp = fp8z.hparams(step=4)
    fp8z.fp8z_adamw(lists([d for _, d in pairs]), hp)
    torch.cuda.synchronize()
    for (t, d), (_, bits, _) in zip(pairs, kinds):
        if bits == 32:
            compare([d], [host_step(t, hp, 1.0)])
        else:
            close(d, host_step(t, hp, 1.0), t, hp, 1.0)


@pytest.mark.parametrize("post", [0, 1])
def test_fp32_moments_are_the_step_s(oracle, post):
    t, d = make(3 * 16384, F32, 32, None, 5)
    hp = fp8z.hparams(step=7, decay_mode=post)
    hp.given = {}                                              # the 32-bit numbers, as the step takes them
    o = {k: x.copy() for k, x in t.items()}
    oracle.adamw_requant_step(o["p"], o["g"], o["m"], o["v"], np.zeros(3 * 16384, np.uint8), np.zeros(3, f), 0, 3,
                              oracle.Hparams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, hp.step, hp.fp8_max, hp.min_scale,
                                             hp.scale_mode, hp.decay_mode))
    fp8z.fp8z_adamw(lists([d]), hp)
    torch.cuda.synchronize()
    compare([d], [{k: o[k] for k in "pmv"}])


@pytest.mark.parametrize("bits", [8, 32])
def test_formula(bits):
    """64 bits: the update is off by at most 12 roundings of its factors, p by two more of its own size."""
    t, d = make(50000, BF16, bits, None, 8)
    hp = fp8z.hparams(lr=1e-2, step=3)
    b1, b2, lr, wd, eps = (hp.given[k] for k in ("beta1", "beta2", "lr", "weight_decay", "eps"))
    m, v = t["m"].astype(np.float64), t["v"].astype(np.float64)
    if bits == 8:
        m = value(t["m"]).astype(np.float64) * np.repeat(t["m_scale"], 128)[:m.size]
        v = (value(t["v"]).astype(np.float64) * np.repeat(t["v_scale"], 128)[:v.size]) ** 2
    g = t["g"].astype(np.float64)
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    size = b1 * np.abs(m) + (1 - b1) * np.abs(g)               # m' may cancel
    den = np.sqrt(v1 / (1 - b2 ** 3)) + eps
    u = lr / (1 - b1 ** 3) / den
    p = t["p"] * (1 - lr * wd) - u * m1
    fp8z.fp8z_adamw(lists([d]), hp)
    got = d["p"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - p) <= 2.0 ** -24 * (12 * u * size + 3 * np.abs(t["p"]) + np.abs(p))).all()
    if bits == 8:
        for key, x in (("m", m1), ("v", np.sqrt(v1))):
            s = np.repeat(d[key + "_scale"].cpu().numpy().astype(np.float64), 128)[:x.size]
            back = value(d[key].cpu().numpy()).astype(np.float64) * s
            half = np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) if key == "m" else np.maximum(x * 2.0 ** -4, s * 2.0 ** -9)
            assert (np.abs(back - x) <= half * 1.0001 + 2.0 ** -20 * np.abs(x).max()).all()


def test_small_v_stays_above_zero_and_extremes():
    """One element of a run far above the others: their v keeps the smallest code and the next step is bounded."""
    n = 256
    t, d = make(n, F32, 8, None, 1)
    for k in ("m", "v"):
        t[k][:] = 0
        t[k + "_scale"][:] = 1.0
        d[k].zero_()
        d[k + "_scale"].fill_(1.0)
    t["g"][:] = 1e-6
    t["g"][5] = 1e3
    t["g"][128:] = 0.0
    t["g"][130] = 1e-42
    d["g"].copy_(torch.from_numpy(t["g"]))
    table = lists([d])
    for step in (1, 2):
        hp = fp8z.hparams(lr=1e-3, step=step, weight_decay=0.0)
        before = {k: d[k].cpu().numpy() for k in ("p", "g", "m", "v", "m_scale", "v_scale")}
        fp8z.fp8z_adamw(table, hp)
        torch.cuda.synchronize()
        close(d, host_step(before, hp, 1.0), before, hp, 1.0)
        d["g"].zero_()
    assert (d["v"][:128] > 0).all() and (d["v"][131:] == 0).all()
    assert torch.isfinite(d["p"]).all() and (np.abs(d["p"].cpu().numpy() - t["p"]) <= 1e-2).all()


def test_zero_factor_and_lost_step():
    t, d = make(2000, F32, 32, None, 2)
    t["g"][3] = np.inf
    d["g"].copy_(torch.from_numpy(t["g"]))
    fp8z.fp8z_adamw(lists([d]), fp8z.hparams(step=2), grad_factor=torch.zeros(1, device="cuda"))
    got = d["p"].cpu().numpy()
    assert np.isnan(got[3]) and np.isfinite(np.delete(got, 3)).all()


def test_list_is_empty():
    fp8z.fp8z_adamw(lists([]), fp8z.hparams())
    t, d = make(0, F32, 8, None, 2)
    fp8z.fp8z_adamw(lists([d]), fp8z.hparams())
