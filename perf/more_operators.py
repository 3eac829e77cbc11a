"""Timed cases of the operators that use and make what the FP8 optimizer step
writes: the product of row-wise quantized activations with blockwise E4M3
weights (a dense layer and a bank of experts, forward, input gradient and weight
gradient), layer norm with an optional row-wise E4M3 output and its gradient, and
AdamW over the many tensors that are not kept in FP8 blocks, with moments in 32 or
in 8 bits.

Every case is a dict of plain values.  `prepare` makes what a training or serving
program has in hand before the call, `run` makes one pass, `exact` computes the
same outputs from the definitions in 64 bits, and `work` counts the bytes and
operations a pass cannot do without.  With `own` false `run` computes the plain
form in elementary torch operations in 32 bits, rounded once at the end.

E4M3 codes are uint8 tensors; as outputs they are viewed as torch.float8_e4m3fn,
the values the codes stand for before the scale, beside their scales.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
FLT_MIN, FLT_MAX = 2.0 ** -126, (2.0 - 2.0 ** -23) * 2.0 ** 127
ADAM = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}


def listed():
    return [
        # One decoding step of eight requests through the up projection (18432 x 7168 blocks): the
        # weights are read once, for eight rows.
        {"name": "matmul_decode", "op": "matmul", "m": 8, "n": 18432, "k": 7168, "scales": "blocks", "out": "bf16",
         "accumulate": False, "groups": 0},
        # A training micro-batch through the same projection.
        {"name": "matmul_train", "op": "matmul", "m": 4096, "n": 18432, "k": 7168, "scales": "blocks", "out": "bf16",
         "accumulate": False, "groups": 0},
        # The input gradient of the KV-down projection (576 outputs, not whole tiles of 128) for a
        # ragged batch, from the column-major copy of its weights, in half precision.
        {"name": "matmul_ragged", "op": "matmul", "m": 1003, "n": 7168, "k": 576, "scales": "blocks", "out": "f16",
         "accumulate": False, "groups": 0},
        # A weight gradient: both operands column-wise quantized, scales along the tokens, added to
        # the FP32 gradient of earlier micro-batches.
        {"name": "matmul_weight_grad", "op": "matmul", "m": 2048, "n": 7168, "k": 8192, "scales": "rows", "out": "f32",
         "accumulate": True, "groups": 0},
        # The gate projection of a bank of 64 experts; tokens sorted by expert, uneven counts.
        {"name": "experts_forward", "op": "matmul", "m": 8192, "n": 2048, "k": 7168, "scales": "blocks", "out": "bf16",
         "accumulate": False, "groups": 64},
        # The weight gradient of 16 experts, each expert's tokens padded to whole tiles of 128.
        {"name": "experts_weight_grad", "op": "matmul", "m": 2048, "n": 7168, "k": 8192, "scales": "rows", "out": "f32",
         "accumulate": False, "groups": 16},
        # The norm of a decoding step's rows.  Latency.
        {"name": "norm_decode", "op": "norm", "rows": 8, "cols": 7168, "x": "bf16", "param": "bf16", "bias": True,
         "y": True, "q": False, "pow2": False},
        # The norm before an FP8 product, whose operand it writes.
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 7168, "x": "bf16", "param": "f32", "bias": True,
         "y": False, "q": True, "pow2": False},
        # A ragged batch, odd row length, half precision throughout.
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 1021, "cols": 2001, "x": "f16", "param": "f16",
         "bias": False, "accumulate": False},
        # The gradient of that micro-batch, added to FP32 gradients of weight and bias.
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 16384, "cols": 7168, "x": "bf16", "param": "f32",
         "bias": True, "accumulate": True},
        # The vectors and one small matrix of a fine-tuned adapter, FP32 moments.  Latency.
        {"name": "adamw_few", "op": "adamw", "tensors": 4, "elems": 106240, "g": "f32", "states": 32, "copy": "none",
         "factor": False, "step": 3},
        # A model of many matrices of uneven sizes and odd vectors: BF16 gradients, moments in 8 bits, a BF16
        # copy for the next forward pass, the clipping coefficient taken from device memory.
        {"name": "adamw_8bit", "op": "adamw", "tensors": 61, "elems": 200000000, "g": "bf16", "states": 8,
         "copy": "bf16", "factor": True, "step": 1000},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "experts", "norm", "norm_grad", "adamw"])
    if op == "matmul":
        if rng.random() < 0.35:
            return {"op": op, "m": _log_uniform(rng, 100, 7168), "n": _log_uniform(rng, 100, 7168),
                    "k": 128 * _log_uniform(rng, 1, 64), "scales": "rows", "out": rng.choice(["f32", "f32", "bf16"]),
                    "accumulate": False, "groups": 0}
        return {"op": op, "m": _log_uniform(rng, 1, 4096), "n": rng.choice([_log_uniform(rng, 100, 18432), 128 * _log_uniform(rng, 1, 144)]),
                "k": 64 * _log_uniform(rng, 2, 112), "scales": "blocks", "out": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "accumulate": False, "groups": 0}
    if op == "experts":
        by_k = rng.random() < 0.3
        n, k = 128 * _log_uniform(rng, 2, 16), 128 * _log_uniform(rng, 2, 56)
        m = _log_uniform(rng, 1, 8192)
        if by_k:
            return {"op": "matmul", "m": n, "n": k, "k": m, "scales": "rows", "out": "f32",
                    "accumulate": rng.random() < 0.5, "groups": _log_uniform(rng, 2, 16)}
        return {"op": "matmul", "m": m, "n": n, "k": k, "scales": "blocks", "out": rng.choice(["bf16", "bf16", "f16"]),
                "accumulate": False, "groups": _log_uniform(rng, 2, 64)}
    if op == "norm":
        q = rng.random() < 0.5
        cols = 128 * _log_uniform(rng, 1, 56) if q else _log_uniform(rng, 32, 7168)
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        return {"op": op, "rows": _log_uniform(rng, 1, 16384), "cols": cols, "x": x, "param": rng.choice(["f32", x]),
                "bias": rng.random() < 0.5, "y": not q or rng.random() < 0.3, "q": q, "pow2": rng.random() < 0.3}
    if op == "norm_grad":
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        return {"op": op, "rows": _log_uniform(rng, 1, 16384),
                "cols": rng.choice([_log_uniform(rng, 32, 7168), 8 * _log_uniform(rng, 8, 896)]), "x": x,
                "param": rng.choice(["f32", x]), "bias": rng.random() < 0.5, "accumulate": False}
    few = rng.random() < 0.4
    return {"op": op, "tensors": rng.randint(1, 9) if few else rng.randint(10, 200),
            "elems": _log_uniform(rng, 1000, 1e6) if few else _log_uniform(rng, 1e6, 2e8),
            "g": rng.choice(["f32", "bf16", "f16"]), "states": rng.choice([8, 32]),
            "copy": rng.choice(["none", "bf16", "f16"]), "factor": rng.random() < 0.5, "step": rng.choice([1, 7, 1000])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std):
    """N(0, std^2) drawn in pieces, so that the 32-bit draws stay small."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(std))
    return out


def _codes(x):
    """E4M3 codes (nearest, ties to even) of values within +-448."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(q):
    return q.view(torch.float8_e4m3fn).float()


def _padded_tiles(x):
    """[.., cols] as [.., tiles, 128], zeros after the last column."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % 128)).unflatten(-1, (-1, 128))


def _row_quantize(x):
    """Codes and scales of rows in tiles of 128: s = amax / 448, 1 for a tile of zeros."""
    t = _padded_tiles(x)
    amax = t.abs().amax(-1)
    s = torch.where(amax > 0, (amax / 448.0).clamp(min=FLT_MIN), torch.ones_like(amax))
    return _codes((t / s.unsqueeze(-1)).flatten(-2)[..., :x.shape[-1]]).contiguous(), s


def _block_quantize(w):
    """Codes and inverse scales of 128 x 128 blocks of w [n, k]."""
    n, k = w.shape
    b = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128))
    b = b.view(b.shape[0] // 128, 128, b.shape[1] // 128, 128)
    s = 448.0 / b.abs().amax((1, 3)).clamp(min=1e-30)
    q = _codes(b * s[:, None, :, None])
    return q.reshape(q.shape[0] * 128, -1)[:n, :k].contiguous(), 1.0 / s


def _group_counts(case):
    """Rows, or tokens padded to whole tiles of 128, of each group: fixed by the case alone."""
    e, total = case["groups"], case["m"] if case["scales"] == "blocks" else case["k"]
    r = random.Random(total * 1000003 + e)
    share = [r.expovariate(1.0) for _ in range(e)]
    cut = [round(total * sum(share[:i]) / sum(share)) for i in range(e + 1)]
    counts = [b - a for a, b in zip(cut, cut[1:])]
    return counts if case["scales"] == "blocks" else [-(-c // 128) * 128 for c in counts]


def _tensor_sizes(case):
    """Element counts of the tensors: fixed by the case alone."""
    if case["tensors"] == 4 and case["elems"] == 106240:
        return [256 * 384, 384, 384, 7168]
    r = random.Random(case["tensors"] * 1000003 + case["elems"])
    share = [math.exp(r.uniform(0.0, 5.0)) for _ in range(case["tensors"])]
    return [max(1, int(case["elems"] * s / sum(share))) for s in share]


def _prepare_matmul(case, g, s):
    m, n, k, e = case["m"], case["n"], case["k"], case["groups"]
    out = DTYPES[case["out"]]
    if case["scales"] == "blocks":
        s["a"], s["a_scale"] = _row_quantize(_normal(g, (m, k), torch.float32, 1.0))
        parts = [_block_quantize(_normal(g, (n, k), torch.float32, 1.0 / math.sqrt(k))) for _ in range(max(e, 1))]
        s["b"], s["b_scale"] = (torch.stack([p[i] for p in parts]) if e else parts[0][i] for i in (0, 1))
        s["out"] = torch.empty(m, n, dtype=out, device="cuda")
    else:
        s["counts"] = _group_counts(case) if e else [k]
        k = sum(s["counts"])
        # tokens differ in size; the gradient is small
        size = torch.exp(torch.randn(k, generator=g, device="cuda"))
        s["a"], s["a_scale"] = _row_quantize(_normal(g, (m, k), torch.float32, 1e-3) * size)
        s["b"], s["b_scale"] = _row_quantize(_normal(g, (n, k), torch.float32, 1.0))
        shape = (e, m, n) if e else (m, n)
        s["out"] = _normal(g, shape, out, 0.1) if case["accumulate"] else torch.empty(shape, dtype=out, device="cuda")
    if e:
        s["counts"] = _group_counts(case)
        at = torch.tensor([0] + s["counts"], dtype=torch.int64).cumsum(0)
        s["offsets"] = at.to("cuda", torch.int32)
    if own:
        from blockwise_fp8_zero_gb300 import fp8z
        size = fp8z.fp8z_matmul_workspace(s["a"], s["b"], s["out"], offsets=s.get("offsets"))
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


def _prepare_norm(case, g, s):
    rows, cols = case["rows"], case["cols"]
    dt, pt = DTYPES[case["x"]], DTYPES[case["param"]]
    # a residual stream: columns and rows of their own sizes, not centred
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    x += 0.3 * torch.randn(rows, 1, generator=g, device="cuda")
    s["x"] = x.to(dt)
    s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(pt)
    s["bias"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(pt) if case["bias"] else None
    s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if case["op"] == "norm":
        s["y"] = torch.empty(rows, cols, dtype=dt, device="cuda") if case["y"] else None
        s["q"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda") if case["q"] else None
        s["q_scale"] = torch.empty(rows, cols // 128, device="cuda") if case["q"] else None
        return
    d = s["x"].double()
    mean = d.mean(1)
    s["mean"] = mean.float()
    s["rstd"] = (1.0 / ((d - mean.unsqueeze(1)).square().mean(1) + 1e-5).sqrt()).float()
    s["dy"] = _normal(g, (rows, cols), dt, 1e-2)
    s["dx"] = torch.empty(rows, cols, dtype=dt, device="cuda")
    fresh = (lambda: _normal(g, cols, pt, 0.1)) if case["accumulate"] else (lambda: torch.empty(cols, dtype=pt, device="cuda"))
    s["dweight"] = fresh()
    s["dbias"] = fresh() if case["bias"] else None
    if own:
        from blockwise_fp8_zero_gb300 import fp8z
        size = fp8z.fp8z_layer_norm_grad_workspace(rows, cols)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


def _moment_codes(x):
    """Codes and inverse scales of a flat moment in runs of 128."""
    t = _padded_tiles(x)
    amax = t.abs().amax(-1)
    s = torch.where(amax > 0, (448.0 / amax).clamp(max=FLT_MAX), torch.ones_like(amax))
    return (t * s.unsqueeze(-1)), 1.0 / s


def _starts(sizes):
    """Where each tensor starts in the optimizer's flat buffers (whole runs of 128), and their length."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // 128) * 128)
    return at[:-1], at[-1]


def _prepare_adamw(case, g, s):
    sizes = _tensor_sizes(case)
    starts, total = _starts(sizes)
    used = torch.zeros(total, dtype=torch.bool, device="cuda")
    for n, at in zip(sizes, starts):
        used[at:at + n] = True
    s["flat"] = {"p": _normal(g, total, torch.float32, 0.02) * used}
    m = _normal(g, total, torch.float32, 2e-4) * used
    v = (torch.rand(total, generator=g, device="cuda") + 0.5) * 4e-7 * used
    s["g"] = [_normal(g, n, DTYPES[case["g"]], 1e-3) for n in sizes]
    if case["copy"] != "none":
        s["flat"]["copy"] = torch.zeros(total, dtype=DTYPES[case["copy"]], device="cuda")
    if case["states"] == 8:
        for key, x in (("m", m), ("v", v.sqrt())):
            t, s["flat"][key + "_scale"] = _moment_codes(x)
            s["flat"][key] = _codes(t).view(-1)
    else:
        s["flat"].update(m=m, v=v)
    for key, flat in s["flat"].items():
        per = 128 if key.endswith("_scale") else 1
        s[key] = [flat[at // per:at // per + -(-n // per)] for n, at in zip(sizes, starts)]
    s["factor"] = torch.full((1,), 0.37, device="cuda") if case["factor"] else None
    if own:
        from blockwise_fp8_zero_gb300 import fp8z
        s["list"] = fp8z.fp8z_encode_adamw_list(s["p"], s["g"], s["m"], s["v"], copies=s.get("copy"),
                                                exp_avg_scales=s.get("m_scale"), exp_avg_sq_scales=s.get("v_scale"))
        s["hp"] = fp8z.hparams(step=case["step"], **ADAM)


def prepare(case, seed):
    s = {"case": case}
    {"matmul": _prepare_matmul, "norm": _prepare_norm, "norm_grad": _prepare_norm,
     "adamw": _prepare_adamw}[case["op"]](case, _gen(seed), s)
    return s


# -------------------------------------------------------------- one pass
def _codes_out(q):
    return q.view(torch.float8_e4m3fn)


def _adamw_outputs(s):
    return {k: _codes_out(t) if t.dtype == torch.uint8 else t for k, t in s["flat"].items()}


def _norm_outputs(s):
    out = {"mean": s["mean"], "rstd": s["rstd"]}
    if s["y"] is not None:
        out["y"] = s["y"]
    if s["q"] is not None:
        out["q"], out["q_scale"] = _codes_out(s["q"]), s["q_scale"]
    return out


def _norm_grad_outputs(s):
    out = {"dx": s["dx"], "dweight": s["dweight"]}
    if s["dbias"] is not None:
        out["dbias"] = s["dbias"]
    return out


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from blockwise_fp8_zero_gb300 import fp8z
    case, op = s["case"], s["case"]["op"]
    if op == "matmul":
        fp8z.fp8z_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], offsets=s.get("offsets"),
                         accumulate=case["accumulate"], workspace=s["workspace"])
        return {"out": s["out"]}
    if op == "norm":
        fp8z.fp8z_layer_norm(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=1e-5, q=s["q"],
                             q_scale=s["q_scale"], pow2=case["pow2"])
        return _norm_outputs(s)
    if op == "norm_grad":
        fp8z.fp8z_layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"],
                                  s["dbias"], s["workspace"], accumulate=case["accumulate"])
        return _norm_grad_outputs(s)
    fp8z.fp8z_adamw(s["list"], s["hp"], grad_factor=s["factor"])
    return _adamw_outputs(s)


def _row_values(q, scale):
    """float32 values of row-wise quantized codes."""
    return _values(q) * scale.repeat_interleave(128, -1)[..., :q.shape[-1]]


def _block_values(q, scale):
    n, k = q.shape
    return _values(q) * scale.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def _run_plain(s):
    return {"matmul": _plain_matmul, "norm": _plain_norm, "norm_grad": _plain_norm_grad,
            "adamw": _plain_adamw}[s["case"]["op"]](s)


def _plain_matmul(s):
    case, out = s["case"], s["out"]
    if case["scales"] == "blocks":
        a = _row_values(s["a"], s["a_scale"])
        if not case["groups"]:
            return {"out": (a @ _block_values(s["b"], s["b_scale"]).t()).to(out.dtype)}
        at = 0
        for i, c in enumerate(s["counts"]):
            if c:
                out[at:at + c] = (a[at:at + c] @ _block_values(s["b"][i], s["b_scale"][i]).t()).to(out.dtype)
            at += c
        return {"out": out}
    a, b = _row_values(s["a"], s["a_scale"]), _row_values(s["b"], s["b_scale"])
    at, parts = 0, out.unsqueeze(0) if not case["groups"] else out
    for i, c in enumerate(s["counts"]):
        p = a[:, at:at + c] @ b[:, at:at + c].t()
        parts[i].copy_(parts[i] + p if case["accumulate"] else p)
        at += c
    return {"out": out}


def _plain_norm(s):
    case, cols = s["case"], s["case"]["cols"]
    x = s["x"].float()
    mean = x.sum(1, keepdim=True) / cols
    x = x - mean
    rstd = 1.0 / ((x * x).sum(1, keepdim=True) / cols + 1e-5).sqrt()
    y = x * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    s["mean"].copy_(mean.squeeze(1))
    s["rstd"].copy_(rstd.squeeze(1))
    if s["y"] is not None:
        s["y"].copy_(y)
    if s["q"] is not None:
        t = _padded_tiles(y)
        scale = t.abs().amax(-1) / 448.0
        scale = torch.where(scale > 0, scale.clamp(min=FLT_MIN), torch.ones_like(scale))
        if case["pow2"]:
            scale = torch.exp2(torch.ceil(torch.log2(scale)))
        s["q"].copy_(_codes(t / scale.unsqueeze(-1)).view(s["q"].shape))
        s["q_scale"].copy_(scale)
    return _norm_outputs(s)


def _plain_norm_grad(s):
    case, cols = s["case"], s["case"]["cols"]
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"].unsqueeze(1)) * s["rstd"].unsqueeze(1)
    g = dy * s["weight"].float()
    dx = (g - g.sum(1, keepdim=True) / cols - xh * ((g * xh).sum(1, keepdim=True) / cols)) * s["rstd"].unsqueeze(1)
    s["dx"].copy_(dx)
    for out, part in ((s["dweight"], dy * xh), (s["dbias"], dy)):
        if out is not None:
            total = part.sum(0)
            out.copy_(out.float() + total if case["accumulate"] else total)
    return _norm_grad_outputs(s)


def _plain_adamw(s):
    case, b1, b2 = s["case"], ADAM["beta1"], ADAM["beta2"]
    step_size = ADAM["lr"] / (1.0 - b1 ** case["step"])
    rs = 1.0 / math.sqrt(1.0 - b2 ** case["step"])
    for i, p in enumerate(s["p"]):
        n = p.numel()
        g = s["g"][i].float()
        if s["factor"] is not None:
            g = g * s["factor"]
        if "m_scale" not in s:
            m, v = s["m"][i], s["v"][i]
        else:
            m = _row_values(s["m"][i], s["m_scale"][i])
            v = _row_values(s["v"][i], s["v_scale"][i]).square()
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + g * g * (1.0 - b2)
        r = v.sqrt()
        p.mul_(1.0 - ADAM["lr"] * ADAM["weight_decay"]).sub_(m / (r * rs + ADAM["eps"]) * step_size)
        if "copy" in s:
            s["copy"][i].copy_(p)
        if "m_scale" not in s:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
        else:
            t, inv = _moment_codes(m)
            s["m"][i].copy_(_codes(t).view(-1)[:n])
            s["m_scale"][i].copy_(inv)
            t, inv = _moment_codes(r)
            q = _codes(t)
            s["v"][i].copy_(torch.where((q == 0) & (t > 0), torch.ones_like(q), q).view(-1)[:n])
            s["v_scale"][i].copy_(inv)
    return _adamw_outputs(s)


# ------------------------------------------------------------ definitions
def _code_table():
    """The value of each E4M3 code, from sign, exponent and fraction."""
    c = torch.arange(256, device="cuda")
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f / 512.0, (1.0 + f / 8.0) * torch.exp2((e - 7).double()))
    v[(c & 127) == 127] = math.nan
    return torch.where(c > 127, -v, v)


def _nearest(x):
    """The nearest E4M3 value of each number, ties to the even fraction."""
    _, e = torch.frexp(x)
    ulp = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / ulp) * ulp).clamp(-448.0, 448.0)


def _exact_matmul(case, s):
    e = case["groups"]
    if 2.0 * case["m"] * case["n"] * s["a"].shape[1] > 4e12:
        return None
    table = _code_table()
    ta = [table[s["a"][:, i:i + 128].long()] * s["a_scale"][:, i // 128].double().unsqueeze(1)
          for i in range(0, s["a"].shape[1], 128)]
    if case["scales"] == "blocks":
        def product(rows, q, scale):
            total = 0
            for i, t in enumerate(ta):
                w = table[q[:, i * 128:i * 128 + 128].long()]
                by_row = torch.arange(q.shape[0], device="cuda") // 128
                total = total + t[rows] @ (w * scale[:, i].double()[by_row].unsqueeze(1)).t()
            return total
        if not e:
            return {"out": product(slice(None), s["b"], s["b_scale"])}
        ends = torch.tensor(s["counts"]).cumsum(0).tolist()
        return {"out": torch.cat([product(slice(z - c, z), s["b"][i], s["b_scale"][i])
                                  for i, (c, z) in enumerate(zip(s["counts"], ends))])}
    out = s["out"].double() if case["accumulate"] else torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    parts = out if e else out.unsqueeze(0)
    group = [i for i, c in enumerate(s["counts"]) for _ in range(c // 128)]
    for i, t in enumerate(ta):
        w = table[s["b"][:, i * 128:i * 128 + 128].long()] * s["b_scale"][:, i].double().unsqueeze(1)
        parts[group[i] if e else 0].addmm_(t, w.t())
    return {"out": out}


def _exact_norm(case, s):
    x = s["x"].double()
    mean, var = x.mean(1), x.var(1, unbiased=False)
    rstd = (var + 1e-5).rsqrt()
    out = {"mean": mean, "rstd": rstd}
    y = torch.addcmul(torch.zeros((), dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double(),
                      (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), s["weight"].double())
    if case["y"]:
        out["y"] = y
    if case["q"]:
        t = y.view(y.shape[0], -1, 128)
        scale = t.abs().max(-1).values / 448.0
        scale[scale == 0] = 1.0
        if case["pow2"]:
            f, e = torch.frexp(scale)
            scale = torch.exp2((e - (f == 0.5).int()).double())
        out["q"], out["q_scale"] = _nearest(t / scale.unsqueeze(-1)).view(y.shape), scale
    return out


def _exact_norm_grad(case, s):
    dy, w, rstd = s["dy"].double(), s["weight"].double(), s["rstd"].double().unsqueeze(1)
    xh = (s["x"].double() - s["mean"].double().unsqueeze(1)) * rstd
    g = dy * w
    # the gradient is what is left of g without its parts along 1 and along xh
    out = {"dx": rstd * (g - g.mean(1, keepdim=True) - xh * torch.einsum("ij,ij->i", g, xh).unsqueeze(1) / case["cols"])}
    start = {k: s[k].double() if case["accumulate"] else 0.0 for k in ("dweight", "dbias") if s[k] is not None}
    out["dweight"] = start["dweight"] + torch.einsum("ij,ij->j", dy, xh)
    if case["bias"]:
        out["dbias"] = start["dbias"] + dy.sum(0)
    return out


def _exact_adamw(case, s):
    table = _code_table()
    # the library's hyper-parameters are 32-bit numbers
    lr, b1, b2, eps, wd = (float(torch.tensor(ADAM[k], dtype=torch.float32)) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    out = {k: t.double() if t.dtype != torch.uint8 else table[t.long()] for k, t in s["flat"].items()}
    for i, at in enumerate(_starts(_tensor_sizes(case))[0]):
        n = s["p"][i].numel()
        here, tile = slice(at, at + n), torch.arange(n, device="cuda") // 128
        g = s["g"][i].double() * (1.0 if s["factor"] is None else s["factor"].double())
        m, v = out["m"][here], out["v"][here]
        if case["states"] == 8:
            m = m * s["m_scale"][i].double()[tile]
            v = (v * s["v_scale"][i].double()[tile]) ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        new = s["p"][i].double() * (1 - lr * wd) - lr * (m / (1 - b1 ** case["step"])) / ((v / (1 - b2 ** case["step"])).sqrt() + eps)
        out["p"][here] = new
        if "copy" in out:
            out["copy"][here] = new
        if case["states"] == 32:
            out["m"][here], out["v"][here] = m, v
            continue
        for key, x in (("m", m), ("v", v.sqrt())):
            tiles = int(tile[-1]) + 1
            top = torch.zeros(tiles, dtype=torch.float64, device="cuda").scatter_reduce_(0, tile, x.abs(), "amax")
            inv = torch.where(top > 0, top / 448.0, torch.ones_like(top))
            code = _nearest(x / inv[tile])
            if key == "v":
                code = torch.where((code == 0) & (x > 0), 2.0 ** -9, code)
            out[key][here] = code
            out[key + "_scale"][at // 128:at // 128 + tiles] = inv
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"matmul": _exact_matmul, "norm": _exact_norm, "norm_grad": _exact_norm_grad,
            "adamw": _exact_adamw}[case["op"]](case, s)


def work(case):
    op = case["op"]
    if op == "matmul":
        m, n, k, e = case["m"], case["n"], case["k"], case["groups"]
        out, passes = BYTES[case["out"]], 2 if case["accumulate"] else 1
        if case["scales"] == "blocks":
            banks = sum(c > 0 for c in _group_counts(case)) if e else 1       # experts without a token are not read
            kb = -(-k // 128)
            return {"bytes": m * (k + 4 * kb) + banks * (n * k + 4 * kb * -(-n // 128)) + m * n * out * passes,
                    "flops": 2 * m * n * k}
        k = sum(_group_counts(case)) if e else k
        return {"bytes": (m + n) * (k + 4 * (k // 128)) + max(e, 1) * m * n * out * passes, "flops": 2 * m * n * k}
    if op in ("norm", "norm_grad"):
        r, c, b, pb = case["rows"], case["cols"], BYTES[case["x"]], BYTES[case["param"]]
        vectors = (2 if case["bias"] else 1) * c * pb
        if op == "norm":
            return {"bytes": r * c * b * (2 if case["y"] else 1) + (r * c + 4 * r * (c // 128) if case["q"] else 0) + vectors + 8 * r,
                    "flops": 8 * r * c}
        return {"bytes": 3 * r * c * b + c * pb + vectors * (2 if case["accumulate"] else 1) + 8 * r, "flops": 13 * r * c}
    n = sum(_tensor_sizes(case))
    states = 4 * (1 + 4 / 128) if case["states"] == 8 else 16
    return {"bytes": int(n * (8 + BYTES[case["g"]] + states + (0 if case["copy"] == "none" else 2))), "flops": 16 * n}
