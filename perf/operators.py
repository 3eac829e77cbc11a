"""Timed cases of the operators around the optimizer step: global gradient norm
and clipping, embedding lookup and its gradient, and the softmax cross entropy
of a vocabulary projection with its gradient.

Every case is a dict of plain values.  `prepare` makes what a training or
evaluation program has in hand before the call (inputs, output buffers and,
where the library's own calls are made, the list of tensors and the workspace
that such a program keeps), `run` makes one pass, `exact` computes the same
outputs from the definitions in 64 bits, and `work` counts the bytes and
operations a pass cannot do without.  With `own` false `run` computes the plain
form in elementary torch operations in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
IGNORE = -100


def listed():
    return [
        # One small weight (256x384, its gradient and bias) and two vectors: a
        # fine-tuned adapter's gradients.  Latency.
        {"name": "clip_few", "op": "clip", "set": "few", "tensors": 4, "elems": 106240,
         "src": "f32", "dst": "f32", "grad_scale": 1.0, "max_norm": 1.0},
        # A model of many matrices of uneven sizes and odd vectors, bf16 gradients
        # summed over 4 micro-batches, clipped into the optimizer's FP32 gradients.
        {"name": "clip_mixed", "op": "clip", "set": "mixed", "tensors": 61, "elems": 200000000,
         "src": "bf16", "dst": "f32", "grad_scale": 0.25, "max_norm": 1.0},
        # The hidden-7168 dense layer set (Q, O, KV-down, up, gate, down) in FP32.
        {"name": "clip_dense", "op": "clip", "set": "dense", "tensors": 6, "elems": 503250944,
         "src": "f32", "dst": "f32", "grad_scale": 1.0, "max_norm": 1.0},
        # The rows of one decoding step of eight requests.  Latency.
        {"name": "embed_decode", "op": "embed", "tokens": 8, "vocab": 65536, "hidden": 7168,
         "src": "bf16", "dst": "bf16", "scale": 1.0},
        # A training micro-batch of 16384 tokens, rows scaled by sqrt(hidden).
        {"name": "embed_train", "op": "embed", "tokens": 16384, "vocab": 65536, "hidden": 7168,
         "src": "bf16", "dst": "bf16", "scale": 84.66},
        # A short ragged batch into an existing FP32 gradient (a tied table whose
        # gradient the loss has written already); odd row length.
        {"name": "embed_grad_ragged", "op": "embed_grad", "tokens": 1021, "vocab": 32003, "hidden": 577,
         "src": "bf16", "dst": "f32", "scale": 1.0, "accumulate": True},
        # The gradient of that micro-batch: the whole FP32 table is written, with
        # word frequencies that fall as 1/rank.
        {"name": "embed_grad_train", "op": "embed_grad", "tokens": 16384, "vocab": 65536, "hidden": 7168,
         "src": "bf16", "dst": "f32", "scale": 84.66, "accumulate": False},
        # Scoring a few tokens of one answer.  Latency.
        {"name": "loss_few", "op": "loss", "tokens": 7, "vocab": 32000, "hidden": 2048, "src": "bf16"},
        # Evaluation of one 2048-token document; a vocabulary of odd size.
        {"name": "loss_eval", "op": "loss", "tokens": 2048, "vocab": 65537, "hidden": 7168, "src": "bf16"},
        # A ragged batch in training: odd counts of tokens and of words, FP32 weight gradient.
        {"name": "loss_grad_ragged", "op": "loss_grad", "tokens": 1000, "vocab": 50001, "hidden": 2000,
         "src": "bf16", "dw": "f32", "grad_scale": 1.0},
        # Half-precision training of a small model with a loss scale, gradients in the weights' type.
        {"name": "loss_grad_f16", "op": "loss_grad", "tokens": 509, "vocab": 32768, "hidden": 2048,
         "src": "f16", "dw": "f16", "grad_scale": 1024.0},
        # A training micro-batch with a large vocabulary, FP32 weight gradient
        # as the optimizer step takes it.
        {"name": "loss_grad_train", "op": "loss_grad", "tokens": 4096, "vocab": 131072, "hidden": 7168,
         "src": "bf16", "dw": "f32", "grad_scale": 1.0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["clip", "embed", "embed_grad", "loss", "loss_grad"])
    if op == "clip":
        kind = rng.choice(["few", "mixed"])
        src = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "set": kind, "tensors": rng.randint(1, 9) if kind == "few" else rng.randint(10, 200),
                "elems": _log_uniform(rng, 1000, 1e6) if kind == "few" else _log_uniform(rng, 1e6, 4e8),
                "src": src, "dst": rng.choice(["f32", src]), "grad_scale": rng.choice([1.0, 0.125]),
                "max_norm": rng.choice([0.5, 1.0, 1e6])}
    hidden = rng.choice([_log_uniform(rng, 64, 7168), 8 * _log_uniform(rng, 8, 896)])
    src = rng.choice(["bf16", "bf16", "f16"])
    if op == "embed":
        return {"op": op, "tokens": _log_uniform(rng, 1, 16384), "vocab": _log_uniform(rng, 1000, 65536),
                "hidden": hidden, "src": rng.choice([src, "f32"]), "dst": src, "scale": rng.choice([1.0, 12.5])}
    if op == "embed_grad":
        return {"op": op, "tokens": _log_uniform(rng, 1, 16384), "vocab": _log_uniform(rng, 1000, 65536),
                "hidden": hidden, "src": src, "dst": rng.choice(["f32", "f32", src]), "scale": rng.choice([1.0, 12.5]),
                "accumulate": rng.random() < 0.5}
    c = {"op": op, "tokens": _log_uniform(rng, 1, 4096), "vocab": _log_uniform(rng, 1000, 131072),
         "hidden": hidden, "src": src}
    if op == "loss_grad":
        c["dw"] = rng.choice(["f32", src])
        c["grad_scale"] = 1024.0 if src == "f16" else 1.0
    return c


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


def _words(g, tokens, vocab):
    """Word ids whose frequency falls as 1/rank."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab)).long() - 1).clamp_(0, vocab - 1)


def _clip_sizes(case):
    """Element counts of the tensors: fixed by the case alone."""
    if case["set"] == "dense":
        h, f = 7168, 18432
        return [h * h, h * h, h * 576, h * f, h * f, f * h]
    if case["set"] == "few" and case["tensors"] == 4 and case["elems"] == 106240:
        return [256 * 384, 384, 384, 7168]
    r = random.Random(case["tensors"] * 1000003 + case["elems"])
    share = [math.exp(r.uniform(0.0, 5.0)) for _ in range(case["tensors"])]
    total = sum(share)
    return [max(1, int(case["elems"] * s / total)) for s in share]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "clip":
        src, dst = DTYPES[case["src"]], DTYPES[case["dst"]]
        s["grads"] = [_normal(g, n, src, 1e-3) for n in _clip_sizes(case)]
        # the optimizer's gradients lie in one flat buffer, each from a multiple of 64 elements
        sizes = [t.numel() for t in s["grads"]]
        s["flat"] = torch.zeros(sum(-(-n // 64) * 64 for n in sizes), dtype=dst, device="cuda")
        at = [0]
        for n in sizes:
            at.append(at[-1] + -(-n // 64) * 64)
        s["outs"] = [s["flat"][i:i + n] for i, n in zip(at, sizes)]
        s["norm"] = torch.zeros(2, device="cuda")
        if own:
            from blockwise_fp8_zero_gb300 import fp8z
            s["list"] = fp8z.fp8z_encode_tensor_list(s["grads"], s["outs"])
            s["workspace"] = torch.zeros(fp8z.fp8z_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
        return s
    n, v, h = case["tokens"], case["vocab"], case["hidden"]
    src = DTYPES[case["src"]]
    if op == "embed":
        s["ids"] = _words(g, n, v)
        s["table"] = _normal(g, (v, h), src, 0.02)
        s["out"] = torch.empty(n, h, dtype=DTYPES[case["dst"]], device="cuda")
    elif op == "embed_grad":
        s["ids"] = _words(g, n, v)
        s["ids"][5::17] = 0                                  # padding
        s["d_out"] = _normal(g, (n, h), src, 1e-3)
        s["d_table"] = torch.zeros(v, h, dtype=DTYPES[case["dst"]], device="cuda")
        if case["accumulate"]:
            s["d_table"].copy_(_normal(g, (v, h), DTYPES[case["dst"]], 1e-3))
        if own:
            from blockwise_fp8_zero_gb300 import fp8z
            s["workspace"] = torch.empty(fp8z.fp8z_embedding_grad_workspace(n, v, h), dtype=torch.uint8, device="cuda")
    else:
        s["w"] = _normal(g, (v, h), src, 1.7 / math.sqrt(h))
        t = _words(g, n, v)
        # hidden states after a norm; some lean towards their word, as a trained model's do
        x = torch.randn(n, h, generator=g, device="cuda")
        lean = torch.rand(n, 1, generator=g, device="cuda") * 4.0
        x += lean * s["w"][t].float()
        s["x"] = x.to(src)
        t[torch.rand(n, generator=g, device="cuda") < 0.05] = IGNORE
        s["targets"] = t
        s["loss"] = torch.empty(n, device="cuda")
        s["total"] = torch.empty(2, device="cuda")
        if op == "loss_grad":
            s["dx"] = torch.empty(n, h, dtype=src, device="cuda")
            s["dw"] = torch.empty(v, h, dtype=DTYPES[case["dw"]], device="cuda")
        if own:
            from blockwise_fp8_zero_gb300 import fp8z
            size = fp8z.fp8z_linear_xent_workspace(s["x"], s["w"], dw=s.get("dw"))
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from blockwise_fp8_zero_gb300 import fp8z
    case, op = s["case"], s["case"]["op"]
    if op == "clip":
        fp8z.fp8z_grad_clip(s["list"], case["max_norm"], s["norm"], s["workspace"], grad_scale=case["grad_scale"])
        return {"norm": s["norm"], "grads": s["flat"]}
    if op == "embed":
        fp8z.fp8z_embedding(s["ids"], s["table"], s["out"], scale=case["scale"])
        return {"out": s["out"]}
    if op == "embed_grad":
        fp8z.fp8z_embedding_grad(s["ids"], s["d_out"], s["d_table"], s["workspace"], scale=case["scale"],
                                 padding_idx=0, accumulate=case["accumulate"])
        return {"d_table": s["d_table"]}
    if op == "loss":
        fp8z.fp8z_linear_xent(s["x"], s["w"], s["targets"], s["loss"], s["total"], s["workspace"], ignore_index=IGNORE)
        return {"loss": s["loss"], "total": s["total"]}
    fp8z.fp8z_linear_xent_grad(s["x"], s["w"], s["targets"], s["loss"], s["total"], s["dx"], s["dw"], s["workspace"],
                               ignore_index=IGNORE, grad_scale=case["grad_scale"])
    return {"loss": s["loss"], "total": s["total"], "dx": s["dx"], "dw": s["dw"]}


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "clip":
        scale = abs(case["grad_scale"])
        norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt() * scale
        coef = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        factor = coef * case["grad_scale"]
        _ = [o.copy_(t.float() * factor) for t, o in zip(s["grads"], s["outs"])]
        return {"norm": torch.stack([norm, coef]), "grads": s["flat"]}
    if op == "embed":
        return {"out": (s["table"][s["ids"]].float() * case["scale"]).to(DTYPES[case["dst"]])}
    if op == "embed_grad":
        d = s["d_out"].float() * case["scale"] * (s["ids"] != 0).unsqueeze(1)
        t = s["d_table"]
        # an FP32 table is its own sum; a narrower one is summed in 32 bits and rounded once
        base = t if t.dtype == torch.float32 else t.float()
        if not case["accumulate"]:
            base.zero_()
        base.index_add_(0, s["ids"], d)
        if base is not t:
            t.copy_(base)
        return {"d_table": t}
    x, w, t = s["x"].float(), s["w"].float(), s["targets"]
    keep = t != IGNORE
    count = keep.sum().clamp(min=1).float()
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    e = (logits - top).exp()
    z = e.sum(1, keepdim=True)
    at = t.clamp(min=0).unsqueeze(1)
    loss = (z.log() + top - logits.gather(1, at)).squeeze(1) * keep
    out = {"loss": loss, "total": torch.stack([loss.sum() / count, keep.sum().float()])}
    if op == "loss_grad":
        p = e / z
        p.scatter_add_(1, at, torch.full(at.shape, -1.0, device="cuda"))
        p *= (keep * case["grad_scale"] / count).unsqueeze(1)
        out["dx"] = (p @ w).to(s["dx"].dtype)
        out["dw"] = (p.t() @ x).to(s["dw"].dtype)
    return out


# ------------------------------------------------------------ definitions
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "clip":
        sq = sum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"])
        norm = abs(case["grad_scale"]) * math.sqrt(sq)
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        factor, pad = case["grad_scale"] * coef, lambda t: torch.nn.functional.pad(t.double(), (0, -t.numel() % 64))
        return {"norm": torch.tensor([norm, coef], dtype=torch.float64),
                "grads": torch.cat([pad(t) for t in s["grads"]]) * factor}
    if op == "embed":
        return {"out": s["table"].index_select(0, s["ids"]).double() * case["scale"]}
    if op == "embed_grad":
        # sorted words: a word's sum is the difference of two running sums
        ids, order = torch.sort(s["ids"], stable=True)
        run = torch.cumsum(s["d_out"][order].double(), 0)
        last = torch.cat([ids[1:] != ids[:-1], torch.ones(1, dtype=torch.bool, device="cuda")])
        ends, words = run[last], ids[last]
        sums = ends - torch.cat([torch.zeros_like(ends[:1]), ends[:-1]])
        out = s["d_table"].double() if case["accumulate"] else torch.zeros(s["d_table"].shape, dtype=torch.float64, device="cuda")
        use = words != 0
        out[words[use]] += case["scale"] * sums[use]
        return {"d_table": out}
    n, v, h = case["tokens"], case["vocab"], case["hidden"]
    if 8.0 * n * v * h > 1e13:
        return None
    x, t = s["x"].double(), s["targets"]
    keep = t != IGNORE
    pieces = range(0, v, 8192)
    logz = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
    for i in pieces:
        logz = torch.logaddexp(logz, torch.logsumexp(x @ s["w"][i:i + 8192].double().t(), 1))
    own_word = s["w"][t.clamp(min=0)].double()
    loss = torch.where(keep, logz - (x * own_word).sum(1), torch.zeros_like(logz))
    count = max(1, int(keep.sum()))
    out = {"loss": loss, "total": torch.stack([loss.sum() / count, keep.sum().double()])}
    if op == "loss_grad":
        dx = torch.zeros(n, h, dtype=torch.float64, device="cuda")
        dw = torch.zeros(v, h, dtype=torch.float64, device="cuda")
        weight = keep.double().unsqueeze(1) * (case["grad_scale"] / count)
        for i in pieces:
            wi = s["w"][i:i + 8192].double()
            p = torch.exp(x @ wi.t() - logz.unsqueeze(1)) * weight
            dx += p @ wi
            dw[i:i + 8192] = p.t() @ x
        dx -= weight * own_word
        dw.index_add_(0, t[keep], -(x * weight)[keep])
        out["dx"], out["dw"] = dx, dw
    return out


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(_clip_sizes(case))
        return {"bytes": n * (BYTES[case["src"]] + BYTES[case["dst"]]), "flops": 3 * n}
    n, v, h = case["tokens"], case["vocab"], case["hidden"]
    b = BYTES[case["src"]]
    if op == "embed":
        return {"bytes": 8 * n + n * h * (b + BYTES[case["dst"]]), "flops": n * h}
    if op == "embed_grad":
        d = BYTES[case["dst"]]
        # rows that are written: all of them, or about as many as there are different words
        rows = v * (1.0 - math.exp(-n / v)) if case["accumulate"] else v
        return {"bytes": 8 * n + n * h * b + rows * h * d * (2 if case["accumulate"] else 1), "flops": 2 * n * h}
    if op == "loss":
        return {"bytes": (n + v) * h * b + 12 * n, "flops": 2 * n * v * h}
    return {"bytes": 2 * n * h * b + v * h * (b + BYTES[case["dw"]]) + 12 * n, "flops": 6 * n * v * h}
