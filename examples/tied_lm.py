"""A small tied-table language model trained with the library's own operators.

One step is what a training step around the FP8 optimizer looks like:

  x    = scale * E[ids]                      fp8z_embedding
  h    = x M                                 the body, one matrix here (torch.matmul)
  loss = cross entropy of softmax(h E^T)     fp8z_linear_xent_grad: loss, dh, dE
  dM, dx through the body                    torch.matmul
  dE  += scale * sum of dx by token          fp8z_embedding_grad, into the same FP32 dE
  clip dE and dM by their global norm        fp8z_grad_clip, in place
  AdamW and FP8 blocks                       fp8z_adamw_requant_step_rowmajor

The FP32 main params and moments stay folded (the optimizer's own layout); the
step reads the row-major FP32 gradients and writes E4M3 weights with one scale
per 128x128 block.  The next step computes with the new weights in BF16, from the
main params (fp8z_unfold).  The text is a noisy cycle of words, so the loss has a
floor to fall to.

  python examples/tied_lm.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

BLK = fp8z.BLOCK_ELEMS


def text(tokens, vocab, gen):
    """Words and the words that follow them: after w comes 5 w + 3, one time in
    eight any word; every 50th target is padding."""
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    after = (5 * ids + 3) % vocab
    noise = torch.rand(tokens, generator=gen, device="cuda") < 0.125
    after = torch.where(noise, torch.randint(0, vocab, (tokens,), generator=gen, device="cuda"), after)
    after[::50] = -100
    return ids, after


def train(steps=60, vocab=500, hidden=256, tokens=1024, lr=4e-3, max_norm=1.0, seed=0):
    """Losses and gradient norms of `steps` steps, one float each."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shapes = [(1, vocab, hidden), (1, hidden, hidden)]
    params, shards, blocks, summary = fp8z.fp8z_plan_shards(shapes, dp=1)
    cap = int(summary["capacity_blocks"])
    desc, table = fp8z.table_to_device(blocks), fp8z.table_to_device(params)
    p, m, v = (torch.zeros(cap * BLK, device="cuda") for _ in range(3))
    init = [torch.randn(vocab, hidden, generator=gen, device="cuda") * 0.05,
            torch.randn(hidden, hidden, generator=gen, device="cuda") / math.sqrt(hidden)]
    for w, entry in zip(init, params):
        fp8z.fp8z_fold(w, entry, p)
    main = [torch.empty_like(w) for w in init]                       # row-major view of p, for the next step
    grads = [torch.zeros_like(w) for w in init]
    g_maps = fp8z.fp8z_encode_grad_maps(grads, params)
    w_row = torch.empty(sum(e * r * c for e, r, c in shapes), dtype=torch.uint8, device="cuda")
    inv_scale = torch.empty(cap, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    scale = math.sqrt(hidden)
    e16 = torch.empty(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    m16 = torch.empty(hidden, hidden, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    dh = torch.empty_like(x)
    loss, total, norm = torch.empty(tokens, device="cuda"), torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    xent_ws = torch.empty(fp8z.fp8z_linear_xent_workspace(x, e16, dw=grads[0]), dtype=torch.uint8, device="cuda")
    embed_ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(tokens, vocab, hidden), dtype=torch.uint8, device="cuda")
    norm_ws = torch.zeros(fp8z.fp8z_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
    grad_list = fp8z.fp8z_encode_tensor_list(grads)

    losses, norms = [], []
    for step in range(1, steps + 1):
        for w, entry in zip(main, params):
            fp8z.fp8z_unfold(p, entry, w)
        e16.copy_(main[0])
        m16.copy_(main[1])
        ids, after = text(tokens, vocab, gen)
        fp8z.fp8z_embedding(ids, e16, x, scale=scale, dev_status=status)
        h = x @ m16
        fp8z.fp8z_linear_xent_grad(h, e16, after, loss, total, dh, grads[0], xent_ws, dev_status=status)
        torch.matmul(x.t().float(), dh.float(), out=grads[1])
        dx = dh @ m16.t()
        fp8z.fp8z_embedding_grad(ids, dx, grads[0], embed_ws, scale=scale, accumulate=True, dev_status=status)
        fp8z.fp8z_grad_clip(grad_list, max_norm, norm, norm_ws)
        fp8z.fp8z_adamw_requant_step_rowmajor(p, m, v, g_maps, w_row, inv_scale, int(shards[0]["blk_begin"]),
                                              int(shards[0]["blk_count_real"]),
                                              fp8z.hparams(lr=lr, weight_decay=0.01, step=step), desc, table, len(params),
                                              dev_status=status)
        losses.append(float(total[0]))
        norms.append(float(norm[0]))
    assert int(status.item()) == 0, fp8z.fp8z_status_string(int(status.item()))
    return losses, norms


if __name__ == "__main__":
    got, norms = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i in range(0, len(got), 10):
        print(f"step {i + 1:4d}  loss {got[i]:.3f}  gradient norm {norms[i]:.3f}")
    print(f"step {len(got):4d}  loss {got[-1]:.3f}  gradient norm {norms[-1]:.3f}")
