"""A residual block with FP8 weights, trained with the library's operators alone.

One step of y = x + relu(norm(x) W1^T) W2^T against a target:

  forward    norm(x) -> E4M3 rows             fp8z_layer_norm (q)
             h = q W1^T                       fp8z_matmul, 128x128 block scales
             relu(h) -> E4M3 rows             fp8z_quantize_rowwise
             y = x + q W2^T                   fp8z_matmul
  backward   dy -> E4M3 rows                  fp8z_quantize_rowwise
             da = dy W2, dn = dh W1           fp8z_matmul on the column-major copies
             dW2 = dy^T a, dW1 = dh^T n       fp8z_transpose_rowwise, fp8z_matmul with row scales, FP32
             dw, db of the norm               fp8z_layer_norm_grad
  clip       all gradients by their norm      fp8z_grad_clip
  update     W1, W2: AdamW and new blocks     fp8z_adamw_requant_step_rowmajor
             the norm's vectors: AdamW        fp8z_adamw, moments in 8 bits

The FP32 main params of the matrices stay folded; the FP8 weights are the row-major bytes and the
column-major copy that the step writes.

  python examples/fp8_layer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

BLK = fp8z.BLOCK_ELEMS


class Block:
    """The block's parameters and the buffers of one step over `tokens` rows (multiples of 128)."""

    def __init__(self, tokens=512, hidden=256, inner=384, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.hidden, self.inner = tokens, hidden, inner
        shapes = [(1, inner, hidden), (1, hidden, inner)]
        self.entries, self.shards, blocks, summary = fp8z.fp8z_plan_shards(shapes, dp=1)
        cap = int(summary["capacity_blocks"])
        self.desc, self.table = fp8z.table_to_device(blocks), fp8z.table_to_device(self.entries)
        self.p, self.m, self.v = (torch.zeros(cap * BLK, device="cuda") for _ in range(3))
        for (_, rows, cols), entry in zip(shapes, self.entries):
            fp8z.fp8z_fold(torch.randn(rows, cols, generator=gen, device="cuda") / cols ** 0.5, entry, self.p)
        size = sum(e * r * c for e, r, c in shapes)
        self.w_row, self.w_col = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.inv, self.inv_t = torch.empty(cap, device="cuda"), torch.empty(cap, device="cuda")
        self.grads = [torch.zeros(r, c, device="cuda") for _, r, c in shapes]
        self.maps = fp8z.fp8z_encode_grad_maps(self.grads, self.entries)
        self.vectors = [torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")]
        self.vector_grads = [torch.zeros(hidden, device="cuda") for _ in range(2)]
        codes = [[torch.zeros(hidden, dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
        scales = [[torch.ones(-(-hidden // 128), device="cuda") for _ in range(2)] for _ in range(2)]
        self.vector_list = fp8z.fp8z_encode_adamw_list(self.vectors, self.vector_grads, *codes, exp_avg_scales=scales[0],
                                                       exp_avg_sq_scales=scales[1])
        self.clip_list = fp8z.fp8z_encode_tensor_list([*self.grads, *self.vector_grads])
        self.norm = torch.zeros(2, device="cuda")
        self.norm_ws = torch.zeros(fp8z.fp8z_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
        self.ln_ws = torch.empty(fp8z.fp8z_layer_norm_grad_workspace(tokens, hidden), dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.mean, self.rstd = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.update(fp8z.hparams(lr=0.0, weight_decay=0.0, step=1))          # the first FP8 weights
        self.m.zero_()
        self.v.zero_()

    def weight(self, i, column_major=False):
        """(codes, scales) of matrix i as fp8z_matmul takes them: [out, in], or its transpose."""
        e = self.entries[i]
        rows, cols, at = int(e["rows"]), int(e["cols"]), int(e["t_offset"])
        hb, wb = int(e["hb"]), int(e["wb"])
        if column_major:
            first = int(e["t_scale_offset"])
            return self.w_col[at:at + rows * cols].view(cols, rows), self.inv_t[first:first + hb * wb].view(wb, hb)
        first = int(e["blk_offset"])
        return self.w_row[at:at + rows * cols].view(rows, cols), self.inv[first:first + hb * wb].view(hb, wb)

    def quantize(self, x):
        q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        s = torch.empty(x.shape[0], x.shape[1] // 128, device="cuda")
        fp8z.fp8z_quantize_rowwise(x, False, q, s)
        return q, s

    def product(self, a, b, cols):
        out = torch.empty(a[0].shape[0], cols, device="cuda")
        fp8z.fp8z_matmul(*a, *b, out, dev_status=self.status)
        return out

    def columns(self, a):
        """The column-wise layout of row-wise codes."""
        q, s = a
        qt = torch.empty(q.shape[1], q.shape[0], dtype=torch.uint8, device="cuda")
        st = torch.empty(q.shape[1], q.shape[0] // 128, device="cuda")
        fp8z.fp8z_transpose_rowwise(q, s, qt, st)
        return qt, st

    def forward(self, x):
        n = (torch.empty(x.shape, dtype=torch.uint8, device="cuda"), torch.empty(x.shape[0], x.shape[1] // 128, device="cuda"))
        fp8z.fp8z_layer_norm(x, *self.vectors, None, self.mean, self.rstd, q=n[0], q_scale=n[1])
        h = self.product(n, self.weight(0), self.inner)
        a = self.quantize(torch.relu(h))
        return x + self.product(a, self.weight(1), self.hidden), (n, h, a)

    def backward(self, x, dy, kept):
        """Gradients of the matrices and vectors, and of x."""
        n, h, a = kept
        g = self.quantize(dy)
        dh = self.product(g, self.weight(1, True), self.inner) * (h > 0)
        gh = self.quantize(dh)
        dn = self.product(gh, self.weight(0, True), self.hidden)
        gt, ght = self.columns(g), self.columns(gh)
        fp8z.fp8z_matmul(*gt, *self.columns(a), self.grads[1], dev_status=self.status)
        fp8z.fp8z_matmul(*ght, *self.columns(n), self.grads[0], dev_status=self.status)
        dx = torch.empty_like(x)
        fp8z.fp8z_layer_norm_grad(dn, x, self.vectors[0], self.mean, self.rstd, dx, *self.vector_grads, self.ln_ws)
        return dx + dy

    def update(self, hp):
        fp8z.fp8z_adamw_requant_step_rowmajor(self.p, self.m, self.v, self.maps, self.w_row, self.inv,
                                              int(self.shards[0]["blk_begin"]), int(self.shards[0]["blk_count_real"]), hp,
                                              self.desc, self.table, len(self.entries), w_fp8_t=self.w_col,
                                              inv_scale_t=self.inv_t, dev_status=self.status)

    def step(self, x, target, hp, max_norm=1.0):
        y, kept = self.forward(x)
        diff = y - target
        self.backward(x, diff * (2.0 / diff.numel()), kept)
        fp8z.fp8z_grad_clip(self.clip_list, max_norm, self.norm, self.norm_ws)
        self.update(hp)
        fp8z.fp8z_adamw(self.vector_list, hp)
        return diff.square().mean()


def train(steps=40, seed=0, **sizes):
    block = Block(seed=seed, **sizes)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    mix = torch.randn(block.hidden, block.hidden, generator=gen, device="cuda") / block.hidden ** 0.5
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(block.tokens, block.hidden, generator=gen, device="cuda")
        losses.append(float(block.step(x, x + torch.relu(x @ mix), fp8z.hparams(lr=2e-3, weight_decay=0.0, step=step))))
    assert int(block.status.item()) == 0, fp8z.fp8z_status_string(int(block.status.item()))
    return losses


if __name__ == "__main__":
    got = train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
    for i in range(0, len(got), 10):
        print(f"step {i + 1:4d}  loss {got[i]:.4f}")
    print(f"step {len(got):4d}  loss {got[-1]:.4f}")
