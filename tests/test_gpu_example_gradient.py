"""The tied-table example's gradients against the definition in 64 bits, and its clipping.

The example's calls are watched in two steps of a run: what goes into them, the gradients
before the clipping and after it.  The reference takes the same BF16 table and matrix and
computes in 64 bits throughout.  The example rounds x, h, dh, dx and P to BF16 on the way, each by
2^-9 of its size in the norm at the most: five of them, 0.01, against the whole gradient; the
table's two parts are also held against their own sizes, so that one that is lost, has the
wrong sign or lacks its scale is off by more than its own norm."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _reference(ids, after, e, m, scale):
    """(gradient of the table by the loss, by the lookup, gradient of the matrix)"""
    keep = after >= 0
    x = scale * e[ids]
    h = x @ m
    p = torch.softmax(h @ e.t(), 1)
    p.scatter_add_(1, after.clamp(min=0)[:, None], torch.full_like(p[:, :1], -1.0))
    p *= keep[:, None] / keep.sum()
    dh = p @ e
    by_lookup = torch.zeros_like(e).index_add_(0, ids, scale * (dh @ m.t()))
    return p.t() @ h, by_lookup, x.t() @ dh


def test_gradients_and_clipping_of_the_example(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import tied_lm
    from blockwise_fp8_zero_gb300 import build, fp8z
    build.build()
    seen = []
    lookup, loss, clip, unfold = (getattr(fp8z, "fp8z_" + name) for name in (
        "embedding", "linear_xent_grad", "grad_clip", "unfold"))
    main = []

    def watch_unfold(p, entry, w, *a, **kw):
        unfold(p, entry, w, *a, **kw)
        main.append(w)

    def watch_lookup(ids, table, out, scale=1.0, **kw):
        seen.append({"ids": ids.clone(), "e": table.clone(), "m": main[-1].bfloat16(), "scale": scale})
        lookup(ids, table, out, scale=scale, **kw)

    def watch_loss(h, w, after, loss_out, total, dh, dw, ws, **kw):
        loss(h, w, after, loss_out, total, dh, dw, ws, **kw)
        seen[-1].update(after=after.clone(), by_loss=dw.clone())

    def watch_clip(tensors, max_norm, norm, ws, **kw):
        grads = tensors.tensors[0]
        seen[-1].update(before=[g.clone() for g in grads])
        clip(tensors, max_norm, norm, ws, **kw)
        seen[-1].update(clipped=[g.clone() for g in grads], norm=norm.clone(), max_norm=max_norm)

    for name, f in (("unfold", watch_unfold), ("embedding", watch_lookup), ("linear_xent_grad", watch_loss),
                    ("grad_clip", watch_clip)):
        monkeypatch.setattr(fp8z, "fp8z_" + name, f)
    tied_lm.train(steps=2, max_norm=0.5)
    assert len(seen) == 2
    off = lambda got, want, size: float((got.double() - want).norm() / size.norm())  # noqa: E731
    clipped = 0
    for s in seen:
        by_loss, by_lookup, dm = _reference(s["ids"], s["after"], s["e"].double(), s["m"].double(), s["scale"])
        table, matrix = s["before"]
        assert off(s["by_loss"], by_loss, by_loss) <= 0.01
        assert off(table - s["by_loss"], by_lookup, by_lookup) <= 0.01
        assert off(matrix, dm, dm) <= 0.01
        norm = float(torch.cat([g.double().flatten() for g in s["before"]]).norm())
        coef = min(1.0, s["max_norm"] / (norm + 1e-6))
        clipped += coef < 1.0
        assert s["norm"].tolist() == pytest.approx([norm, coef], rel=1e-6)
        for g, b in zip(s["clipped"], s["before"]):
            assert bool(((g.double() - coef * b.double()).abs() <= 2.0 ** -22 * (coef * b.double()).abs() + 1e-45).all())
    assert clipped > 0                               # the limit was below the norm at least once
