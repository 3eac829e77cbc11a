"""The second moment of fp8z_adamw in 8 bits over many steps, beside FP32's.

Three fraction bits.  While the scale of a run of 128 stands (its largest root does), a root r^ that is
kept goes to the nearest code Q(x) of x = sqrt(b2 r^2 + (1 - b2) g^2).  For b2 > (31/32)^2 x is never below the middle
to the next code down, so that no code falls; a code rises where x passes the middle above it, 1/32 to 1/16 of r^
away.  With K^2 = 1 + ((17/16)^2 - 1) / (1 - b2) a root r that is not rounded obeys r <= K r^ by induction:
 |g| <= K r^:  b2 r^2 + (1 - b2) g^2 <= K^2 r^^2, and r^ does not fall;
 |g| >  K r^:  x > 17/16 r^, so that the code is the nearest of x, at least 16/17 x, and
               K^2 (16/17)^2 (b2 r^^2 + (1 - b2) g^2) >= b2 K^2 r^^2 + (1 - b2) g^2  <=>  (1 - b2) g^2 (K^2 (16/17)^2 - 1)
               >= b2 K^2 r^^2 (1 - (16/17)^2), which holds at g = K r^ with equality and beyond it.
 r^ itself is at most 17/16 of the largest |g| so far, or its start.
A step's FP32 operations move the scale by at most 8 u, u = 2^-24: over T = 100 steps 2^-14; 2^-10 is allowed."""
import numpy as np
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

from test_gpu_adamw import f, lists, value

pytestmark = pytest.mark.gpu

T = 100


def run_states(beta2, kind, seed):
    """T steps from one state with 8-bit and with FP32 moments: roots and codes of every step, gradients, the runs' largest."""
    rng = np.random.default_rng(seed)
    runs = 32
    n, top = runs * 128, f(1e-2)
    size = (top * np.exp2(-rng.random(n) * 9)).astype(f)
    size[::128] = top                                        # one element of each run keeps its scale
    codes = torch.from_numpy(size.reshape(-1, 128) * (f(448) / top)).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)
    scale = torch.full((runs,), float(top / f(448)))
    root = value(codes.numpy()) * np.repeat(scale.numpy(), 128)
    zero = torch.zeros(n)
    eight = dict(p=zero.cuda(), g=zero.cuda(), m=codes.cuda() * 0, v=codes.cuda(), m_scale=torch.ones(runs, device="cuda"), v_scale=scale.cuda(), copy=None)
    wide = dict(p=zero.cuda(), g=eight["g"], m=zero.cuda(), v=torch.from_numpy(root * root).cuda(), copy=None)
    tables = lists([eight]), lists([wide])
    gs, roots, exact, codes = [], [root.astype(np.float64)], [root.astype(np.float64)], [codes.numpy()]
    for i in range(T):
        if kind == "stop":
            g = np.zeros(n)
        elif kind == "fade":
            g = np.clip(rng.normal(size=n) * size * 0.97 ** i, -top, top)
        elif kind == "noise":
            g = np.clip(rng.normal(size=n) * size, -top, top)
        else:
            g = np.minimum(size * 16.0, top)                  # sixteen times what they were
        g = g.astype(f)
        g[::128] = top
        eight["g"].copy_(torch.from_numpy(g))
        for table in tables:
            fp8z.fp8z_adamw(table, fp8z.hparams(lr=1e-3, beta2=beta2, weight_decay=0.0, step=1000 + i))
        gs.append(np.abs(g.astype(np.float64)))
        codes.append(eight["v"].cpu().numpy())
        roots.append(value(codes[-1]).astype(np.float64) * np.repeat(eight["v_scale"].cpu().numpy(), 128))
        exact.append(np.sqrt(wide["v"].cpu().numpy().astype(np.float64)))
    return np.array(gs), np.array(roots), np.array(exact), np.array(codes)


@pytest.mark.parametrize("kind", ["stop", "fade", "noise", "rise"])
@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_second_moment_of_many_steps(beta2, kind):
    g, roots, exact, codes = run_states(beta2, kind, 7)
    slack = 1 + 2.0 ** -10
    assert (np.abs(roots[:, ::128] / roots[0, ::128] - 1) <= 2.0 ** -14).all()            # the runs' largest, and so the scales
    assert (codes[1:] >= codes[:-1]).all()                                                # no code falls
    k = np.sqrt(1 + ((17 / 16) ** 2 - 1) / (1 - beta2))
    assert (exact <= k * roots * slack).all()
    so_far = np.maximum.accumulate(g, 0)
    assert (roots[1:] <= np.maximum(roots[0], 17 / 16 * so_far) * slack).all()
    if kind == "stop":                                       # FP32's fall by sqrt(beta2) a step, these do not
        assert (codes[-1] == codes[0]).all() and (exact[-1, 1::128] < roots[-1, 1::128] * beta2 ** (T / 2) * slack).all()
