"""8-bit moments of fp8z_adamw wherever they lie: whole runs of an aligned tensor, runs of a tensor that starts between
boundaries, and the ends of tensors take the same roots and quotients, so that the same numbers give the same bits."""
import numpy as np
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

from test_gpu_adamw import BF16, lists

pytestmark = pytest.mark.gpu

SHORT = 1280                                                 # ten runs: too few to be taken several at a time


def everywhere(d, n, hp, some):
    """A step of d, of the same one element behind a boundary, and of its first `some` elements in short tensors."""
    lead = {k: torch.cat([x[:1], x])[1:] for k, x in d.items()}
    short = {k: x.clone() for k, x in d.items()}
    parts = [{k: x[i // 128:(i + SHORT) // 128] if k.endswith("scale") else x[i:i + SHORT] for k, x in short.items()}
             for i in range(0, some, SHORT)]
    assert lead["p"].data_ptr() % 16 and lead["m"].data_ptr() % 4
    for ds in ([d], [lead], parts):
        fp8z.fp8z_adamw(lists(ds), hp)
    torch.cuda.synchronize()
    for other, until in ((lead, n), (short, some)):
        for k in ("p", "m", "v", "m_scale", "v_scale", "copy"):
            end = until // 128 if k.endswith("scale") else until
            a, b = d[k][:end].view(torch.uint8), other[k][:end].contiguous().view(torch.uint8)
            assert torch.equal(a, b), (k, int((a != b).sum()))


def test_the_same_bits_wherever_they_lie():
    n = 1 << 25
    g = torch.Generator(device="cuda").manual_seed(3)
    q = lambda: torch.randint(1, 127, (n,), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    s = lambda: 1e-6 * torch.exp(torch.randn(n // 128, generator=g, device="cuda"))
    d = dict(p=torch.zeros(n, device="cuda"), g=torch.randn(n, generator=g, device="cuda") * 1e-3, m=q(), v=q(), m_scale=s(),
             v_scale=s(), copy=torch.zeros(n, dtype=BF16, device="cuda"))
    everywhere(d, n, fp8z.hparams(lr=1.0, weight_decay=0.0, step=5), SHORT * 800)        # p starts at 0: it becomes the update
    assert d["p"].isfinite().all()


def test_quotients_that_an_approximation_rounds_otherwise():
    """Pairs m', d whose approximate quotient with one correction is a unit off the IEEE one: with beta1 = 1/2, beta2 = 1/4, no gradient
    and codes of 1 the update is m_scale / 2 over v_scale / 2."""
    pairs = np.array([0x3f9b5d8e, 0x3ffdc0bb, 0x3fc46121, 0x3fe4bef1, 0x3ff3009d, 0x3ffd23cd, 0x3fba00ce, 0x3fdcf3bf, 0x3fdfbee6,
                      0x3fe6c387, 0x3fd39477, 0x3ffbf539], np.uint32).view(np.float32).reshape(-1, 2)
    runs = 120
    n = runs * 128
    each = torch.from_numpy(np.resize(pairs, (runs, 2)) * np.float32(2)).cuda()
    one = torch.full((n,), 0x38, dtype=torch.uint8, device="cuda")
    d = dict(p=torch.zeros(n, device="cuda"), g=torch.zeros(n, device="cuda"), m=one, v=one.clone(), m_scale=each[:, 0].contiguous(),
             v_scale=each[:, 1].contiguous(), copy=torch.zeros(n, dtype=BF16, device="cuda"))
    hp = fp8z.hparams(lr=1.0, beta1=0.5, beta2=0.25, eps=1e-30, weight_decay=0.0, step=1000)
    everywhere(d, n, hp, n)
    got, want = -d["p"].cpu().numpy().reshape(runs, 128)[:6, 0], pairs[:, 0].astype(np.float64) / pairs[:, 1]
    assert (np.abs(got - want) <= 2.0 ** -23 * want).all()
