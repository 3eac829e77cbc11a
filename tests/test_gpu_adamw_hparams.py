"""One hparams() object in fp8z_adamw and in the FP8 step.  The step takes its 32-bit fields, fp8z_adamw the numbers that
hparams() was given: the same bits where FP32 holds the numbers, else what the scalars differ by."""
import numpy as np
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

from test_gpu_adamw import F32, bits_of, f, lists, make, scalars

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rounded(**kw):
    return {k: float(f(x)) for k, x in kw.items()}


@pytest.mark.parametrize("post", [0, 1])
def test_numbers_of_32_bits_move_a_parameter_as_the_step_does(oracle, post):
    """hparams() of numbers that FP32 holds exactly: the FP8 step's bits."""
    t, d = make(3 * 16384, F32, 32, None, 5)
    hp = fp8z.hparams(step=7, decay_mode=post, **rounded(lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1))
    o = {k: x.copy() for k, x in t.items()}
    oracle.adamw_requant_step(o["p"], o["g"], o["m"], o["v"], np.zeros(3 * 16384, np.uint8), np.zeros(3, f), 0, 3,
                              oracle.Hparams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, hp.step, hp.fp8_max, hp.min_scale,
                                             hp.scale_mode, hp.decay_mode))
    fp8z.fp8z_adamw(lists([d]), hp)
    torch.cuda.synchronize()
    for k in "pmv":
        assert np.array_equal(bits_of(d[k]), bits_of(o[k])), k


def test_other_numbers_move_it_by_their_rounding(oracle):
    """hparams() of other numbers: the steps differ by what their scalars differ, and by the roundings of both."""
    t, d = make(3 * 16384, F32, 32, None, 6)
    kw = dict(lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    hp = fp8z.hparams(step=7, **kw)
    wide, narrow = scalars(hp), scalars(fp8z.hparams(step=7, **rounded(**kw)))
    off = {k: abs(float(wide[k]) - float(narrow[k])) for k in wide}
    assert off["omb1"] <= 2.0 ** -25 * 0.9 + 2 * U * 0.1 and off["omb2"] <= 2.0 ** -25 * 0.95 + 2 * U * 0.05
    o = {k: x.copy() for k, x in t.items()}
    oracle.adamw_requant_step(o["p"], o["g"], o["m"], o["v"], np.zeros(3 * 16384, np.uint8), np.zeros(3, f), 0, 3,
                              oracle.Hparams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, hp.step, hp.fp8_max, hp.min_scale,
                                             hp.scale_mode, hp.decay_mode))
    fp8z.fp8z_adamw(lists([d]), hp)
    torch.cuda.synchronize()
    g, m, v, p = (np.abs(t[k].astype(np.float64)) for k in "gmvp")
    got = {k: d[k].cpu().numpy().astype(np.float64) for k in "pmv"}
    big_m = float(wide["b1"]) * m + float(wide["omb1"]) * g
    em = (off["b1"] * m + off["omb1"] * g) + 4 * U * big_m
    big_v = float(wide["b2"]) * v + float(wide["omb2"]) * g * g
    ev = (off["b2"] * v + off["omb2"] * g * g) + 6 * U * big_v
    assert (np.abs(got["m"] - o["m"]) <= em).all() and (np.abs(got["v"] - o["v"]) <= ev).all()
    den = np.sqrt(big_v) * float(wide["rs"]) + float(wide["eps"])
    rel = off["size"] / float(wide["size"]) + ev / (2 * big_v + 1e-300) + off["rs"] / float(wide["rs"]) + off["eps"] / float(wide["eps"]) + 16 * U
    upd = float(wide["size"]) / den * (em + big_m * rel)
    assert (np.abs(got["p"] - o["p"]) <= upd + (off["decay"] + 4 * U) * p).all()
