"""Argument checks of the operators of a layer with FP8 weights, on the host: every call
below returns before any CUDA call, so no pointer here is dereferenced."""
import ctypes
import math

import numpy as np
import pytest

from blockwise_fp8_zero_gb300 import fp8z

P, ODD = 0x10000, 0x10001
F32, BF16, F16, I32, I64 = fp8z.FP8Z_F32, fp8z.FP8Z_BF16, fp8z.FP8Z_F16, fp8z.FP8Z_I32, fp8z.FP8Z_I64
EINVAL, EALIGN, ENOSPACE, OK = fp8z.FP8Z_EINVAL, fp8z.FP8Z_EALIGN, fp8z.FP8Z_ENOSPACE, fp8z.FP8Z_OK
ROWS, K = fp8z.FP8Z_GROUP_ROWS, fp8z.FP8Z_GROUP_K


@pytest.fixture(scope="module")
def L():
    from blockwise_fp8_zero_gb300 import build
    build.build()
    return fp8z.lib()


def test_sizes_of_structures_match_the_header():
    assert ctypes.sizeof(fp8z.fp8z_matmul_args) == 112 and ctypes.sizeof(fp8z.fp8z_layer_norm_args) == 72
    assert ctypes.sizeof(fp8z.fp8z_adamw_params) == 56
    assert fp8z.adamw_tensor_dtype.itemsize == 80 and fp8z.adamw_chunk_dtype.itemsize == 64


def test_matmul(L):
    def args(**kw):
        a = dict(m=4, n=200, k=256, a_ld=256, b_ld=256, out_ld=200, a_scale_ld=2, b_scale_ld=2, b_group=0, b_scale_group=0,
                 out_group=0, b_scale_rows=128, out_dtype=BF16, accumulate=0, groups=0, group_by=ROWS, offsets_dtype=I32)
        a.update(kw)
        return ctypes.byref(fp8z.fp8z_matmul_args(**a))

    base = dict(a=P, sa=P, b=P, sb=P, off=P, out=P, ws=None, wsb=0, st=None)

    def call(shape=None, **kw):
        c = {**base, **kw}
        return L.fp8z_matmul(c["a"], c["sa"], c["b"], c["sb"], shape or args(), c["off"], c["out"], c["ws"], c["wsb"], c["st"], None)

    bank = dict(groups=3, b_group=200 * 256, b_scale_group=4)
    grads = dict(groups=3, group_by=K, b_scale_rows=1, out_group=4 * 200, out_dtype=F32)
    assert call(args(m=0)) == OK and call(args(n=0, out_ld=0)) == OK
    for bad in (dict(m=-1), dict(n=2 ** 31), dict(k=-1), dict(a_ld=255), dict(b_ld=100), dict(out_ld=199), dict(a_scale_ld=1),
                dict(b_scale_ld=1), dict(b_scale_rows=64), dict(out_dtype=I32), dict(accumulate=2), dict(accumulate=1),
                dict(groups=-1), dict(groups=257, **{k: v for k, v in bank.items() if k != "groups"}), dict(bank, group_by=2),
                dict(bank, offsets_dtype=F32), dict(bank, b_scale_rows=1), dict(bank, b_group=200 * 256 - 1), dict(bank, b_scale_group=3),
                dict(grads, b_scale_rows=128), dict(grads, out_group=4 * 200 - 1), dict(m=2 ** 30, n=2 ** 30, out_ld=2 ** 30)):
        assert call(args(**bad)) == EINVAL, bad
        assert L.fp8z_matmul_workspace(P, P, args(**bad)) == EINVAL, bad
    for bad in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None)):
        assert call(**bad) == EINVAL, bad
    assert call(args(**bank), off=None) == EINVAL
    for bad in (dict(sa=P + 2), dict(sb=P + 1), dict(out=ODD), dict(st=P + 2), dict(ws=P + 16)):
        assert call(**bad) == EALIGN, bad
    assert call(args(out_dtype=F32), out=P + 2) == EALIGN
    assert call(args(**bank), off=P + 2) == EALIGN and call(args(**bank, offsets_dtype=I64), off=P + 4) == EALIGN
    # operands that a tensor map cannot step over need workspace
    assert L.fp8z_matmul_workspace(P, P, args()) == 0
    need = L.fp8z_matmul_workspace(P, ODD, args())
    assert need == 200 * 256 and L.fp8z_matmul_workspace(P, P, args(a_ld=257)) == 1024
    assert L.fp8z_matmul_workspace(P, ODD, args(**bank)) == 3 * 200 * 256
    assert call(b=ODD) == EINVAL and call(b=ODD, ws=P, wsb=need - 1) == ENOSPACE


def test_layer_norm(L):
    def args(**kw):
        a = dict(rows=4, cols=256, x_ld=256, y_ld=256, dy_ld=256, dx_ld=256, dtype=BF16, param_dtype=F32, pow2=0, accumulate=0,
                 eps=1e-5, reserved=0)
        a.update(kw)
        return ctypes.byref(fp8z.fp8z_layer_norm_args(**a))

    base = dict(x=P, w=P, b=P, y=P, mean=P, rstd=P, q=None, s=None)

    def fwd(a=None, **kw):
        c = {**base, **kw}
        return L.fp8z_layer_norm(c["x"], c["w"], c["b"], a or args(), c["y"], c["mean"], c["rstd"], c["q"], c["s"], None)

    assert fwd(args(rows=0)) == OK
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=2 ** 25), dict(x_ld=255), dict(y_ld=255), dict(dtype=I32), dict(param_dtype=F16),
                dict(pow2=2), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)):
        assert fwd(args(**bad)) == EINVAL, bad
    for bad in (dict(x=None), dict(y=None, mean=None, rstd=None), dict(q=P), dict(s=P)):
        assert fwd(**bad) == EINVAL, bad
    assert fwd(args(cols=200), q=P, s=P) == EINVAL
    for bad in (dict(x=ODD), dict(y=ODD), dict(w=P + 2), dict(b=P + 1), dict(mean=P + 2), dict(rstd=P + 2), dict(q=P + 8, s=P),
                dict(q=P, s=P + 2), dict(q=P, s=P, x=P + 8), dict(q=P, s=P, w=P + 4)):
        assert fwd(**bad) == EALIGN, bad
    size = L.fp8z_layer_norm_grad_workspace(4, 256)
    assert size > 0 and L.fp8z_layer_norm_grad_workspace(-1, 256) == EINVAL and L.fp8z_layer_norm_grad_workspace(4, 0) == EINVAL
    gb = dict(dy=P, x=P, w=P, mean=P, rstd=P, dx=P, dw=P, db=P, ws=P, wsb=size)

    def grad(a=None, **kw):
        c = {**gb, **kw}
        return L.fp8z_layer_norm_grad(c["dy"], c["x"], c["w"], c["mean"], c["rstd"], a or args(), c["dx"], c["dw"], c["db"], c["ws"],
                                      c["wsb"], None)
    for bad in (dict(rows=-1), dict(dy_ld=255), dict(dx_ld=255), dict(accumulate=2), dict(param_dtype=F16)):
        assert grad(args(**bad)) == EINVAL, bad
    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(ws=None)):
        assert grad(**bad) == EINVAL, bad
    for bad in (dict(dy=ODD), dict(dx=ODD), dict(dw=P + 2), dict(db=P + 2), dict(mean=P + 1), dict(ws=P + 8)):
        assert grad(**bad) == EALIGN, bad
    assert grad(wsb=size - 1) == ENOSPACE


def tensor(**kw):
    t = np.zeros(1, fp8z.adamw_tensor_dtype)
    v = dict(p=P, g=2 * P, m=3 * P, v=4 * P, m_scale=0, v_scale=0, copy=0, count=8193, g_dtype=BF16, copy_dtype=BF16, state_bits=32)
    v.update(kw)
    for k, x in v.items():
        t[k] = x
    return t


def encode(L, t, cap=None):
    chunks = ctypes.c_int64(-1)
    out = None if cap is None else np.zeros(max(cap, 1), fp8z.adamw_chunk_dtype)
    rc = L.fp8z_encode_adamw_list(None if t is None else t.ctypes.data, 0 if t is None else len(t),
                                  None if out is None else out.ctypes.data, cap or 0, ctypes.byref(chunks))
    return rc, chunks.value, out


def test_encode_adamw_list(L):
    assert encode(L, None)[:2] == (OK, 0)
    assert encode(L, tensor())[:2] == (OK, 2)
    t = np.concatenate([tensor(state_bits=8, m_scale=5 * P, v_scale=6 * P, copy=7 * P), tensor(count=0, p=0), tensor(count=1, g_dtype=F32)])
    rc, n, out = encode(L, t, 3)
    assert (rc, n) == (OK, 3) and out["count"].tolist() == [8192, 1, 1]
    assert out["p"].tolist() == [P, P + 8192 * 4, P] and out["g"].tolist() == [2 * P, 2 * P + 8192 * 2, 2 * P]
    assert out["m"].tolist() == [3 * P, 3 * P + 8192, 3 * P] and out["m_scale"].tolist() == [5 * P, 5 * P + 64 * 4, 0]
    assert out["copy"].tolist() == [7 * P, 7 * P + 8192 * 2, 0] and out["copy_dtype"].tolist() == [BF16, BF16, -1]
    assert encode(L, t, 2)[0] == ENOSPACE
    for bad in (dict(p=0), dict(g=0), dict(m=0), dict(v=0), dict(count=-1), dict(g_dtype=I32), dict(state_bits=16),
                dict(copy=P, copy_dtype=F32), dict(state_bits=8, m_scale=P), dict(state_bits=8, v_scale=P)):
        assert encode(L, tensor(**bad))[0] == EINVAL, bad
    for bad in (dict(p=P + 2), dict(g=ODD), dict(m=P + 2), dict(v=ODD), dict(copy=ODD), dict(state_bits=8, m_scale=P + 2, v_scale=P)):
        assert encode(L, tensor(**bad))[0] == EALIGN, bad
    chunks = ctypes.c_int64(0)
    assert L.fp8z_encode_adamw_list(None, 1, None, 0, ctypes.byref(chunks)) == EINVAL
    assert L.fp8z_encode_adamw_list(None, 0, None, 0, None) == EINVAL


def test_adamw(L):
    def call(list_=P, chunks=1, factor=None, hp=True, **kw):
        p = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1, decay_mode=0)
        p.update(kw)
        return L.fp8z_adamw(list_, chunks, ctypes.byref(fp8z.fp8z_adamw_params(**p)) if hp else None, factor, None)
    assert call(chunks=0, list_=None) == OK
    for bad in (dict(list_=None), dict(chunks=-1), dict(chunks=2 ** 31), dict(hp=False), dict(lr=-1.0), dict(lr=math.nan), dict(beta1=1.0),
                dict(beta1=1.0 - 1e-12), dict(beta2=-0.1), dict(eps=0.0), dict(eps=1e-60), dict(weight_decay=math.inf), dict(step=0),
                dict(decay_mode=2)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(list_=P + 4), dict(factor=P + 2)):
        assert call(**bad) == EALIGN, bad


def test_hparams_keep_their_64_bits():
    hp = fp8z.hparams(lr=1e-4, beta1=0.9)
    p = fp8z._adamw_params(hp)
    assert p.lr == 1e-4 and p.beta1 == 0.9 and p.beta2 == 0.95
    hp.lr = 3e-4                                     # the field wins once it is another number
    assert fp8z._adamw_params(hp).lr == ctypes.c_float(3e-4).value and fp8z._adamw_params(hp).beta1 == 0.9
    raw = fp8z.fp8z_adamw_hparams(1e-4, 0.9, 0.95, 1e-8, 0.1, 7, 448.0, 1e-6, 0, 1)
    p = fp8z._adamw_params(raw)
    assert p.beta1 == ctypes.c_float(0.9).value and p.step == 7 and p.decay_mode == 1


def test_binding_refuses_host_tensors():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("the binding asks for the current device first")
    with pytest.raises(ValueError):
        fp8z.fp8z_layer_norm(torch.zeros(2, 8), None, None, None, None, None)


def test_matmul_tiles_of_all_groups(L):
    """Rows of a bank are counted once, results of groups of columns for each group: at most 2^26 tiles."""
    def size(**kw):
        a = dict(m=2 ** 18, n=7168, k=2048, a_ld=2048, b_ld=2048, out_ld=7168, a_scale_ld=16, b_scale_ld=16, b_group=7168 * 2048,
                 b_scale_group=56 * 16, out_group=2 ** 18 * 7168, b_scale_rows=128, out_dtype=F32, accumulate=0, groups=256,
                 group_by=ROWS, offsets_dtype=I32)
        a.update(kw)
        return L.fp8z_matmul_workspace(P, P, ctypes.byref(fp8z.fp8z_matmul_args(**a)))
    assert size() == 0 and size(m=2 ** 24) == 0 and size(m=2 ** 25) == EINVAL
    assert size(group_by=K, b_scale_rows=1) == EINVAL and size(group_by=K, b_scale_rows=1, m=2 ** 14, out_group=2 ** 14 * 7168) == 0
