"""Argument checks of the operators around the optimizer step, on the host: every
call below returns before any CUDA call, so no pointer here is dereferenced."""
import ctypes
import math

import numpy as np
import pytest

from blockwise_fp8_zero_gb300 import fp8z

P, ODD = 0x10000, 0x10001
F32, BF16, F16, I32, I64 = fp8z.FP8Z_F32, fp8z.FP8Z_BF16, fp8z.FP8Z_F16, fp8z.FP8Z_I32, fp8z.FP8Z_I64
EINVAL, EALIGN, ENOSPACE, OK = fp8z.FP8Z_EINVAL, fp8z.FP8Z_EALIGN, fp8z.FP8Z_ENOSPACE, fp8z.FP8Z_OK


@pytest.fixture(scope="module")
def L():
    from blockwise_fp8_zero_gb300 import build
    build.build()
    return fp8z.lib()


def _encode(L, srcs, numels, sd, dsts=None, dd=None, cap=None, n=None):
    n = len(srcs) if n is None else n
    a = np.array(srcs, np.uint64)
    b = None if dsts is None else np.array(dsts, np.uint64)
    m, s = np.array(numels, np.int64), np.array(sd, np.int32)
    d = None if dd is None else np.array(dd, np.int32)
    chunks = ctypes.c_int64(-1)
    out = None if cap is None else np.zeros(max(cap, 1), fp8z.tensor_chunk_dtype)
    ptr = lambda x: None if x is None else x.ctypes.data
    rc = L.fp8z_encode_tensor_list(ptr(a), ptr(b), ptr(m), ptr(s), ptr(d), n, ptr(out), cap or 0, ctypes.byref(chunks))
    return rc, chunks.value, out


def test_encode_tensor_list(L):
    rc, chunks, _ = _encode(L, [P, 0, P], [8193, 0, 1], [F32, BF16, F16])
    assert (rc, chunks) == (OK, 3)
    rc, chunks, out = _encode(L, [P, 0, 2 * P], [8193, 0, 1], [F32, BF16, F16], [3 * P, 0, 4 * P], [BF16, F32, F32], cap=3)
    assert rc == OK
    assert out["src"].tolist() == [P, P + 8192 * 4, 2 * P] and out["dst"].tolist() == [3 * P, 3 * P + 8192 * 2, 4 * P]
    assert out["count"].tolist() == [8192, 1, 1] and out["src_dtype"].tolist() == [F32, F32, F16]
    assert out["dst_dtype"].tolist() == [BF16, BF16, F32]
    assert _encode(L, [P], [8193], [F32], cap=1)[0] == ENOSPACE
    assert _encode(L, [], [], [])[:2] == (OK, 0)
    for bad in (dict(numels=[-1]), dict(sd=[7]), dict(sd=[I32]), dict(srcs=[0]), dict(dsts=[P], dd=[BF16]),
                dict(dsts=[0], dd=[F32]), dict(dsts=[P]), dict(n=-1)):
        assert _encode(L, **{**dict(srcs=[P], numels=[5], sd=[F32]), **bad})[0] == EINVAL, bad
    assert _encode(L, [ODD], [5], [BF16])[0] == EALIGN
    assert _encode(L, [P + 2], [5], [F32])[0] == EALIGN


def test_grad_norm_and_clip(L):
    def clip(list_=P, chunks=1, scale=1.0, limit=1.0, eps=1e-6, norm=P, ws=P):
        return L.fp8z_grad_clip(list_, chunks, scale, limit, eps, norm, ws, None)
    for bad in (dict(list_=None), dict(chunks=-1), dict(chunks=2 ** 31), dict(scale=math.inf), dict(scale=math.nan),
                dict(limit=-1.0), dict(limit=math.nan), dict(eps=-1.0), dict(eps=math.inf), dict(norm=None), dict(ws=None)):
        assert clip(**bad) == EINVAL, bad
    for bad in (dict(list_=P + 4), dict(norm=P + 2), dict(ws=P + 8)):
        assert clip(**bad) == EALIGN, bad
    assert L.fp8z_grad_norm(P, 1, 1.0, None, P, None) == EINVAL


def test_embedding(L):
    base = dict(ids=P, it=I64, n=4, table=P, tt=BF16, v=9, h=8, ld=8, out=P, ot=BF16, old=8, scale=1.0, st=None)

    def call(**kw):
        a = {**base, **kw}
        return L.fp8z_embedding(a["ids"], a["it"], a["n"], a["table"], a["tt"], a["v"], a["h"], a["ld"], a["out"],
                                a["ot"], a["old"], a["scale"], a["st"], None)
    assert call(n=0) == OK
    for bad in (dict(ids=None), dict(it=F32), dict(n=-1), dict(table=None), dict(tt=I32), dict(v=0), dict(h=0), dict(ld=7),
                dict(out=None), dict(ot=9), dict(old=7), dict(scale=math.nan), dict(n=2 ** 31), dict(h=2 ** 24)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(ids=P + 4), dict(table=ODD), dict(out=P + 2, ot=F32), dict(st=P + 2)):
        assert call(**bad) == EALIGN, bad


def test_embedding_grad(L):
    size = L.fp8z_embedding_grad_workspace(4, 9, 8)
    assert size > 0 and L.fp8z_embedding_grad_workspace(-1, 9, 8) == EINVAL
    assert L.fp8z_embedding_grad_workspace(0, 9, 8) > 0
    base = dict(ids=P, it=I64, n=4, d=P, dt=BF16, ld=8, table=P, tt=F32, v=9, h=8, tld=8, scale=1.0, pad=-1, acc=0, ws=P,
                wsb=size, st=None)

    def call(**kw):
        a = {**base, **kw}
        return L.fp8z_embedding_grad(a["ids"], a["it"], a["n"], a["d"], a["dt"], a["ld"], a["table"], a["tt"], a["v"],
                                     a["h"], a["tld"], a["scale"], a["pad"], a["acc"], a["ws"], a["wsb"], a["st"], None)
    assert call(n=0, acc=1) == OK
    assert call(wsb=size - 1) == ENOSPACE
    for bad in (dict(ids=None), dict(it=BF16), dict(d=None), dict(dt=I64), dict(ld=7), dict(table=None), dict(tt=I64),
                dict(tld=7), dict(acc=2), dict(ws=None), dict(scale=math.inf), dict(n=-1), dict(v=0)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(ids=P + 4), dict(d=ODD), dict(table=P + 2), dict(ws=P + 8), dict(st=ODD)):
        assert call(**bad) == EALIGN, bad


def test_linear_xent(L):
    def args(**kw):
        a = dict(tokens=4, hidden=16, vocab=100, x_ld=16, w_ld=16, dx_ld=16, dw_ld=16, ignore_index=-100, dtype=BF16,
                 targets_dtype=I64, dw_dtype=F32, accumulate_dw=0, reduction=fp8z.FP8Z_MEAN, grad_scale=1.0)
        a.update(kw)
        return ctypes.byref(fp8z.fp8z_xent_args(**a))

    base = dict(x=P, w=P, t=P, loss=P, lse=None, total=P, dx=P, dw=P, ws=P, wsb=1 << 30, st=None)

    def grad(a=None, **kw):
        b = {**base, **kw}
        return L.fp8z_linear_xent_grad(b["x"], b["w"], b["t"], a or args(), b["loss"], b["lse"], b["total"], b["dx"],
                                       b["dw"], b["ws"], b["wsb"], b["st"], None)

    def loss(a=None, **kw):
        b = {**base, **kw}
        return L.fp8z_linear_xent(b["x"], b["w"], b["t"], a or args(), b["loss"], b["lse"], b["total"], b["ws"], b["wsb"],
                                  b["st"], None)
    for bad in (dict(tokens=-1), dict(tokens=2 ** 25), dict(hidden=0), dict(vocab=0), dict(vocab=2 ** 29), dict(tokens=2 ** 24, vocab=2 ** 28),
                dict(hidden=2 ** 20, vocab=2 ** 28, x_ld=2 ** 20, w_ld=2 ** 20), dict(x_ld=15),
                dict(w_ld=15), dict(dtype=F32), dict(targets_dtype=F32), dict(reduction=2)):
        assert loss(args(**bad)) == EINVAL and grad(args(**bad)) == EINVAL, bad
        assert L.fp8z_linear_xent_workspace(P, P, args(**bad), 0, 0) == EINVAL, bad
    for bad in (dict(dx_ld=15), dict(dw_ld=15), dict(dw_dtype=F16), dict(accumulate_dw=2), dict(grad_scale=math.nan)):
        assert grad(args(**bad)) == EINVAL, bad
    for bad in ("x", "w", "t", "loss", "total", "ws"):
        assert loss(**{bad: None}) == EINVAL and grad(**{bad: None}) == EINVAL, bad
    assert grad(dx=None) == EINVAL and grad(dw=None) == EINVAL
    for bad in (dict(x=ODD), dict(w=ODD), dict(t=P + 4), dict(loss=P + 2), dict(lse=ODD), dict(total=ODD), dict(ws=P + 128),
                dict(st=ODD)):
        assert loss(**bad) == EALIGN and grad(**bad) == EALIGN, bad
    assert grad(dw=P + 2) == EALIGN and grad(dx=ODD) == EALIGN


def test_linear_xent_workspace_pieces(L):
    a = fp8z.fp8z_xent_args(tokens=3000, hidden=512, vocab=100000, x_ld=512, w_ld=512, dx_ld=512, dw_ld=512,
                            ignore_index=-100, dtype=BF16, targets_dtype=I64, dw_dtype=F32, accumulate_dw=0, reduction=0,
                            grad_scale=1.0)
    size = lambda grad, words, x=P: L.fp8z_linear_xent_workspace(x, P, ctypes.byref(a), grad, words)
    assert 0 < size(0, 0) < size(1, 256) < size(1, 4096) < size(1, 0)
    assert size(1, 4096) - size(1, 2048) == 2048 * 3000 * 4         # four bytes a word and token
    assert size(1, 0) < size(1, 256) + (1 << 30)                    # the default is at most 1 GiB of one piece
    assert size(0, 0, x=P + 2) >= size(0, 0) + 3000 * 512 * 2       # rows off 16 bytes are copied
    assert L.fp8z_linear_xent_workspace(P, P, ctypes.byref(a), 1, -1) == EINVAL
