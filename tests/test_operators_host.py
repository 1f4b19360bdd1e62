"""Argument checks of the training operators that need no GPU: every call below is refused (or finds
nothing to do) before any CUDA work, with the documented status; pointers are never dereferenced."""
import ctypes

import pytest

from mxfp8_master_weight_gb300 import _capi
from mxfp8_master_weight_gb300 import build as libbuild

F32, BF16, U8 = _capi.DTYPE_F32, _capi.DTYPE_BF16, _capi.DTYPE_U8
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _capi.load()


def T(dtype, *shape, ptr=P):
    sh = list(shape) + [0] * (2 - len(shape))
    return _capi.Tensor(ctypes.c_void_p(ptr), dtype, len(shape), (ctypes.c_int64 * 2)(*sh))


E = _capi.empty_tensor


def call(fn, tensors, *scalars):
    return fn(*[ctypes.byref(t) for t in tensors], *scalars, None)


def test_checkpoint_save(lib):
    f = lib.mxfp8_checkpoint_save
    x, q, s = T(F32, 100, 200), T(U8, 100, 208), T(U8, 512)
    assert call(f, (x, q, s, E(), E()), -1, 200) == 1
    assert call(f, (x, q, s, E(), E()), 2 ** 31, 1) == 1
    assert call(f, (x, q, s, E(), E()), 2 ** 21, 2 ** 20) == 1      # more than 2^40 elements
    assert call(f, (E(), E(), E(), E(), E()), 0, 200) == 0          # nothing to do
    assert call(f, (E(), q, s, E(), E()), 100, 200) == 4
    assert call(f, (x, E(), E(), E(), E()), 100, 200) == 4
    assert call(f, (x, q, E(), E(), E()), 100, 200) == 4
    assert call(f, (x, E(), E(), q, E()), 100, 200) == 4
    assert call(f, (x, q, s, E(), E()), 101, 200) == 2
    assert call(f, (T(F32, 19999), q, s, E(), E()), 100, 200) == 2  # dense 1-D, too short
    assert call(f, (x, T(U8, 100, 199), s, E(), E()), 100, 200) == 2
    assert call(f, (x, q, T(U8, 511), E(), E()), 100, 200) == 2
    assert call(f, (x, E(), E(), q, T(U8, 1023)), 100, 200) == 2    # columnwise: [200][1] takes 2 tiles
    assert b"1024" in lib.mxfp8_last_error()
    assert call(f, (T(U8, 100, 200), q, s, E(), E()), 100, 200) == 3
    assert call(f, (x, T(F32, 100, 200), s, E(), E()), 100, 200) == 3
    assert call(f, (x, q, T(U8, 512, ptr=P + 8), E(), E()), 100, 200) == 1
    assert call(f, (T(F32, 100, 200, ptr=P + 2), q, s, E(), E()), 100, 200) == 1


def test_checkpoint_restore(lib):
    f = lib.mxfp8_checkpoint_restore
    q, s, y = T(U8, 100, 208), T(U8, 512), T(BF16, 100, 200)
    assert call(f, (q, s, y), 100, 200, 2) == 1
    assert call(f, (E(), E(), E()), 100, 0, 0) == 0
    assert call(f, (E(), s, y), 100, 200, 0) == 4
    assert call(f, (q, E(), y), 100, 200, 0) == 4
    assert call(f, (q, s, E()), 100, 200, 0) == 4
    assert call(f, (q, s, y), 100, 200, 1) == 2                     # columnwise scales are larger
    assert call(f, (q, s, T(U8, 100, 200)), 100, 200, 0) == 3
    assert call(f, (y, s, y), 100, 200, 0) == 3


def test_gemm(lib):
    f = lib.mxfp8_gemm
    a, sa, b, sb, o = T(U8, 64, 256), T(U8, 512), T(U8, 200, 256), T(U8, 1024), T(F32, 64, 200)
    ok = (64, 200, 256, 0, 0, 128, 128)
    t = (a, sa, b, sb, E(), o)

    def with_(scalars=ok, **kw):
        names = ("a", "sa", "b", "sb", "c", "o")
        return call(f, [kw.get(n, v) for n, v in zip(names, t)], *scalars)

    assert with_((-1, 200, 256, 0, 0, 128, 128)) == 1
    assert with_((2 ** 31, 200, 256, 0, 0, 128, 128)) == 1
    assert with_((64, 200, 256, 2, 0, 128, 128)) == 1
    assert with_((64, 200, 256, 0, 0, 64, 128)) == 1
    assert with_((0, 200, 256, 0, 0, 128, 128)) == 0
    assert with_((64, 200, 257, 0, 0, 128, 128)) == 2
    assert with_((64, 200, 256, 1, 0, 128, 128)) == 2               # columnwise: 256 x 64 is another shape
    assert with_((64, 200, 256, 0, 0, 128, 32)) == 2                # scales per 32 take two tiles per 128 rows
    assert with_(a=E()) == 4 and with_(sa=E()) == 4 and with_(b=E()) == 4 and with_(sb=E()) == 4 and with_(o=E()) == 4
    assert with_(a=T(F32, 64, 256)) == 3 and with_(sb=T(F32, 1024)) == 3 and with_(o=T(U8, 64, 200)) == 3
    assert with_(c=T(BF16, 64, 200, ptr=2 * P)) == 3
    assert with_(o=T(F32, 64, 199)) == 2 and with_(c=T(F32, 63, 200, ptr=64 * P)) == 2
    assert with_(sa=T(U8, 512, ptr=P + 4)) == 1
    assert with_(c=T(F32, 64, 200, ptr=P + 64)) == 1                # overlaps out
    assert b"overlaps" in lib.mxfp8_last_error()


def test_layer_norm(lib):
    f, g = lib.mxfp8_layer_norm_forward, lib.mxfp8_layer_norm_backward
    x, w, m = T(BF16, 10, 64), T(F32, 64), T(F32, 10)
    eps = ctypes.c_float(1e-5)
    t = (x, w, E(), x, m, m)
    assert call(f, t, -1, 64, eps) == 1
    assert call(f, t, 10, 64, ctypes.c_float(float("nan"))) == 1
    assert call(f, (E(),) * 6, 0, 64, eps) == 0
    assert call(f, t, 11, 64, eps) == 2 and call(f, t, 10, 65, eps) == 2
    assert call(f, (x, T(F32, 63), E(), x, m, m), 10, 64, eps) == 2
    assert call(f, (x, w, T(BF16, 64), x, m, m), 10, 64, eps) == 3
    assert call(f, (x, w, E(), T(F32, 10, 64), m, m), 10, 64, eps) == 3
    assert call(f, (x, w, E(), x, T(BF16, 10), m), 10, 64, eps) == 3
    assert call(f, (x, E(), E(), x, m, m), 10, 64, eps) == 4
    need = lib.mxfp8_layer_norm_workspace_size(10, 64)
    assert need > 0 and lib.mxfp8_layer_norm_workspace_size(-1, 64) == -1
    assert lib.mxfp8_layer_norm_workspace_size(10 ** 6, 64) >= need
    ws, q, s = T(U8, need), T(U8, 10, 64), T(U8, 512)

    def back(dy=x, x_=x, xs=None, w_=w, mean=m, rstd=m, dx=x, dw=w, db=None, ws_=ws, rows=10, cols=64):
        return call(g, (dy, x_, xs or E(), w_, mean, rstd, dx, dw, db or E(), ws_), rows, cols)

    assert back(rows=-1) == 1 and back(cols=0) == 0
    assert back(dw=E()) == 4 and back(dy=E()) == 4 and back(x_=E()) == 4 and back(ws_=E()) == 4
    assert back(x_=T(F32, 10, 64)) == 3 and back(dx=T(F32, 10, 64)) == 3 and back(dw=T(BF16, 64)) == 3
    assert back(x_=q) == 4                                          # codes without their scales
    assert back(xs=s) == 1                                          # scales without codes
    assert back(x_=q, xs=T(U8, 511)) == 2 and back(x_=q, xs=T(U8, 512, ptr=P + 1)) == 1
    assert back(ws_=T(U8, need - 1)) == 2 and back(ws_=T(U8, need, ptr=P + 8)) == 1
    assert back(db=T(F32, 63)) == 2 and back(w_=T(F32, 63)) == 2
