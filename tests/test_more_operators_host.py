"""Argument checks of RMS norm, NVFP4 operands and their layers that need no GPU: every call below is refused (or finds
nothing to do) before any CUDA work, with the documented status; pointers are never dereferenced."""
import ctypes

import pytest
import torch

from mxfp8_master_weight_gb300 import _capi, api, linear
from mxfp8_master_weight_gb300 import build as libbuild

F32, BF16, U8 = _capi.DTYPE_F32, _capi.DTYPE_BF16, _capi.DTYPE_U8
P = 0x10000
FAR = 1 << 24  # buffers this far apart do not overlap


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


def test_rms_norm_forward(lib):
    at = lambda i: P + i * FAR  # noqa: E731
    base = dict(x=T(BF16, 10, 200), r=T(BF16, 10, 200, ptr=at(1)), w=T(F32, 200, ptr=at(2)), s=T(BF16, 10, 200, ptr=at(3)),
                y=T(BF16, 10, 200, ptr=at(4)), q=T(U8, 10, 208, ptr=at(5)), qs=T(U8, 512, ptr=at(6)), a=T(F32, 1, ptr=at(7)),
                rs=T(F32, 10, ptr=at(8)))

    def f(rows=10, cols=200, eps=1e-5, **kw):
        return call(lib.mxfp8_rms_norm_forward, [kw.get(k, v) for k, v in base.items()], rows, cols, ctypes.c_float(eps))

    assert f(rows=-1) == 1 and f(cols=2 ** 31) == 1 and f(eps=-1.0) == 1 and f(eps=float("nan")) == 1
    assert f(rows=0) == 0 and f(cols=0) == 0
    assert f(x=E()) == 4 and f(w=E()) == 4 and f(y=E(), q=E()) == 4 and f(qs=E()) == 4
    assert f(rows=11) == 2 and f(cols=201) == 2 and f(w=T(F32, 199)) == 2 and f(q=T(U8, 10, 199)) == 2
    assert f(qs=T(U8, 511, ptr=at(6))) == 2 and f(rs=T(F32, 9)) == 2 and f(r=T(BF16, 9, 200)) == 2
    assert f(x=T(U8, 10, 200)) == 3 and f(r=T(F32, 10, 200, ptr=at(1))) == 3 and f(s=T(F32, 10, 200, ptr=at(3))) == 3
    assert f(y=T(F32, 10, 200, ptr=at(4))) == 3 and f(q=T(BF16, 10, 208)) == 3 and f(a=T(BF16, 1)) == 3 and f(rs=T(BF16, 10)) == 3
    assert f(w=T(U8, 200)) == 3
    assert f(qs=T(U8, 512, ptr=at(6) + 8)) == 1
    # outputs that lie over an input without being it, or over one another
    assert f(s=T(BF16, 10, 200, ptr=P + 16)) == 1 and f(y=T(BF16, 10, 200, ptr=at(1) + 4)) == 1
    assert f(s=T(BF16, 10, 208)) == 1 and f(y=base["s"]) == 1
    assert b"overlaps" in lib.mxfp8_last_error()


def test_rms_norm_backward(lib):
    need = lib.mxfp8_rms_norm_workspace_size(10, 64)
    assert need > 0 and lib.mxfp8_rms_norm_workspace_size(-1, 64) == -1 and lib.mxfp8_rms_norm_workspace_size(0, 64) == 0
    assert lib.mxfp8_rms_norm_workspace_size(10 ** 6, 64) >= need
    at = lambda i: P + i * FAR  # noqa: E731
    base = dict(dy=T(BF16, 10, 64), ds=T(BF16, 10, 64, ptr=at(1)), x=T(BF16, 10, 64, ptr=at(2)), w=T(F32, 64, ptr=at(3)),
                rs=T(F32, 10, ptr=at(4)), dx=T(BF16, 10, 64, ptr=at(5)), dw=T(F32, 64, ptr=at(6)), ws=T(U8, need, ptr=at(7)))

    def f(rows=10, cols=64, **kw):
        return call(lib.mxfp8_rms_norm_backward, [kw.get(k, v) for k, v in base.items()], rows, cols)

    assert f(rows=-1) == 1 and f(cols=0) == 0
    assert f(dy=E()) == 4 and f(x=E()) == 4 and f(w=E()) == 4 and f(rs=E()) == 4 and f(dx=E()) == 4 and f(dw=E()) == 4 and f(ws=E()) == 4
    assert f(rows=11) == 2 and f(cols=65) == 2 and f(ws=T(U8, need - 1, ptr=at(7))) == 2 and f(dw=T(F32, 63)) == 2
    assert f(ds=T(F32, 10, 64, ptr=at(1))) == 3 and f(x=T(F32, 10, 64, ptr=at(2))) == 3 and f(dx=T(F32, 10, 64, ptr=at(5))) == 3
    assert f(dw=T(BF16, 64)) == 3 and f(dy=T(U8, 10, 64)) == 3 and f(ws=T(F32, need, ptr=at(7))) == 3
    assert f(ws=T(U8, need, ptr=at(7) + 8)) == 1
    assert f(dx=T(BF16, 10, 64, ptr=P + 2)) == 1 and f(dx=T(BF16, 10, 72, ptr=at(2))) == 1


def test_nvfp4_amax_quantize_restore(lib):
    f = lib.nvfp4_tensor_amax
    x, a = T(F32, 10, 64), T(F32, 1)
    assert call(f, (x, a), -1, 64, 0) == 1 and call(f, (x, a), 10, 64, 2) == 1
    assert call(f, (x, E()), 10, 64, 0) == 4 and call(f, (E(), a), 10, 64, 0) == 4
    assert call(f, (x, a), 11, 64, 0) == 2 and call(f, (T(U8, 10, 64), a), 10, 64, 0) == 3 and call(f, (x, T(BF16, 1)), 10, 64, 0) == 3
    assert call(f, (E(), a), 0, 64, 1) == 0

    f = lib.nvfp4_quantize
    q, s, qc, sc = T(U8, 10, 32), T(U8, 512), T(U8, 64, 5), T(U8, 512)
    assert call(f, (x, a, q, s, qc, sc), 10, -1) == 1 and call(f, (E(),) * 6, 0, 64) == 0
    assert call(f, (E(), a, q, s, qc, sc), 10, 64) == 4 and call(f, (x, E(), q, s, qc, sc), 10, 64) == 4
    assert call(f, (x, a, E(), E(), E(), E()), 10, 64) == 4 and call(f, (x, a, q, E(), E(), E()), 10, 64) == 4
    assert call(f, (x, a, E(), E(), qc, E()), 10, 64) == 4
    assert call(f, (x, a, T(U8, 10, 31), s, qc, sc), 10, 64) == 2 and call(f, (x, a, q, s, T(U8, 64, 4), sc), 10, 64) == 2
    assert call(f, (x, a, q, T(U8, 511), qc, sc), 10, 64) == 2 and call(f, (x, a, q, s, T(U8, 63, 5), sc), 10, 64) == 2
    assert call(f, (T(U8, 10, 64), a, q, s, qc, sc), 10, 64) == 3 and call(f, (x, a, T(F32, 10, 32), s, qc, sc), 10, 64) == 3
    assert call(f, (x, T(BF16, 1), q, s, qc, sc), 10, 64) == 3
    assert call(f, (x, a, q, T(U8, 512, ptr=P + 4), qc, sc), 10, 64) == 1

    f = lib.nvfp4_restore
    y = T(BF16, 10, 64)
    assert call(f, (q, s, a, y), 2 ** 31, 64) == 1 and call(f, (E(),) * 4, 10, 0) == 0
    assert call(f, (E(), s, a, y), 10, 64) == 4 and call(f, (q, E(), a, y), 10, 64) == 4 and call(f, (q, s, E(), y), 10, 64) == 4
    assert call(f, (q, s, a, E()), 10, 64) == 4 and call(f, (q, s, a, y), 10, 65) == 2 and call(f, (q, s, a, T(U8, 10, 64)), 10, 64) == 3


def test_nvfp4_lay_out(lib):
    f = lib.nvfp4_lay_out
    q, o, t = T(U8, 10, 32), T(U8, 10, 32, ptr=P + FAR), T(U8, 64, 16, ptr=P + FAR)
    assert call(f, (q, o), 10, 63, 0) == 1 and call(f, (q, o), 10, 64, 2) == 1 and call(f, (q, o), -1, 64, 0) == 1
    assert call(f, (E(), E()), 0, 64, 0) == 0
    assert call(f, (E(), o), 10, 64, 0) == 4 and call(f, (q, E()), 10, 64, 0) == 4
    assert call(f, (q, o), 11, 64, 0) == 2 and call(f, (q, o), 10, 64, 1) == 2 and call(f, (q, T(U8, 64, 4, ptr=P + FAR)), 10, 64, 1) == 2
    assert call(f, (T(F32, 10, 32), o), 10, 64, 0) == 3 and call(f, (q, T(F32, 64, 16, ptr=P + FAR)), 10, 64, 1) == 3
    assert call(f, (q, q), 10, 64, 0) == 1 and call(f, (q, T(U8, 64, 16, ptr=P + 16)), 10, 64, 1) == 1


def test_nvfp4_gemm(lib):
    base = dict(a=T(U8, 64, 128), sa=T(U8, 2048), ga=T(F32, 1), b=T(U8, 200, 128), sb=T(U8, 4096), gb=T(F32, 1), c=E(),
                o=T(F32, 64, 200, ptr=P + FAR))

    def f(m=64, n=200, k=256, **kw):
        return call(lib.nvfp4_gemm, [kw.get(i, v) for i, v in base.items()], m, n, k)

    assert f(m=-1) == 1 and f(k=2 ** 31) == 1 and f(m=0) == 0 and f(n=0) == 0
    for name in ("a", "sa", "ga", "b", "sb", "gb", "o"):
        assert f(**{name: E()}) == 4, name
    assert f(k=257) == 2 and f(m=65) == 2 and f(n=201) == 2 and f(sa=T(U8, 2047)) == 2 and f(o=T(F32, 64, 199, ptr=P + FAR)) == 2
    assert f(a=T(F32, 64, 128)) == 3 and f(ga=T(BF16, 1)) == 3 and f(o=T(U8, 64, 200, ptr=P + FAR)) == 3
    assert f(c=T(BF16, 64, 200, ptr=P + 2 * FAR)) == 3
    # operands are fetched as they lie: base and row stride on 16 bytes
    assert f(a=T(U8, 64, 128, ptr=P + 8)) == 1 and f(b=T(U8, 200, 136)) == 1 and f(sb=T(U8, 4096, ptr=P + 8)) == 1
    assert f(a=T(U8, 64 * 125), k=250) == 1
    assert f(c=T(F32, 64, 200, ptr=P + FAR + 64)) == 1
    assert b"overlaps" in lib.mxfp8_last_error()


def test_python_views_narrower_than_the_matrix():
    """A slice of a wider buffer keeps the buffer's stride: its own width is checked before the library sees it."""
    with pytest.raises(ValueError):
        api.nvfp4_quantize(torch.zeros(4, 16), torch.zeros(1), None, None, None, None, 4, 16)  # not on the GPU


def refused(status, fn, *a, **kw):
    with pytest.raises(api.MXFP8Error) as e:
        fn(*a, **kw)
    return e.value.status == status


def test_layers():
    assert refused(1, linear.RMSNormLinear, 8, 16, 16, device="cpu", weights="fp4")
    assert refused(1, linear.RMSNormLinear, 8, 15, 16, device="cpu", weights="nvfp4")
    assert refused(1, linear.RMSNormLinear, 8, 16, 16, device="cpu", weights="nvfp4", bounds=[0, 100, 256])
    layer = linear.RMSNormLinear(8, 16, 32, device="cpu", weights="nvfp4")
    x, dy = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.bfloat16)
    for bad in (x[:7], torch.cat([x, x]), torch.cat([x, x], 1), x.view(1, 8, 16)):
        assert refused(2, layer.forward, bad) and refused(2, layer.forward, x, bad) and refused(2, layer.backward, dy, bad)
    assert refused(3, layer.forward, x.float()) and refused(3, layer.forward, x, x.float()) and refused(2, layer.backward, x)
    assert refused(1, layer.refresh, [x, x]) and refused(2, layer.refresh, [x])
    assert refused(2, layer.weights.h4.save, dy) and refused(2, layer.weights.h4.quantize, x[:4])
    serving = linear.RMSNormLinear(8, 16, 32, device="cpu", weights="nvfp4", training=False)
    assert refused(1, serving.backward, dy)
