"""Layer norm and its gradients against float64.  A thread adds at most 32 values of a row in order
and about 11 more in the reductions (rows past 32768 columns: cols / 8192 * 8); with u = 2^-24 and
T the number of additions, a sum is off by at most T u sum |terms|, and what follows is a
handful of roundings.  Tolerances are those bounds, and half a unit of BF16 where it is stored."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
EPS = 1e-5


def adds(cols):
    return 48 + cols / 1024


def within(got, want, tol, dtype=torch.float32):
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(ref.as64(got) - want)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


def data(rows, cols, dtype, wdtype, seed=0, shift=1.0, stride=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows * 13 + cols)
    wide = torch.zeros(rows, cols + stride, dtype=DT[dtype], device="cuda")
    x = wide[:, :cols]
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") + shift)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(DT[wdtype])
    b = torch.randn(cols, generator=g, device="cuda").to(DT[wdtype])
    return x, w, b


def forward(x, w, b, out=None, eps=EPS):
    rows, cols = x.shape
    y = torch.empty(rows, cols, dtype=x.dtype, device="cuda") if out is None else out
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    api.mxfp8_layer_norm_forward(x, w, b, y, mean, rstd, rows, cols, eps)
    return y, mean, rstd


def check_forward(x64, w64, b64, y, mean, rstd, eps=EPS):
    wy, wm, wr = ref.norm_forward(x64, w64, b64, eps)
    t = adds(x64.shape[1]) * U
    dm = t * np.abs(x64).mean(1)                                  # error of the mean
    within(mean, wm, dm)
    # the mean's error enters the deviations (d) and, squared, the variance; t relative for the rest
    dr = wr * (t + (dm * wr) ** 2 + 2 * U * np.abs(wm) * wr) + 4 * U * wr
    within(rstd, wr, dr)
    dev = np.abs(x64 - wm[:, None])
    tol = np.abs(w64) * (wr[:, None] * (dm[:, None] + 2 * U * (dev + np.abs(x64))) + dev * dr[:, None])
    tol = tol + 8 * U * (np.abs(wy) + (0 if b64 is None else np.abs(b64)))
    within(y, wy, tol, y.dtype)


COLS = [1, 2, 7, 8, 64, 255, 256, 513, 1000, 1024, 1025, 2047, 4096, 6144, 8192, 8200, 16384, 16392, 32768, 40001]


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("cols", COLS)
def test_forward(cols, dtype, wdtype):
    for rows in (1, 9):
        x, w, b = data(rows, cols, dtype, wdtype)
        check_forward(ref.as64(x), ref.as64(w), ref.as64(b), *forward(x, w, b))
        check_forward(ref.as64(x), ref.as64(w), None, *forward(x, w, None))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_far_from_zero(dtype):
    """Rows whose mean is a thousand deviations away: the variance must not cancel."""
    for cols in (100, 3000):
        x, w, b = data(5, cols, dtype, "f32", shift=1000.0 if dtype == "f32" else 100.0)
        check_forward(ref.as64(x), ref.as64(w), ref.as64(b), *forward(x, w, b))


def test_forward_constant_rows():
    """No variance: the deviations are zero (powers of two add exactly) and y is the bias."""
    x = torch.full((4, 1024), 2.0, device="cuda")
    w, b = torch.ones(1024, device="cuda"), torch.randn(1024, device="cuda")
    y, mean, rstd = forward(x, w, b)
    assert torch.equal(y, b.expand(4, -1)) and bool((mean == 2).all())
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [100, 1031, 5000])
def test_strides_and_in_place(cols, dtype):
    x, w, b = data(11, cols, dtype, "f32", stride=5)
    x64 = ref.as64(x)
    wide = torch.full((11, cols + 3), 9.0, dtype=x.dtype, device="cuda")
    y, mean, rstd = forward(x, w, b, wide[:, :cols])
    check_forward(x64, ref.as64(w), ref.as64(b), y, mean, rstd)
    assert bool((wide[:, cols:] == 9.0).all())
    z, m2, r2 = forward(x, w, b, x)
    assert torch.equal(z, y) and torch.equal(m2, mean) and torch.equal(r2, rstd)


def test_nan_and_infinity_stay_in_their_rows():
    x, w, b = data(6, 300, "f32", "f32")
    x[1, 5], x[4, 299] = float("nan"), float("inf")
    y, mean, rstd = forward(x, w, b)
    bad = torch.isnan(y).any(1).cpu()
    assert bad.tolist() == [False, True, False, False, True, False]


def backward(dy, x, s, w, mean, rstd, bias=True, out=None):
    rows, cols = dy.shape
    dx = torch.empty_like(dy) if out is None else out
    dw = torch.full((cols,), 7.0, device="cuda")
    db = torch.full((cols,), 7.0, device="cuda") if bias else None
    ws = torch.full((api.mxfp8_layer_norm_workspace_size(rows, cols) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    api.mxfp8_layer_norm_backward(dy, x, s, w, mean, rstd, dx, dw, db, ws[:ws.numel() - 16], rows, cols)
    assert bool((ws[-16:] == 0xFF).all())
    return dx, dw, db


def check_backward(dy64, x64, w64, mean64, rstd64, dx, dw, db):
    wx, ww, wb = ref.norm_backward(dy64, x64, w64, mean64, rstd64)
    rows, cols = dy64.shape
    t = adds(cols) * U
    xh = np.abs((x64 - mean64[:, None]) * rstd64[:, None])
    dxh = 2 * U * (np.abs(x64) + np.abs(mean64)[:, None]) * rstd64[:, None] + 2 * U * xh
    g = np.abs(dy64 * w64)
    mg, mgx = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    tol = rstd64[:, None] * ((t + 4 * U) * (g + mg + xh * mgx) + dxh * mgx + xh * (g * dxh).mean(1, keepdims=True))
    within(dx, wx, tol + 4 * U * np.abs(wx), dx.dtype)
    tr = (rows / 8 + 64) * U  # a block adds its rows in order, then the partial rows
    within(dw, ww, tr * (np.abs(dy64) * xh).sum(0) + (np.abs(dy64) * dxh).sum(0))
    if db is not None:
        within(db, wb, tr * np.abs(dy64).sum(0))


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("cols", COLS)
def test_backward(cols, dtype, wdtype):
    for rows in (1, 3, 700 if cols <= 8192 else 310):
        x, w, b = data(rows, cols, dtype, wdtype)
        dy = torch.randn(rows, cols, device="cuda").to(x.dtype)
        _, mean, rstd = forward(x, w, b)
        check_backward(*map(ref.as64, (dy, x, w, mean, rstd)), *backward(dy, x, None, w, mean, rstd))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1, 100, 129, 1000, 1024, 3000, 6144, 16400])
def test_backward_from_checkpoint(cols, dtype):
    for rows, pad in ((5, 0), (260, 7), (330, -cols % 16)):
        x, w, b = data(rows, cols, dtype, "f32")
        dy = torch.randn(rows, cols, device="cuda").to(x.dtype)
        _, mean, rstd = forward(x, w, b)
        q = torch.empty(rows, cols + pad, dtype=torch.uint8, device="cuda")
        s = torch.empty(api.mxfp8_swizzled_scales_size(rows, -(-cols // 128)), dtype=torch.uint8, device="cuda")
        api.mxfp8_checkpoint_save(x, q, s, None, None, rows, cols)
        kept = ref.quantise(ref.as64(x))[0]
        check_backward(ref.as64(dy), kept, ref.as64(w), ref.as64(mean), ref.as64(rstd), *backward(dy, q, s, w, mean, rstd))


@pytest.mark.parametrize("cols", [60, 1031, 5000])
def test_backward_strides_in_place_and_no_bias(cols):
    x, w, b = data(40, cols, "bf16", "bf16", stride=3)
    wide = torch.randn(40, cols + 9, device="cuda").bfloat16()
    dy = wide[:, 1:cols + 1]
    keep, dy64 = wide.clone(), ref.as64(dy)
    _, mean, rstd = forward(x, w, b)
    first = backward(dy, x, None, w, mean, rstd, bias=False)
    check_backward(dy64, *map(ref.as64, (x, w, mean, rstd)), *first)
    again = backward(dy, x, None, w, mean, rstd, out=dy)
    assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert torch.equal(wide[:, 0], keep[:, 0]) and torch.equal(wide[:, cols + 1:], keep[:, cols + 1:])


def test_backward_repeatable():
    x, w, b = data(5000, 768, "bf16", "f32")
    dy = torch.randn(5000, 768, device="cuda").bfloat16()
    _, mean, rstd = forward(x, w, b)
    runs = [backward(dy, x, None, w, mean, rstd) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))


@pytest.mark.parametrize("cols", [48, 1500])
def test_gradients_against_differences(cols):
    """Directional derivatives of the 64-bit forward pass, by central differences."""
    x, w, b = data(6, cols, "f32", "f32")
    dy = torch.randn(6, cols, device="cuda")
    _, mean, rstd = forward(x, w, b)
    dx, dw, db = map(ref.as64, backward(dy, x, None, w, mean, rstd))
    x64, w64, b64, dy64 = map(ref.as64, (x, w, b, dy))
    rng = np.random.default_rng(0)
    loss = lambda x_, w_, b_: float((ref.norm_forward(x_, w_, b_, EPS)[0] * dy64).sum())  # noqa: E731
    h = 1e-5
    for k, (grad, base) in enumerate(((dx, x64), (dw, w64), (db, b64))):
        for _ in range(4):
            d = rng.standard_normal(base.shape)
            args = [[x64, w64, b64], [x64, w64, b64]]
            args[0][k], args[1][k] = base + h * d, base - h * d
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            scale = np.linalg.norm(grad) * np.linalg.norm(d)
            # the gradients' own F32 error, and the differences' (h^2 and roundings over h)
            assert abs(diff - float((grad * d).sum())) <= 1e-6 * scale + 1e-6


def test_empty_and_refusals():
    w = torch.ones(64, device="cuda")
    x, m = torch.zeros(4, 64, device="cuda"), torch.zeros(4, device="cuda")
    e = x[:0]
    api.mxfp8_layer_norm_forward(e, w, None, e, m[:0], m[:0], 0, 64)
    dw, db = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    api.mxfp8_layer_norm_backward(e, e, None, w, m[:0], m[:0], e, dw, db, None, 0, 64)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    ws = torch.zeros(api.mxfp8_layer_norm_workspace_size(4, 64), dtype=torch.uint8, device="cuda")

    def status(fn, *a):
        with pytest.raises(api.MXFP8Error) as err:
            fn(*a)
        return err.value.status

    f, g = api.mxfp8_layer_norm_forward, api.mxfp8_layer_norm_backward
    assert status(f, x, None, None, x, m, m, 4, 64) == 4
    assert status(f, x, w[:63], None, x, m, m, 4, 64) == 2
    assert status(f, x, w, w.bfloat16(), x, m, m, 4, 64) == 3
    assert status(f, x, w, None, x.bfloat16(), m, m, 4, 64) == 3
    assert status(f, x, w, None, x, m[:3], m, 4, 64) == 2
    assert status(f, x, w, None, x, m, m, 4, 64, -1.0) == 1
    assert status(f, x, w, None, x, m, m, 5, 64) == 2
    assert status(g, x, x, None, w, m, m, x, dw, db, ws[:-1], 4, 64) == 2
    assert status(g, x, x, None, w, m, m, x, dw, db, None, 4, 64) == 4
    assert status(g, x, x.bfloat16(), None, w, m, m, x, dw, db, ws, 4, 64) == 3
    assert status(g, x, x.to(torch.uint8), None, w, m, m, x, dw, db, ws, 4, 64) == 4
    assert status(g, x, x, ws, w, m, m, x, dw, db, ws, 4, 64) == 1
    assert status(g, x, x, None, w, m, m, x, dw.bfloat16(), db, ws, 4, 64) == 3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [64, 72, 129, 255, 512, 1000, 1024, 1537, 3000, 4095, 6144, 8190, 8192])
def test_many_rows(cols, dtype):
    """Enough rows for persistent blocks: forward, and backward from the input and from its checkpoint
    (odd widths, whose rows start anywhere, among them), from buffers off 16 bytes too."""
    rows = 1900
    for shift in (0, 1):
        flat = lambda: torch.empty(rows * cols + 8, dtype=DT[dtype], device="cuda")[shift:shift + rows * cols].view(rows, cols)  # noqa: E731
        x, w, b = data(rows, cols, dtype, "f32")
        xs, dy, y = flat(), flat(), flat()
        xs.copy_(x)
        dy.copy_(torch.randn(rows, cols, device="cuda"))
        y, mean, rstd = forward(xs, w, b, y)
        check_forward(ref.as64(xs), ref.as64(w), ref.as64(b), y, mean, rstd)
        check_backward(*map(ref.as64, (dy, xs, w, mean, rstd)), *backward(dy, xs, None, w, mean, rstd, out=flat()))
        q = torch.empty(rows * cols + 8, dtype=torch.uint8, device="cuda")[shift:shift + rows * cols].view(rows, cols)
        s = torch.empty(api.mxfp8_swizzled_scales_size(rows, -(-cols // 128)), dtype=torch.uint8, device="cuda")
        api.mxfp8_checkpoint_save(xs, q, s, None, None, rows, cols)
        kept, dy64 = ref.quantise(ref.as64(xs))[0], ref.as64(dy)
        got = backward(dy, q, s, w, mean, rstd, out=dy)  # in place
        check_backward(dy64, kept, ref.as64(w), ref.as64(mean), ref.as64(rstd), *got)
    api.mxfp8_device_status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1217, 256), (2500, 512), (3700, 1024), (1900, 2048), (1400, 4096), (700, 8192)])
def test_many_rows_of_each_ring(rows, cols, dtype):
    """Row counts that fill the blocks of a ring unevenly, each number of blocks per SM; statistics and scales
    that differ from row to row."""
    x, w, b = data(rows, cols, dtype, "f32", shift=0.5)
    x *= torch.exp2(torch.arange(rows, device="cuda") % 9 - 4.0)[:, None].to(x.dtype)
    y, mean, rstd = forward(x, w, b)
    check_forward(ref.as64(x), ref.as64(w), ref.as64(b), y, mean, rstd)
    dy = torch.randn(rows, cols, device="cuda").to(x.dtype)
    check_backward(*map(ref.as64, (dy, x, w, mean, rstd)), *backward(dy, x, None, w, mean, rstd))
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(api.mxfp8_swizzled_scales_size(rows, -(-cols // 128)), dtype=torch.uint8, device="cuda")
    api.mxfp8_checkpoint_save(x, q, s, None, None, rows, cols)
    kept = ref.quantise(ref.as64(x))[0]
    check_backward(ref.as64(dy), kept, ref.as64(w), ref.as64(mean), ref.as64(rstd), *backward(dy, q, s, w, mean, rstd))
    api.mxfp8_device_status()
