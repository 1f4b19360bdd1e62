"""RMS norm and its gradients against float64.

Tolerances, in units of u = 2^-24: a row's sum of squares takes at most `adds` roundings one after another (a thread's
values, then the joining), so rstd is off by (adds / 2 + 4) u; y adds three products and the addition of the residual; a BF16
result half a unit, 2^-8.  ds = rstd (g - xh c) + dsum with c = mean(g xh): the error of c is (adds + 6) u mean|g xh|, every
other step one rounding of its own magnitude.  dw adds at most `rows` terms one after another.  Codes: the scale is that of
a maximum off by y's error, the code that of a value off by as much."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
SHAPES = [(1, 1), (1, 7), (1, 8), (3, 127), (5, 128), (9, 129), (17, 256), (2, 520), (8, 1024), (3, 1031), (4, 4096), (3, 4099),
          (2, 8200), (2, 16384), (1, 16392), (2, 33000), (1, 40001), (130, 64), (300, 200)]
MANY = [(2000, 64), (2000, 65), (1900, 257), (1900, 512), (700, 1000), (1900, 1001), (1900, 2048), (1900, 2047), (1900, 3001),
        (700, 4096), (1900, 4097), (700, 6144), (1900, 6143), (650, 8192), (1900, 8191)]


def adds(cols):
    return max(40, cols // 1024 + 16) + 40


def dirty(shape, dtype):
    return torch.full(shape, -3.0, dtype=dtype, device="cuda")


def inputs(rows, cols, dtype, wdtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 3 * rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dtype])
    r = (torch.randn(rows, cols, generator=g, device="cuda") * 2).to(DT[dtype])
    w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(DT[wdtype])
    return x, r, w


def check_codes(codes, scale, y, tol):
    """Codes and scales of y, whose values are known to a relative `tol`."""
    rows, cols = y.shape
    blocks = -(-cols // 128)
    lo, hi = ref.quantise(y * (1 - tol))[2], ref.quantise(y * (1 + tol))[2]
    tile = scale.cpu().numpy()
    at = lambda r, c: ((r // 128) * (-(-blocks // 4)) + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4  # noqa: E731
    i, j = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    byte = tile[at(i, j)]
    assert np.all((byte == lo) | (byte == hi))
    pad = np.ones(tile.shape, bool)
    pad[at(i, j)] = False
    assert np.all(tile[pad] == 0)
    f = np.repeat(np.ldexp(1.0, byte.astype(np.int32) - 127), 128, axis=1)[:, :cols]
    got = ref.codes_to_values(codes[:, :cols])
    a, b = ref.e4m3(y * (1 - tol) / f), ref.e4m3(y * (1 + tol) / f)
    assert np.all((got >= np.minimum(a, b)) & (got <= np.maximum(a, b)))


def check_forward(x, r, w, eps, total, y, codes, scale, top, rstd):
    s = ref.as64(x) + (0.0 if r is None else ref.as64(r))
    want_r = 1 / np.sqrt((s * s).mean(1) + eps)
    want = s * want_r[:, None] * ref.as64(w)
    tol_r = (adds(x.shape[1]) / 2 + 4) * U
    tol = tol_r + 5 * U
    # the sum itself may cancel: one rounding of F32 operands, relative to the result
    if rstd is not None:
        assert np.all(np.abs(ref.as64(rstd) - want_r) <= tol_r * want_r)
    if total is not None:
        assert np.all(np.abs(ref.as64(total) - s) <= (U + HALF[total.dtype]) * np.abs(s))
    if y is not None:
        assert np.all(np.abs(ref.as64(y) - want) <= (tol + HALF[y.dtype] * (1 + tol)) * np.abs(want) + 1e-40)
    if codes is not None:
        check_codes(codes, scale, want, tol)
    if top is not None and y is not None:
        assert float(top) == float(y.float().abs().max())


def forward(rows, cols, dtype, wdtype="f32", res=True, want=("sum", "y", "codes", "amax", "rstd"), eps=1e-5, over=5, seed=0):
    x, r, w = inputs(rows, cols, dtype, wdtype, seed)
    total = dirty((rows, cols + over), DT[dtype]) if "sum" in want else None
    y = dirty((rows, cols + over), DT[dtype]) if "y" in want else None
    codes = torch.full((rows, -(-cols // 16) * 16 + 16), 0xA5, dtype=torch.uint8, device="cuda") if "codes" in want else None
    scale = torch.full((api.mxfp8_swizzled_scales_size(rows, -(-cols // 128)),), 0xA5, dtype=torch.uint8, device="cuda") if "codes" in want else None
    top = torch.zeros(1, device="cuda") if "amax" in want else None
    rstd = dirty((rows,), torch.float32) if "rstd" in want else None
    cut = lambda t: None if t is None else t[:, :cols]  # noqa: E731
    api.mxfp8_rms_norm_forward(x, r if res else None, w, cut(total), cut(y), codes, scale, top, rstd, rows, cols, eps)
    api.mxfp8_device_status()
    check_forward(x, r if res else None, w, eps, cut(total), cut(y), codes, scale, top, rstd)
    for t in (total, y):
        assert t is None or bool((t[:, cols:] == -3.0).all())
    assert codes is None or bool((codes[:, cols:] == 0xA5).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES + MANY)
def test_forward(rows, cols, dtype):
    forward(rows, cols, dtype, over=0)


@pytest.mark.parametrize("dtype,wdtype", [("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", [(3, 200), (2, 4096), (9, 1001), (1900, 640), (700, 6144), (1900, 999)])
@pytest.mark.parametrize("want", [("y",), ("codes",), ("sum", "codes", "rstd"), ("sum", "y", "amax", "rstd"), ("y", "codes")])
def test_forward_parts(rows, cols, dtype, wdtype, want):
    for res in (True, False):
        for over in (0, 5, 8):
            forward(rows, cols, dtype, wdtype, res, want, over=over)


def test_codes_are_the_operand_of_a_product():
    """What the norm writes and what a checkpoint of its F32 output writes: the same, but for y's last places."""
    rows, cols = 200, 384
    x, r, w = inputs(rows, cols, "f32", "f32")
    y, codes = torch.empty_like(x), torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    n = api.mxfp8_swizzled_scales_size(rows, 3)
    scale, want_s = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    want = torch.empty_like(codes)
    api.mxfp8_rms_norm_forward(x, r, w, None, y, codes, scale, None, None, rows, cols)
    api.mxfp8_checkpoint_save(y, want, want_s, None, None, rows, cols)
    assert torch.equal(codes, want) and torch.equal(scale, want_s)


@pytest.mark.parametrize("rows,cols", [(5, 320), (3, 4096), (2, 1001), (700, 4096), (1900, 1001), (1, 40000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(rows, cols, dtype):
    x, r, w = inputs(rows, cols, dtype, "f32")
    y0, s0, y1 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    api.mxfp8_rms_norm_forward(x, r, w, s0, y0, None, None, None, None, rows, cols)
    a, b = x.clone(), r.clone()
    api.mxfp8_rms_norm_forward(a, b, w, b, y1, None, None, None, None, rows, cols)
    assert torch.equal(b, s0) and torch.equal(y1, y0) and torch.equal(a, x)
    b = r.clone()
    api.mxfp8_rms_norm_forward(a, b, w, a, b, None, None, None, None, rows, cols)
    assert torch.equal(a, s0) and torch.equal(b, y0)


@pytest.mark.parametrize("cols", [64, 129, 4096, 40000])
def test_rows_that_are_zero_or_not_finite(cols):
    rows = 700 if cols == 4096 else 20
    x, r, w = inputs(rows, cols, "f32", "f32")
    x[2], r[2] = 0.0, 0.0
    x[4, cols // 2] = float("nan")
    x[6, 1] = float("inf")
    total, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    codes = torch.empty(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda")
    scale = torch.empty(api.mxfp8_swizzled_scales_size(rows, -(-cols // 128)), dtype=torch.uint8, device="cuda")
    top = torch.zeros(1, device="cuda")
    api.mxfp8_rms_norm_forward(x, r, w, total, y, codes, scale, top, rstd, rows, cols)
    assert bool((y[2] == 0).all()) and bool((codes[2, :cols] & 0x7F == 0).all())
    assert bool(torch.isnan(y[4]).all()) and bool((codes[4, :cols] & 0x7F == 0x7F).all())
    # an infinity: rstd is 0, its own place 0 * inf = NaN, the others 0
    assert float(rstd[6]) == 0.0 and bool(torch.isnan(y[6, 1])) and int((y[6] == 0).sum()) == cols - 1
    assert top.view(torch.int32).item() == 0x7FC00000
    fine = [i for i in range(rows) if i not in (4, 6)]
    check_forward(x[fine], r[fine], w, 1e-5, total[fine], y[fine], None, None, None, rstd[fine])


def test_amax_accumulates():
    x, _, w = inputs(900, 512, "bf16", "f32")
    y = torch.empty_like(x)
    for before in (0.0, 1000.0):
        top = torch.full((1,), before, device="cuda")
        api.mxfp8_rms_norm_forward(x, None, w, None, y, None, None, top, None, 900, 512)
        assert float(top) == max(before, float(y.float().abs().max()))


def check_backward(dy, dsum, x, w, rstd, dx, dw):
    d, s, w64, r = ref.as64(dy), ref.as64(x), ref.as64(w), ref.as64(rstd)[:, None]
    xh, g = s * r, d * w64
    c, mag = (g * xh).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
    ds = 0.0 if dsum is None else ref.as64(dsum)
    want = r * (g - xh * c) + ds
    tol = r * (6 * U * np.abs(g) + np.abs(xh) * ((adds(x.shape[1]) + 10) * U * mag)) + 2 * U * (np.abs(ds) + np.abs(want))
    tol = tol + HALF[dx.dtype] * (np.abs(want) + tol)
    err = np.abs(ref.as64(dx) - want)
    assert np.all(err <= tol + 1e-40), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"
    err = np.abs(ref.as64(dw) - (d * xh).sum(0))
    assert np.all(err <= (x.shape[0] + 40) * U * np.abs(d * xh).sum(0) + 1e-40)


def backward(rows, cols, dtype, wdtype="f32", res=True, over=0, place=None):
    x, ds, w = inputs(rows, cols, dtype, wdtype)
    g = torch.Generator(device="cuda").manual_seed(cols)
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dtype])
    rstd = (x.float().square().mean(1) + 1e-5).rsqrt()
    dw = dirty((cols,), torch.float32)
    ws = torch.empty(max(1, api.mxfp8_rms_norm_workspace_size(rows, cols)), dtype=torch.uint8, device="cuda")
    dx = dirty((rows, cols + over), DT[dtype])
    args = {"dy": dy.clone(), "ds": ds.clone() if res else None, "x": x.clone()}
    out = dx[:, :cols] if place is None else args[place]
    api.mxfp8_rms_norm_backward(args["dy"], args["ds"], args["x"], w, rstd, out, dw, ws, rows, cols)
    api.mxfp8_device_status()
    check_backward(dy, ds if res else None, x, w, rstd, out, dw)
    assert bool((dx[:, cols:] == -3.0).all())
    return out.clone(), dw


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES + MANY)
def test_backward(rows, cols, dtype):
    backward(rows, cols, dtype)


@pytest.mark.parametrize("dtype,wdtype", [("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", [(3, 200), (2, 4096), (9, 1001), (1900, 640), (700, 6144), (1900, 999)])
def test_backward_parts(rows, cols, dtype, wdtype):
    for res in (True, False):
        for over in (0, 5):
            backward(rows, cols, dtype, wdtype, res, over)
    want = backward(rows, cols, dtype, wdtype)
    for place in ("dy", "ds", "x"):
        got = backward(rows, cols, dtype, wdtype, place=place)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows,cols", [(4, 96), (3, 131)])
def test_gradients_by_differences(rows, cols):
    """Of a loss sum(a y) + sum(b s), by central differences of the forward pass in F32 at a step of 2^-6: the second-order
    term is h^2 / 6 of the third derivative (of order one here: 4e-5 of the gradient's size), the rounding of two
    losses 2 x 2^-24 sqrt(cols) x the size of their terms over 2 h, 1e-4."""
    x, _, w = inputs(rows, cols, "f32", "f32")
    g = torch.Generator(device="cuda").manual_seed(9)
    a, b = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(2))

    def loss(x, w):  # per row in float64, of the kernel's own outputs
        s, y = torch.empty_like(x), torch.empty_like(x)
        api.mxfp8_rms_norm_forward(x, None, w, s, y, None, None, None, None, rows, cols)
        return (a.double() * y.double() + b.double() * s.double()).sum(1)
    rstd, y = torch.empty(rows, device="cuda"), torch.empty_like(x)
    api.mxfp8_rms_norm_forward(x, None, w, None, y, None, None, None, rstd, rows, cols)
    dx, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
    ws = torch.empty(api.mxfp8_rms_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    api.mxfp8_rms_norm_backward(a, b, x, w, rstd, dx, dw, ws, rows, cols)
    h = 2.0 ** -6
    for c in range(0, cols, 7):
        up, down = x.clone(), x.clone()
        up[:, c] += h
        down[:, c] -= h
        got = (loss(up, w) - loss(down, w)) / (2 * h)
        assert torch.allclose(got, dx[:, c].double(), rtol=0, atol=1e-3)
        up, down = w.clone(), w.clone()
        up[c] += h
        down[c] -= h
        got = (loss(x, up) - loss(x, down)).sum() / (2 * h)
        assert abs(float(got) - float(dw[c])) < 1e-3


def test_backward_without_rows():
    dw = dirty((64,), torch.float32)
    api.mxfp8_rms_norm_backward(None, None, None, None, None, None, dw, None, 0, 64)
    assert bool((dw == 0).all())
