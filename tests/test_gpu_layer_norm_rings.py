"""Layer norm over enough rows for the persistent blocks, on rows that lose digits where the arithmetic
is careless: constant and nearly constant ones, rows far from zero, NaN and infinity.

The backward pass is given x, mean and rstd as they are, so xh = (x - mean) rstd carries two roundings:
3 u |xh| with u = 2^-24, whatever the mean's size.  The row sums and what follows are bounded as in the other
tests (a thread adds at most 32 values in order and about 11 more in the reductions)."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api
from test_gpu_layer_norm import DT, EPS, U, adds, backward, check_forward, forward, within

pytestmark = pytest.mark.gpu

ROWS = 1900  # more than 12 per SM: rings of every width
COLS = [72, 512, 1000, 3001, 6143, 6144, 8192]


def rows_of_all_kinds(cols, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + cols)
    x = torch.randn(ROWS, cols, generator=g, device="cuda")
    kind = torch.arange(ROWS, device="cuda") % 5
    level = 2.0 ** (torch.arange(ROWS, device="cuda") % 11)[:, None] * 1.25
    few = (torch.rand(ROWS, cols, generator=g, device="cuda") < 0.01).float()
    x = torch.where(kind[:, None] == 1, level.expand(-1, cols), x)                    # constant
    x = torch.where(kind[:, None] == 2, 256.0 + 2.0 * few, x)                         # nearly constant
    x = torch.where(kind[:, None] == 3, 100.0 + x, x)                                 # far from zero
    x = torch.where(kind[:, None] == 4, -1000.0 + 0.0 * x, x)                         # constant, not a power of two
    return x.to(DT[dtype])


def statistics(x64):
    """mean and rstd of the rows, in F32: inputs of the backward pass."""
    mean = x64.mean(1)
    rstd = 1.0 / np.sqrt(((x64 - mean[:, None]) ** 2).mean(1) + EPS)
    return tuple(torch.from_numpy(v).float().cuda() for v in (mean, rstd))


def check_given(dy64, x64, w64, mean64, rstd64, dx, dw, db):
    wx, ww, wb = ref.norm_backward(dy64, x64, w64, mean64, rstd64)
    rows, cols = dy64.shape
    t = adds(cols) * U
    r, xh, g = rstd64[:, None], np.abs((x64 - mean64[:, None]) * rstd64[:, None]), np.abs(dy64 * w64)
    mg, mgx = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    within(dx, wx, r * (t + 12 * U) * (g + mg + xh * mgx) + 4 * U * np.abs(wx), dx.dtype)
    tr = (rows / 8 + 64) * U  # a block adds its rows in order, then the partial rows
    within(dw, ww, (tr + 3 * U) * (np.abs(dy64) * xh).sum(0))
    within(db, wb, tr * np.abs(dy64).sum(0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_backward_of_rows_far_from_zero(cols, dtype):
    x = rows_of_all_kinds(cols, dtype)
    dy = torch.randn(ROWS, cols, generator=torch.Generator(device="cuda").manual_seed(cols), device="cuda").to(x.dtype)
    w = 1 + 0.2 * torch.randn(cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    mean, rstd = statistics(ref.as64(x))
    check_given(*map(ref.as64, (dy, x, w, mean, rstd)), *backward(dy, x, None, w, mean, rstd))
    q = torch.empty(ROWS, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(api.mxfp8_swizzled_scales_size(ROWS, -(-cols // 128)), dtype=torch.uint8, device="cuda")
    api.mxfp8_checkpoint_save(x, q, s, None, None, ROWS, cols)
    kept = ref.quantise(ref.as64(x))[0]
    mean, rstd = statistics(kept)
    check_given(ref.as64(dy), kept, ref.as64(w), ref.as64(mean), ref.as64(rstd), *backward(dy, q, s, w, mean, rstd))
    api.mxfp8_device_status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1000, 1024, 3001, 6143, 7168])
def test_forward_of_constant_rows(cols, dtype):
    """Small whole numbers add exactly in any order, and their mean is exact: the deviations are zero, and y
    is the bias to the last bit."""
    value = (torch.arange(ROWS, device="cuda") % 256 + 1).float()
    x = value[:, None].expand(-1, cols).to(DT[dtype]).contiguous()
    w = 1 + 0.2 * torch.randn(cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    b = torch.randn(cols, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(x.dtype).float()
    y, mean, rstd = forward(x, w, b)
    assert torch.equal(mean, value)
    assert torch.equal(y.float(), b.expand(ROWS, -1))
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=1e-6, atol=0.0)
    api.mxfp8_device_status()


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("cols", COLS)
def test_forward_without_bias_and_of_both_weight_types(cols, dtype, wdtype):
    x = torch.randn(ROWS, cols, generator=torch.Generator(device="cuda").manual_seed(cols), device="cuda").to(DT[dtype])
    w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")).to(DT[wdtype])
    b = torch.randn(cols, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(DT[wdtype])
    x64, w64 = ref.as64(x), ref.as64(w)
    check_forward(x64, w64, None, *forward(x, w, None))
    check_forward(x64, w64, ref.as64(b), *forward(x, w, b))
    api.mxfp8_device_status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_nan_and_infinity_stay_where_they_belong(cols, dtype):
    """Forward: in their rows.  Backward: in their rows of dx and their columns of the sums over rows; from a
    checkpoint in the whole block that the NaN scale makes."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(ROWS, cols, generator=g, device="cuda").to(DT[dtype])
    dy = torch.randn(ROWS, cols, generator=g, device="cuda").to(x.dtype)
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    mean, rstd = statistics(ref.as64(x))
    nan, inf = float("nan"), float("inf")
    bad_x = {(3, 0): nan, (611, cols - 1): inf, (1899, cols // 2): -inf}
    bad_dy = {(4, 5): nan, (1500, cols - 2): inf}
    for (r, c), v in bad_x.items():
        x[r, c] = v
    y, m, s = forward(x, w, None)
    rows = torch.zeros(ROWS, dtype=torch.bool, device="cuda")
    rows[[r for r, _ in bad_x]] = True
    assert torch.equal(torch.isnan(y).all(1), rows) and torch.equal((~torch.isfinite(y)).any(1), rows)
    assert m[3].isnan() and m[611] == inf and m[1899] == -inf and torch.equal(~torch.isfinite(s), rows)
    for (r, c), v in bad_dy.items():
        dy[r, c] = v
    rows[[r for r, _ in bad_dy]] = True
    q = torch.empty(ROWS, cols, dtype=torch.uint8, device="cuda")
    sc = torch.empty(api.mxfp8_swizzled_scales_size(ROWS, -(-cols // 128)), dtype=torch.uint8, device="cuda")
    api.mxfp8_checkpoint_save(x, q, sc, None, None, ROWS, cols)
    for saved, scale in ((x, None), (q, sc)):
        dx, dw, db = backward(dy, saved, scale, w, mean, rstd)
        assert torch.equal((~torch.isfinite(dx)).any(1), rows)
        in_dw = torch.zeros(cols, dtype=torch.bool, device="cuda")
        in_db = in_dw.clone()
        for _, c in bad_dy:
            in_dw[c] = in_db[c] = True
        for _, c in bad_x:
            in_dw[c if scale is None else slice(c // 128 * 128, c // 128 * 128 + 128)] = True
        assert torch.equal(~torch.isfinite(dw), in_dw) and torch.equal(~torch.isfinite(db), in_db)
    api.mxfp8_device_status()
