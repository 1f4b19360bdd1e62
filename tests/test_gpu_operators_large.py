"""Products and layer norm on rows so far apart that offsets pass 2^31 elements and 2^32 bytes."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api
from test_gpu_gemm import check, operand
from test_gpu_layer_norm import check_backward, check_forward

pytestmark = pytest.mark.gpu


def far(rows, cols, stride, dtype, start=0):
    """rows x cols of a buffer with that row stride, from element `start` on."""
    return torch.empty(rows * stride + start, dtype=dtype, device="cuda")[start:].as_strided((rows, cols), (stride, 1))


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("m,n,k,stride", [(9, 40, 300, 1 << 28), (130, 140, 200, 1 << 25), (300, 9, 256, 1 << 24)])
def test_product(m, n, k, stride, odd):
    rng = np.random.default_rng(m)
    a, qa, sa = operand(rng, m, k, False, 128)
    b, qb, sb = operand(rng, n, k, False, 128)
    wide = far(m, k, stride + odd, torch.uint8, odd)
    wide.copy_(qa[:, :k])
    out, c = far(m, n, stride, torch.float32), far(m, n, stride, torch.float32)
    c.normal_()
    api.mxfp8_gemm(wide, sa, qb, sb, c, out, m, n, k)
    api.mxfp8_device_status()
    check(out.contiguous(), a, b, k, ref.as64(c))


@pytest.mark.parametrize("rows,cols,stride", [(9, 200, 1 << 28), (700, 256, 1 << 22), (1900, 201, (1 << 21) + 1)])
def test_layer_norm(rows, cols, stride):
    x, y, dy, dx = (far(rows, cols, stride, torch.bfloat16) for _ in range(4))
    g = torch.Generator(device="cuda").manual_seed(rows)
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") + 1)
    dy.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    b = torch.randn(cols, generator=g, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(api.mxfp8_layer_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    api.mxfp8_layer_norm_forward(x, w, b, y, mean, rstd, rows, cols)
    x64, w64 = ref.as64(x), ref.as64(w)
    check_forward(x64, w64, ref.as64(b), y, mean, rstd)
    q = far(rows, cols, 2 * stride, torch.uint8)
    s = torch.empty(api.mxfp8_swizzled_scales_size(rows, -(-cols // 128)), dtype=torch.uint8, device="cuda")
    api.mxfp8_checkpoint_save(x, q, s, None, None, rows, cols)
    for saved, scale, values in ((x, None, x64), (q, s, ref.quantise(x64)[0])):
        api.mxfp8_layer_norm_backward(dy, saved, scale, w, mean, rstd, dx, dw, db, ws, rows, cols)
        check_backward(ref.as64(dy), values, w64, ref.as64(mean), ref.as64(rstd), dx, dw, db)
    api.mxfp8_device_status()
