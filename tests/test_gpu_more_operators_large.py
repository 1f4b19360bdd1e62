"""RMS norm and NVFP4 operands on rows so far apart that offsets pass 2^31 elements and 2^32 bytes."""
import numpy as np
import pytest
import torch

import fp4_ref as fp4
import linear_ref as ref
from mxfp8_master_weight_gb300 import api
from test_gpu_nvfp4_operands import check, operand, scales
from test_gpu_operators_large import far
from test_gpu_rms_norm import check_backward, check_codes, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,stride", [(9, 200, 1 << 28), (700, 512, 1 << 22), (1900, 301, (1 << 21) + 1)])
def test_rms_norm(rows, cols, stride):
    x, r, s, y, dy = (far(rows, cols, stride, torch.bfloat16) for _ in range(5))
    g = torch.Generator(device="cuda").manual_seed(rows)
    for t in (x, r, dy):
        t.copy_(torch.randn(rows, cols, generator=g, device="cuda"))
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    q = far(rows, cols, 2 * stride, torch.uint8)
    scale = torch.empty(api.mxfp8_swizzled_scales_size(rows, -(-cols // 128)), dtype=torch.uint8, device="cuda")
    rstd, dw = torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(api.mxfp8_rms_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    api.mxfp8_rms_norm_forward(x, r, w, s, y, q, scale, None, rstd, rows, cols)
    check_forward(x, r, w, 1e-5, s, y, None, None, None, rstd)
    total = ref.as64(x) + ref.as64(r)
    want = total / np.sqrt((total * total).mean(1, keepdims=True) + 1e-5) * ref.as64(w)
    check_codes(q, scale, want, 100 * 2.0 ** -24)
    rows_rstd = (s.float().square().mean(1) + 1e-5).rsqrt()
    api.mxfp8_rms_norm_backward(dy, r, s, w, rows_rstd, x, dw, ws, rows, cols)
    check_backward(dy, r, s, w, rows_rstd, x, dw)
    api.mxfp8_device_status()


@pytest.mark.parametrize("rows,cols,stride", [(9, 200, 1 << 28), (200, 129, (1 << 24) + 1)])
def test_quantise_and_restore(rows, cols, stride):
    x = far(rows, cols, stride, torch.bfloat16)
    x.copy_(torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))
    top = torch.empty(1, device="cuda")
    api.nvfp4_tensor_amax(x, top, rows, cols)
    v = x.float().cpu().numpy()
    assert float(top) == np.abs(v).max()
    q_r, q_c = far(rows, (cols + 1) // 2, 1 << 29, torch.uint8) if rows < 20 else far(rows, (cols + 1) // 2, 1 << 25, torch.uint8), \
        far(cols, (rows + 1) // 2, 1 << 25, torch.uint8)
    s_r, s_c = scales(rows, cols), scales(cols, rows)
    api.nvfp4_quantize(x, top, q_r, s_r, q_c, s_c, rows, cols)
    for q, s, m in ((q_r, s_r, v), (q_c, s_c, v.T)):
        want, sv = fp4.quantise(m, float(top))
        assert np.array_equal(fp4.unpack(q, *m.shape), want)
        assert np.array_equal(s.cpu().numpy(), ref.tiles(fp4.scale_bytes(sv)))
    out = far(rows, cols, stride, torch.float32)
    api.nvfp4_restore(q_r, s_r, top, out, rows, cols)
    assert np.array_equal(out.cpu().numpy(), fp4.kept(v, float(top)))


@pytest.mark.parametrize("m,n,k,stride", [(9, 40, 300, 1 << 28), (130, 140, 200, 1 << 25), (300, 264, 256, 1 << 23)])
@pytest.mark.parametrize("dtype,addend", [(torch.float32, True), (torch.float32, False), (torch.bfloat16, False)])
def test_product(m, n, k, stride, dtype, addend):
    rng = np.random.default_rng(m)
    a, qa, sa, ta = operand(rng, m, k)
    b, qb, sb, tb = operand(rng, n, k)
    wide = far(m, (k + 1) // 2, stride, torch.uint8)
    wide.copy_(qa[:, :(k + 1) // 2])
    out, c = far(m, n, stride, dtype), far(m, n, stride, torch.float32) if addend else None
    if addend:
        c.normal_()
    ga, gb = torch.tensor([ta], device="cuda"), torch.tensor([tb], device="cuda")
    api.nvfp4_gemm(wide, sa, ga, qb, sb, gb, c, out, m, n, k)
    api.mxfp8_device_status()
    check(out.contiguous(), a, b, k, ta, tb, ref.as64(c) if addend else None)
