"""The training operators together: a layer norm and a linear layer on the cast's MXFP8 weights, a
step checked stage by stage in float64 from the values each stage was given, and against the
unquantised layer."""
import numpy as np
import pytest
import torch

import linear_ref as ref
from mxfp8_master_weight_gb300 import api, linear
from test_gpu_gemm import check as check_product
from test_gpu_layer_norm import check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,ins,outs", [(200, 256, 384), (333, 515, 259), (1, 96, 160)])
def test_step(tokens, ins, outs, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    cut = outs * ins // 3 + 17
    layer = linear.NormLinear(tokens, ins, outs, dtype=dtype, bounds=[0, cut, outs * ins])
    master = torch.randn(outs * ins, generator=g, device="cuda") * 0.02
    layer.norm_weight.copy_(1 + 0.1 * torch.randn(ins, generator=g, device="cuda"))
    layer.norm_bias.copy_(0.1 * torch.randn(ins, generator=g, device="cuda"))
    layer.refresh([master[:cut], master[cut:]])
    w = ref.as64(master.view(outs, ins))
    w16 = ref.as64(master.view(outs, ins).bfloat16())
    w_r, w_c = ref.quantise(w16, 32, w)[0], ref.quantise(w16.T, 32, w.T)[0].T
    x = torch.randn(tokens, ins, generator=g, device="cuda").to(dtype)
    dy = (torch.randn(tokens, outs, generator=g, device="cuda") * 1e-2).to(dtype)
    grads = []
    for step in range(2):
        y = layer.forward(x)
        h = ref.as64(layer.h)
        check_forward(ref.as64(x), ref.as64(layer.norm_weight), ref.as64(layer.norm_bias), layer.h, layer.mean, layer.rstd)
        h_r, h_c = ref.quantise(h)[0], ref.quantise(h.T)[0]
        check_product(y, h_r, w_r, ins)
        before = ref.as64(layer.grad_weight)
        dx = layer.backward(dy)
        dy_r, dy_c = ref.quantise(ref.as64(dy))[0], ref.quantise(ref.as64(dy).T)[0]
        check_product(layer.dh, dy_r, w_c.T, outs)
        check_product(layer.grad_weight, dy_c, h_c, tokens, before)
        check_backward(ref.as64(layer.dh), ref.quantise(ref.as64(x))[0], ref.as64(layer.norm_weight), ref.as64(layer.mean),
                       ref.as64(layer.rstd), dx, layer.grad_norm_weight, layer.grad_norm_bias)
        grads.append(layer.grad_weight.clone())
    assert torch.allclose(grads[1], 2 * grads[0], rtol=1e-5, atol=0.0)  # two equal steps accumulate
    api.mxfp8_device_status()


def test_close_to_the_unquantised_layer():
    """With E4M3's 2^-4 relative rounding of both factors, a sum of `ins` products of independent signs
    is off by about sqrt(2) 2^-5.4 of its own size (uniform rounding errors: 2^-4 / sqrt(12) each
    way); three such steps in a row stay under a tenth."""
    t, i, o = 512, 1024, 768
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = linear.NormLinear(t, i, o)
    master = torch.randn(o * i, generator=g, device="cuda") * 0.02
    layer.refresh([master])
    x = torch.randn(t, i, generator=g, device="cuda").bfloat16()
    dy = (torch.randn(t, o, generator=g, device="cuda") * 1e-2).bfloat16()
    y, w = layer.forward(x), ref.as64(master.view(o, i))
    dx = layer.backward(dy)
    h, mean, rstd = ref.norm_forward(ref.as64(x), np.ones(i), np.zeros(i), layer.eps)
    d = ref.as64(dy)
    want = {"y": h @ w.T, "dw": d.T @ h, "dx": ref.norm_backward(d @ w, ref.as64(x), np.ones(i), mean, rstd)[0]}
    for name, got in (("y", y), ("dw", layer.grad_weight), ("dx", dx)):
        err = np.linalg.norm(ref.as64(got) - want[name]) / np.linalg.norm(want[name])
        assert err < 0.1, (name, err)


def test_checkpoint_restore_and_capture():
    """A checkpoint's buffers through the class, and a whole step replayed from a CUDA graph."""
    t, i, o = 160, 384, 256
    layer = linear.NormLinear(t, i, o)
    master = torch.randn(o * i, device="cuda") * 0.02
    x, dy = torch.randn(t, i, device="cuda").bfloat16(), torch.randn(t, o, device="cuda").bfloat16()
    ck = linear.Checkpoint(t, i, "cuda")
    ck.save(x)
    out = torch.empty(t, i, device="cuda")
    for colwise in (False, True):
        ck.restore(out, colwise)
        x64 = ref.as64(x)
        assert np.array_equal(ref.as64(out), ref.quantise(x64.T)[0].T if colwise else ref.quantise(x64)[0])

    def step():
        layer.refresh([master])
        layer.forward(x)
        layer.backward(dy)
    step()
    want = [v.clone() for v in (layer.y, layer.dx, layer.grad_weight)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    layer.grad_weight.zero_()
    layer.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((layer.y, layer.dx, layer.grad_weight), want):
        assert torch.equal(a, b)
