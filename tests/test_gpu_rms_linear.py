"""RMS norm, its codes and the products together: a layer's step on MXFP8 and on NVFP4 weights, checked stage by stage in
float64 from the values each stage was given, against the unquantised layer, replayed from a graph, and on other streams."""
import numpy as np
import pytest
import torch

import fp4_ref as fp4
import linear_ref as ref
from mxfp8_master_weight_gb300 import api, linear
from test_gpu_gemm import check as check_product
from test_gpu_nvfp4_operands import check as check_product4
from test_gpu_rms_norm import check_backward, check_forward

pytestmark = pytest.mark.gpu
KINDS = ["mxfp8", "nvfp4"]


def make(weights, tokens, ins, outs, dtype=torch.bfloat16, training=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens)
    bounds = [0, outs * ins // 3 + 17, outs * ins] if weights == "mxfp8" else None
    layer = linear.RMSNormLinear(tokens, ins, outs, dtype=dtype, weights=weights, bounds=bounds, training=training)
    master = torch.randn(outs * ins, generator=g, device="cuda") * 0.02
    layer.norm_weight.copy_(1 + 0.1 * torch.randn(ins, generator=g, device="cuda"))
    layer.refresh([master[a:b] for a, b in zip(bounds[:-1], bounds[1:])] if bounds else [master])
    x, r = (torch.randn(tokens, ins, generator=g, device="cuda").to(dtype) for _ in range(2))
    dy, ds = ((torch.randn(tokens, n, generator=g, device="cuda") * 1e-2).to(dtype) for n in (outs, ins))
    return layer, master.view(outs, ins), x, r, dy, ds


@pytest.mark.parametrize("weights", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,ins,outs", [(200, 256, 384), (333, 514, 259), (1, 96, 160), (77, 130, 66)])
def test_step(weights, tokens, ins, outs, dtype):
    layer, master, x, r, dy, ds = make(weights, tokens, ins, outs, dtype)
    w, w16 = ref.as64(master), ref.as64(master.bfloat16())
    for residual, grad in ((r, ds), (None, None)):
        y, total = layer.forward(x, residual)
        check_forward(x, residual, layer.norm_weight, layer.eps, total, layer.h, None, None, None, layer.rstd)
        h = ref.as64(layer.h)
        before = ref.as64(layer.grad_weight)
        dx = layer.backward(dy, grad)
        d = ref.as64(dy)
        if weights == "mxfp8":
            out = torch.empty(tokens, ins, device="cuda")
            layer.weights.h8.restore(out)  # from the unrounded values: as the norm wrote it
            check_product(y, ref.as64(out), ref.quantise(w16, 32, w)[0], ins)
            check_product(layer.dh, ref.quantise(d)[0], ref.quantise(w16.T, 32, w.T)[0], outs)
            check_product(layer.grad_weight, ref.quantise(d.T)[0], ref.quantise(h.T)[0], tokens, before)
        else:
            top = float(layer.h.float().abs().max())
            assert float(layer.weights.h4.amax) == top and float(layer.weights.amax) == float(master.abs().max())
            dt, wt = float(dy.float().abs().max()), float(master.abs().max())
            values = lambda v, t: (lambda q, s: q * fp4.spread(s, q.shape[1]).astype(np.float64))(*fp4.quantise(v, t))  # noqa: E731
            # a weight's block maxima are the master's, its codes those of its BF16 rounding
            w4, w4t = (values_of_weight(m, m16, wt) for m, m16 in ((w, w16), (w.T, w16.T)))
            check_product4(y, values(h, top), w4, ins, top, wt)
            check_product4(layer.dh, values(d, dt), w4t, outs, dt, wt)
            check_product4(layer.grad_weight, values(d.T, dt), values(h.T, top), tokens, dt, top, before)
        check_backward(layer.dh, grad, total, layer.norm_weight, layer.rstd, dx, layer.grad_norm_weight)
    layer.check()


def values_of_weight(master, rounded, top):
    _, s = fp4.quantise(master, top)
    S = fp4.tensor_scale(top)
    mul = np.where(s == 0, np.float32(0), S / np.where(s == 0, np.float32(1), s)).astype(np.float32)
    q = fp4.e2m1(rounded.astype(np.float32) * fp4.spread(mul, master.shape[1]))
    return q * fp4.spread(s, master.shape[1]).astype(np.float64)


@pytest.mark.parametrize("weights", KINDS)
def test_close_to_the_unquantised_layer(weights):
    """E4M3's relative rounding errors are uniform within 2^-4: 2^-4 / sqrt(3) / 2 or so of each factor; E2M1 with a scale per 16
    values rounds by up to a quarter of a value, about 0.1 of its size on the average.  Two factors, three products: under
    a tenth, and under a third."""
    t, i, o = 512, 1024, 768
    layer, master, x, r, dy, ds = make(weights, t, i, o)
    y, total = layer.forward(x, r)
    dx = layer.backward(dy, ds)
    s, w, nw, d = ref.as64(x) + ref.as64(r), ref.as64(master), ref.as64(layer.norm_weight), ref.as64(dy)
    rstd = 1 / np.sqrt((s * s).mean(1, keepdims=True) + layer.eps)
    h, g = s * rstd * nw, (d @ w) * nw
    want = {"y": h @ w.T, "dw": d.T @ h, "dx": rstd * (g - s * rstd * (g * s * rstd).mean(1, keepdims=True)) + ref.as64(ds)}
    for name, got in (("y", y), ("dw", layer.grad_weight), ("dx", dx)):
        err = np.linalg.norm(ref.as64(got) - want[name]) / np.linalg.norm(want[name])
        assert err < (0.1 if weights == "mxfp8" else 0.33), (name, err)


@pytest.mark.parametrize("weights", KINDS)
def test_graph_and_streams(weights):
    """Two layers of a residual stream captured into one graph and replayed; the same eagerly on another stream."""
    t, i = 130, 256
    first, _, x, r, dy, ds = make(weights, t, i, i)
    second = make(weights, t, i, i, seed=5)[0]

    def step():
        a, s = first.forward(x, r)
        b, total = second.forward(a, s)
        dsum = second.backward(dy, ds)
        dx = first.backward(dsum, dsum)  # the sum's gradient is that of both its terms
        return b, total, dx, first.grad_weight, second.grad_weight, first.grad_norm_weight

    want = [v.clone() for v in step()]
    first.grad_weight.zero_(), second.grad_weight.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for v in outs:
        v.zero_()
    for _ in range(2):
        first.grad_weight.zero_(), second.grad_weight.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first.grad_weight.zero_(), second.grad_weight.zero_()
        outs = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    api.mxfp8_device_status()


@pytest.mark.parametrize("weights", KINDS)
@pytest.mark.parametrize("tokens", [1, 64])
def test_serving(weights, tokens):
    """A layer that only serves gives what the training one gives, token by token too."""
    i, o = 512, 384
    train, _, x, r, _, _ = make(weights, tokens, i, o)
    serve = make(weights, tokens, i, o, training=False)[0]
    want = [v.clone() for v in train.forward(x, r)]
    got = serve.forward(x, r)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if weights == "mxfp8":  # a row's codes do not depend on the other rows
        one = make(weights, 1, i, o, training=False)[0]
        one.norm_weight.copy_(serve.norm_weight)
        one.weights.cast, one.weights.scale_r = serve.weights.cast, serve.weights.scale_r
        for k in (0, tokens - 1):
            y, s = one.forward(x[k:k + 1], r[k:k + 1])
            assert torch.equal(s[0], want[1][k])
            assert torch.allclose(y[0].float(), want[0][k].float(), rtol=2.0 ** -7, atol=1e-4)  # another order of sums, rounded to BF16
    assert serve.h is None or weights == "nvfp4"


def test_concurrent_streams():
    """Calls on two streams at once, each with buffers of its own."""
    layers = [make(k, 256, 512, 512, seed=s) for s, k in enumerate(KINDS)]
    want = [[v.clone() for v in (*l.forward(x, r), l.backward(dy, ds))] for l, _, x, r, dy, ds in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for (l, _, x, r, dy, ds), s in zip(layers, streams):
            with torch.cuda.stream(s):
                got.append((*l.forward(x, r), l.backward(dy, ds)))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("weights", KINDS)
def test_no_tokens(weights):
    """A step of no tokens leaves the weight's gradient as it is and sets the norm's to zero."""
    layer, _, x, r, dy, ds = make(weights, 0, 64, 32)
    layer.grad_weight.fill_(3.0)
    layer.grad_norm_weight.fill_(3.0)
    y, s = layer.forward(x, r)
    assert y.shape == (0, 32) and s.shape == (0, 64) and layer.backward(dy, ds).shape == (0, 64)
    assert bool((layer.grad_weight == 3.0).all()) and bool((layer.grad_norm_weight == 0).all())
    layer.check()
