"""A layer's inputs have the layer's shape: everything else is refused before any work, where a buffer argument
of the entry points below may be larger than needed."""
import pytest
import torch

from mxfp8_master_weight_gb300 import api, linear


def refused(status, fn, *a):
    with pytest.raises(api.MXFP8Error) as e:
        fn(*a)
    return e.value.status == status


@pytest.mark.parametrize("shape", [(7, 16), (9, 16), (8, 15), (8, 32), (16, 8), (8, 4, 4), (1, 8, 16), (127,), (129,), (0, 16), ()])
def test_wrong_shapes(shape):
    assert refused(2, linear._check_input, torch.empty(shape), "x", 8, 16)


def test_right_shapes():
    for x in (torch.empty(8, 16), torch.empty(128), torch.empty(8, 20)[:, 2:18], torch.empty(12, 16)[3:11]):
        linear._check_input(x, "x", 8, 16)
    linear._check_input(torch.empty(0, 16), "x", 0, 16)


@pytest.mark.gpu
def test_layer_refuses_other_shapes():
    t, i, o = 24, 64, 48
    layer = linear.NormLinear(t, i, o)
    layer.refresh([torch.randn(o * i, device="cuda") * 0.02])
    x, dy = torch.randn(t, i, device="cuda").bfloat16(), torch.randn(t, o, device="cuda").bfloat16()
    y, dx = layer.forward(x).clone(), layer.backward(dy).clone()
    keep = [v.clone() for v in (layer.x8.codes_r, layer.h8.codes_r, layer.dy8.codes_r, layer.grad_weight)]
    wide = lambda a: torch.cat([a, a], 1)  # noqa: E731
    for bad in (wide(x), torch.cat([x, x]), x[:t - 1], x[:, :i - 1], x.view(1, t, i)):
        assert refused(2, layer.forward, bad) and refused(2, layer.x8.save, bad)
    for bad in (wide(dy), torch.cat([dy, dy]), dy[:t - 1], dy[:, :o - 1]):
        assert refused(2, layer.backward, bad)
    assert refused(3, layer.forward, x.float())
    for a, b in zip((layer.x8.codes_r, layer.h8.codes_r, layer.dy8.codes_r, layer.grad_weight), keep):
        assert torch.equal(a, b)
    # strided and one-dimensional inputs, and a gradient of the other type, are fine
    layer.grad_weight.zero_()
    assert torch.equal(layer.forward(wide(x)[:, i:]), y) and torch.equal(layer.backward(wide(dy)[:, :o]), dx)
    assert torch.equal(layer.forward(x.flatten()), y) and torch.equal(layer.backward(dy.float()), dx)
