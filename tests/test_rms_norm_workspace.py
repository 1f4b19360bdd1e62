"""The workspace of RMS norm's gradients: one row of partial sums per block that runs at once, and nothing written behind it."""
import pytest
import torch

from mxfp8_master_weight_gb300 import _capi, api
from mxfp8_master_weight_gb300 import build as libbuild


@pytest.mark.parametrize("cols,per_sm", [(1, 2), (71, 2), (256, 2), (257, 12), (512, 12), (513, 6), (1024, 6), (1025, 4), (2048, 4),
                                         (2049, 3), (4096, 3), (4097, 2), (6144, 2), (8192, 2), (8193, 2), (40000, 2)])
def test_size(cols, per_sm):
    libbuild.build()
    size = _capi.load().mxfp8_rms_norm_workspace_size
    for rows in (0, 1, 2, 303, 304, 305, 1823, 1824, 1825, 3041, 1 << 30):
        assert size(rows, cols) == min(rows, 152 * per_sm) * cols * 4


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [71, 256, 257, 512, 1000, 1024, 2047, 2048, 4096, 4097, 6144, 8192, 8200, 16400])
def test_nothing_behind_it(cols, dtype):
    """Few rows, as many as the rings start with and more than blocks; the gradient does not see what the workspace held."""
    for rows in (1, 5, 700, 2000):
        g = torch.Generator(device="cuda").manual_seed(rows + cols)
        dy, x = (torch.randn(rows, cols, generator=g, device="cuda").to(dtype) for _ in range(2))
        w, rstd = torch.ones(cols, device="cuda"), torch.ones(rows, device="cuda")
        size = api.mxfp8_rms_norm_workspace_size(rows, cols)
        got = []
        for fill in (0x00, 0xFF):
            room = torch.full((size + 4096,), fill, dtype=torch.uint8, device="cuda")
            dx, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
            api.mxfp8_rms_norm_backward(dy, None, x, w, rstd, dx, dw, room[:size], rows, cols)
            assert bool((room[size:] == fill).all())
            got.append(dw)
        api.mxfp8_device_status()
        assert torch.equal(got[0], got[1])
        want = (dy.double() * x.double()).sum(0)
        # at most `rows` roundings one after another and those of the products
        tol = (rows + 40) * 2.0 ** -24 * (dy.double() * x.double()).abs().sum(0)
        assert bool(((got[0].double() - want).abs() <= tol).all())
