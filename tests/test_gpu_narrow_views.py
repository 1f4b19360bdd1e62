"""A slice of a wider buffer that is narrower than the matrix asked for: its row stride would do, its columns would not.  The
refusal comes before any CUDA work, so it is tested without a GPU too, on tensors that only say that they are on one."""
import pytest
import torch

from mxfp8_master_weight_gb300 import api

R, C, K = 8, 32, 64  # rows and columns; columns of a product's operands
F, B = torch.float32, torch.uint8


class OnGpu:
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


# entry point, arguments (name -> dtype and shape, or a value), which of them are matrices
CASES = {
    "mxfp8_rms_norm_forward": (dict(input=(F, R, C), residual=(F, R, C), weight=(F, C), sum=(F, R, C), output=(F, R, C), codes=(B, R, C),
                                    scale=(B, 512), amax=(F, 1), rstd=(F, R), rows=R, cols=C),
                               ("input", "residual", "sum", "output", "codes")),
    "mxfp8_rms_norm_backward": (dict(grad_output=(F, R, C), grad_sum=(F, R, C), input=(F, R, C), weight=(F, C), rstd=(F, R),
                                     grad_input=(F, R, C), grad_weight=(F, C), workspace=(B, 4 * R * C), rows=R, cols=C),
                                ("grad_output", "grad_sum", "input", "grad_input")),
    "nvfp4_tensor_amax": (dict(input=(F, R, C), amax_tensor=(F, 1), rows=R, cols=C), ("input",)),
    "nvfp4_quantize": (dict(input=(F, R, C), amax_tensor=(F, 1), codes_rowwise=(B, R, C // 2), scale_rowwise=(B, 512),
                            codes_colwise=(B, C, R // 2), scale_colwise=(B, 512), rows=R, cols=C),
                       ("input", "codes_rowwise", "codes_colwise")),
    "nvfp4_restore": (dict(codes=(B, R, C // 2), scale=(B, 512), amax_tensor=(F, 1), output=(F, R, C), rows=R, cols=C),
                      ("codes", "output")),
    "nvfp4_lay_out": (dict(codes=(B, R, C // 2), output=(B, R, C // 2), rows=R, cols=C), ("codes", "output")),
    "nvfp4_lay_out, transposed": (dict(codes=(B, R, C // 2), output=(B, C, R // 2), rows=R, cols=C, transpose=True), ("codes", "output")),
    "nvfp4_gemm": (dict(a=(B, R, K // 2), a_scale=(B, 512), a_amax=(F, 1), b=(B, C, K // 2), b_scale=(B, 512), b_amax=(F, 1),
                        addend=(F, R, C), out=(F, R, C), m=R, n=C, k=K), ("a", "b", "addend", "out")),
}
NARROW = [(case, name) for case, (_, matrices) in CASES.items() for name in matrices]


def refuses(case, narrow, wrap, device):
    entry = case.split(",")[0]
    calls = [getattr(api, entry)]
    if entry != "nvfp4_lay_out":
        calls.append(getattr(api, "prepare_" + entry.removeprefix("mxfp8_")))
    args = {}
    for name, spec in CASES[case][0].items():
        if isinstance(spec, tuple):
            dtype, *shape = spec
            if name in CASES[case][1]:  # a slice of a wider buffer, one column short or just wide enough
                shape[1] += 16
                spec = wrap(torch.zeros(shape, dtype=dtype, device=device)[:, :shape[1] - 16 - (name == narrow)])
            else:
                spec = wrap(torch.zeros(shape, dtype=dtype, device=device))
        args[name] = spec
    for call in calls:
        with pytest.raises(api.MXFP8Error) as e:
            call(**args)
        assert e.value.status == 2 and str(e.value).count(f"{narrow}: shape"), str(e.value)


@pytest.mark.parametrize("case,narrow", NARROW)
def test_refused_on_the_host(case, narrow):
    refuses(case, narrow, OnGpu, "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("case,narrow", NARROW)
def test_refused(case, narrow):
    refuses(case, narrow, lambda t: t, "cuda")


@pytest.mark.gpu
def test_largest_magnitude_of_some_columns():
    """What lies beside the columns asked for counts in neither form of the call."""
    x = torch.tensor([[1.0, -5.0], [2.0, 3.0]], device="cuda")
    top = torch.empty(1, device="cuda")
    api.nvfp4_tensor_amax(x, top, 2, 1)
    assert float(top) == 2.0
    api.nvfp4_tensor_amax(x[:, :1], top, 2, 1)
    assert float(top) == 2.0
    wide = torch.arange(1.0, 1 + 300 * 40, device="cuda").view(300, 40)
    for dtype in (torch.float32, torch.bfloat16):
        w = (wide % 251).to(dtype)
        for lo, hi in ((0, 39), (1, 40), (8, 24), (39, 40)):
            api.nvfp4_tensor_amax(w[:, lo:hi], top, 300, hi - lo)
            assert float(top) == float(w[:, lo:hi].float().max())
