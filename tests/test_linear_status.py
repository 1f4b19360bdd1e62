"""A kernel that gave up a wait is heard of: by a layer's check, and before run_case prints a figure."""
import pytest
import torch

from mxfp8_master_weight_gb300 import api, linear, run_case


@pytest.fixture
def a_wait_given_up(monkeypatch):
    asked = []

    def status(device=None, stream=None):
        asked.append(device)
        raise api.MXFP8Error(6, "a kernel gave up waiting")
    monkeypatch.setattr(api, "mxfp8_device_status", status)
    return asked


def test_check_raises(a_wait_given_up):
    layer = object.__new__(linear.NormLinear)  # its buffers are on the GPU
    layer.device = torch.device("cuda", 0)
    with pytest.raises(api.MXFP8Error) as e:
        layer.check()
    assert e.value.status == 6 and a_wait_given_up == [torch.device("cuda", 0)]


@pytest.mark.gpu
def test_run_case_prints_no_figure_of_invalid_steps(a_wait_given_up, capsys):
    with pytest.raises(api.MXFP8Error):
        run_case.main(["linear", "--calls", "1", "--scale", "64"])
    assert "us per call" not in capsys.readouterr().out


@pytest.mark.gpu
def test_check_of_a_healthy_layer(capsys):
    layer = linear.NormLinear(8, 64, 32)
    layer.refresh([torch.randn(32 * 64, device="cuda")])
    layer.forward(torch.randn(8, 64, device="cuda").bfloat16())
    layer.check()
    run_case.main(["linear", "--calls", "1", "--scale", "64"])
    assert "us per call" in capsys.readouterr().out
