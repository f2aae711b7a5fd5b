"""The torch helpers of the layer's operators on tensors that they must not
hand to the library.  Nothing here reaches a GPU: the tensors are stand-ins,
and the library's calls fail the test."""
import pytest
import torch

from matrix_state_non_gb300 import binding as m


class On:
    """Stands in for a dense CUDA tensor on `gpu`."""

    def __init__(self, shape, dtype=torch.float32, gpu=0):
        self.shape, self.dtype, self.gpu, self.device = torch.Size(shape), dtype, gpu, f"cuda:{gpu}"
        self.streams = []

    def get_device(self):
        return self.gpu

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, s):
        self.streams.append(s)


@pytest.fixture
def current(monkeypatch):
    """cuda:0 is current; a call of the library fails."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "load", lambda: pytest.fail("the library was called"))


def test_tensors_of_another_than_the_current_gpu_are_refused(current):
    f, b = torch.float32, torch.bfloat16
    x, w = On((2, 9, 8), b, 1), On((8, 4), b, 1)
    q, v, dt, A = On((2, 9, 1, 8), b, 1), On((2, 9, 2, 8), b, 1), On((2, 9, 2), b, 1), On((2,), f, 1)
    plan = m.GradPlan.__new__(m.GradPlan)
    plan.gpu, plan.table, plan.workspace, plan.stream = 1, On((64,), torch.uint8, 1), On((8192,), torch.uint8, 1), 0
    for call in (lambda: m.causal_conv(x, w), lambda: m.causal_conv_backward(x, w, None, On((2, 9, 8), f, 1)),
                 lambda: m.causal_conv_step(On((2, 3, 8), b, 1), On((2, 8), b, 1), w),
                 lambda: m.ssm_scan(q, q, v, dt, A), lambda: m.ssm_scan_backward(q, q, v, dt, A, v),
                 lambda: m.ssm_step(On((2, 2, 8, 8), f, 1), On((2, 1, 8), b, 1), On((2, 1, 8), b, 1), On((2, 2, 8), b, 1),
                                    On((2, 2), b, 1), A),
                 lambda: m.grad_plan([x]), lambda: m.grad_norm(plan), lambda: m.grad_clip(plan, 1.0)):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            call()
