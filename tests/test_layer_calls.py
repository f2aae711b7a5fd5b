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


@pytest.mark.parametrize("norm", [On((), gpu=-1), On((), torch.float64), On((), torch.bfloat16), On((0,)), On((2,)),
                                  On((), gpu=1)])
def test_norm_is_checked(current, norm):
    plan = m.GradPlan.__new__(m.GradPlan)
    plan.gpu, plan.table, plan.workspace, plan.stream = 0, On((64,), torch.uint8), On((8192,), torch.uint8), 0
    for call in (lambda: m.grad_norm(plan, norm=norm), lambda: m.grad_clip(plan, 1.0, norm=norm)):
        with pytest.raises(ValueError, match="norm"):
            call()


def test_workspaces_are_checked(monkeypatch):
    """One on the host, on another GPU, or in pieces; one that is too small is replaced."""
    b, made = torch.bfloat16, []
    lib = type("Lib", (), dict(m2rnn_ssm_workspace_size=lambda *a: 1000, m2rnn_ssm_backward_workspace_size=lambda *a: 1000,
                               m2rnn_causal_conv_backward_workspace_size=lambda *a: 1000))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "load", lambda: lib)

    def alloc(like, shape, dtype, stream):
        made.append(On(shape if isinstance(shape, tuple) else (), dtype))
        return made[-1]

    monkeypatch.setattr(m, "_alloc", alloc)
    q, v, dt, A = On((2, 9, 1, 8), b), On((2, 9, 2, 8), b), On((2, 9, 2), b), On((2,))
    pieces = On((2000,), torch.uint8)
    pieces.is_contiguous = lambda: False
    for ws in (On((2000,), torch.uint8, -1), On((2000,), torch.uint8, 1), pieces):
        for call in (lambda: m.ssm_scan(q, q, v, dt, A, workspace=ws),
                     lambda: m.ssm_scan_backward(q, q, v, dt, A, v, workspace=ws),
                     lambda: m.causal_conv_backward(On((2, 9, 8), b), On((8, 4), b), None, On((2, 9, 8)), workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
    good = On((1000,), torch.uint8)
    assert m._scratch(good, 1000, v, None, "") is good
    assert m._scratch(On((999,), torch.uint8), 1000, v, None, "") is made[-1] and made[-1].shape == (1000,)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("call", [m.grad_norm, lambda plan, **kw: m.grad_clip(plan, 1.0, **kw)])
def test_a_plan_used_on_another_stream_stays_until_that_stream_is_done(monkeypatch, call):
    """The table and the workspace belong to the stream that the plan was made
    on; where another stream uses them, the allocator is told."""
    lib = type("Lib", (), dict(m2rnn_grad_norm=lambda *a: 0, m2rnn_grad_clip=lambda *a: 0))
    here = [Stream(7)]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: here[0])
    monkeypatch.setattr(m, "load", lambda: lib)
    monkeypatch.setattr(m, "_on", lambda gpu, stream: (stream or here[0]).cuda_stream)

    def plan():
        p = m.GradPlan.__new__(m.GradPlan)
        p.gpu, p.table, p.workspace, p.stream = 0, On((64,), torch.uint8), On((8192,), torch.uint8), 7
        return p

    norm, p = On(()), plan()
    call(p, norm=norm)
    call(p, norm=norm, stream=here[0])
    assert p.table.streams == [] and p.workspace.streams == []
    side = Stream(9)
    call(p, norm=norm, stream=side)
    assert p.table.streams == [side] and p.workspace.streams == [side]
    p, here[0] = plan(), side
    call(p, norm=norm)
    assert p.table.streams == [side] and p.workspace.streams == [side]


@pytest.mark.gpu
def test_a_dropped_plan_is_not_handed_out_while_a_side_stream_reads_it():
    grads = [torch.randn(70001, device="cuda"), torch.randn(30000, device="cuda").bfloat16()]
    want = float(m.grad_norm(m.grad_plan(grads)))
    side = torch.cuda.Stream()
    for use in (lambda p: m.grad_norm(p, stream=side), lambda p: m.grad_clip(p, 1e9, stream=side)):
        plan = m.grad_plan(grads)
        size, at = plan.table.numel(), {plan.table.data_ptr(), plan.workspace.data_ptr()}
        work = plan.workspace.numel()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # about a tenth of a second
        norm = use(plan)
        del plan
        other = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (size, work) for _ in range(4)]
        busy = not side.query()
        assert not busy or not at & {t.data_ptr() for t in other}
        side.synchronize()
        assert float(norm) == want
