"""Argument checks of the residual norm, the gated linear recurrence and the
orthogonalised update.  None of these calls reaches the device."""
import pytest
import torch

from matrix_state_non_gb300 import binding as m
from test_layer_calls import On

P, Q, R, S = 1 << 20, 1 << 40, 1 << 41, 1 << 42  # fake, 16-byte-aligned addresses far from each other
BF, F32, E4 = m.M2RNN_BF16, m.M2RNN_F32, m.M2RNN_E4M3
BAD, UNSUP, WS = m.M2RNN_ERR_INVALID_ARG, m.M2RNN_ERR_UNSUPPORTED, m.M2RNN_ERR_WORKSPACE
nan, inf = float("nan"), float("inf")


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), kw
    return fn(*dict(defaults, **kw).values())


NORM = dict(x=P, stride=64, residual=2 * P, w=3 * P, eps=1e-6, h=Q, y=R, scale=None, rows=8, D=64, xt=BF, ht=BF, yt=BF,
            stream=None)
NORM_BWD = dict(h=P, w=2 * P, dy=3 * P, dh=4 * P, eps=1e-6, dx=Q, dw=R, rows=8, D=64, ht=BF, dt=BF, ws=S, wsb=1 << 30,
                stream=None)
SCAN = dict(x=P, xs=64, a=2 * P, as_=64, alpha=3 * P, beta=None, H_0=None, lengths=None, y=Q, H_T=None, B=2, T=8, C=64,
            dt=BF, stream=None)
SCAN_BWD = dict(x=P, xs=64, a=2 * P, as_=64, alpha=3 * P, beta=None, H_0=None, lengths=None, dy=4 * P, dH_T=None, dx=Q,
                da=Q + P, dalpha=R, dbeta=None, dH_0=None, B=2, T=8, C=64, dt=BF, ws=S, wsb=1 << 30, stream=None)
STEP = dict(H=Q, x=P, xs=64, a=2 * P, as_=64, alpha=3 * P, beta=None, y=R, B=2, C=64, dt=BF, stream=None)
ORTHO = dict(g=P, out=Q, n=2, rows=64, cols=64, steps=5, eps=1e-7, dt=F32, ws=S, wsb=1 << 40, stream=None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=P + 1), dict(stride=63), dict(residual=P + 8), dict(w=None), dict(w=3 * P + 4), dict(h=Q + 2),
    dict(y=None), dict(y=R + 8), dict(scale=S), dict(yt=E4), dict(yt=E4, scale=S + 4), dict(rows=0), dict(D=0),
    dict(D=-1), dict(xt=E4), dict(ht=E4), dict(yt=3), dict(xt=9), dict(eps=-1e-6), dict(eps=nan), dict(eps=inf),
    dict(residual=None), dict(y=P), dict(y=2 * P), dict(h=P), dict(h=2 * P + 16), dict(y=Q), dict(y=3 * P),
    dict(yt=E4, scale=R), dict(h=R + 16), dict(x=P, residual=P, h=P)])
def test_norm_refuses(kw):
    assert call(m.m2rnn_residual_norm, NORM, **kw) == BAD


def test_norm_limits():
    assert call(m.m2rnn_residual_norm, NORM, D=16385, stride=16385) == UNSUP
    assert call(m.m2rnn_residual_norm, NORM, rows=1 << 40) == UNSUP
    size = m.m2rnn_residual_norm_backward_workspace_size
    assert size(0, 64) == size(8, 0) == size(8, 16385) == 0
    assert 0 < size(1, 64) <= size(100000, 64)


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(h=P + 8), dict(w=None), dict(dy=None), dict(dy=3 * P + 2), dict(dh=4 * P + 4), dict(dx=None),
    dict(dx=Q + 4), dict(dw=None), dict(dw=R + 8), dict(rows=0), dict(D=0), dict(ht=E4), dict(dt=E4), dict(eps=nan),
    dict(dx=P), dict(dx=3 * P), dict(dx=4 * P + 16), dict(dw=Q), dict(dw=2 * P), dict(dh=P, dx=P), dict(ws=P), dict(ws=3 * P),
    dict(ws=4 * P), dict(ws=Q), dict(ws=R)])
def test_norm_backward_refuses(kw):
    assert call(m.m2rnn_residual_norm_backward, NORM_BWD, **kw) == BAD


def test_norm_backward_workspace():
    need = m.m2rnn_residual_norm_backward_workspace_size(8, 64)
    for kw in (dict(ws=None), dict(ws=S + 8), dict(wsb=need - 1)):
        assert call(m.m2rnn_residual_norm_backward, NORM_BWD, **kw) == WS


ROWS_BAD = [dict(x=None), dict(x=P + 1), dict(a=None), dict(a=2 * P + 1), dict(xs=63), dict(as_=1), dict(alpha=None),
            dict(alpha=3 * P + 4), dict(beta=P + 8), dict(B=0), dict(C=0), dict(dt=E4), dict(dt=-1)]


@pytest.mark.parametrize("kw", ROWS_BAD + [
    dict(T=0), dict(y=None), dict(y=Q + 8), dict(H_T=Q + 4), dict(H_0=S + 4), dict(lengths=S + 2), dict(y=P),
    dict(y=2 * P), dict(H_T=Q), dict(H_0=S, H_T=S + 16), dict(H_T=P), dict(y=3 * P), dict(H_0=Q)])
def test_linear_scan_refuses(kw):
    assert call(m.m2rnn_linear_scan, SCAN, **kw) == BAD


@pytest.mark.parametrize("kw", ROWS_BAD + [
    dict(T=0), dict(dy=None), dict(dy=4 * P + 8), dict(dx=None), dict(da=Q + 4), dict(dalpha=None), dict(dbeta=R + 4),
    dict(dH_0=S + 4), dict(dH_T=S + 8), dict(dx=P), dict(da=4 * P), dict(da=Q), dict(dbeta=R), dict(dH_0=3 * P),
    dict(dH_T=S, dH_0=S + 16), dict(H_0=S, dH_0=S), dict(ws=P),
    dict(ws=4 * P), dict(ws=Q), dict(ws=R), dict(dbeta=S), dict(dH_0=S)])
def test_linear_scan_backward_refuses(kw):
    assert call(m.m2rnn_linear_scan_backward, SCAN_BWD, **kw) == BAD


def test_linear_scan_workspace():
    size = m.m2rnn_linear_backward_workspace_size
    assert size(0, 8, 64) == size(2, 0, 64) == size(2, 8, 0) == 0
    assert size(1 << 20, 1 << 20, 64) == 0
    for kw in (dict(ws=None), dict(ws=S + 4), dict(wsb=size(2, 8, 64) - 1)):
        assert call(m.m2rnn_linear_scan_backward, SCAN_BWD, **kw) == WS
    assert call(m.m2rnn_linear_scan, SCAN, B=1 << 16, T=1 << 16) == UNSUP


@pytest.mark.parametrize("kw", ROWS_BAD + [dict(H=None), dict(H=Q + 4), dict(y=None), dict(y=R + 2), dict(y=Q), dict(H=P),
                                           dict(y=2 * P)])
def test_linear_step_refuses(kw):
    assert call(m.m2rnn_linear_step, STEP, **kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(g=None), dict(g=P + 8), dict(out=None), dict(out=Q + 2), dict(n=0), dict(rows=0), dict(cols=0), dict(steps=0),
    dict(steps=33), dict(eps=-1.0), dict(eps=nan), dict(dt=E4), dict(out=P), dict(out=P + 16, dt=BF), dict(ws=P), dict(ws=Q)])
def test_orthogonalize_refuses(kw):
    assert call(m.m2rnn_orthogonalize, ORTHO, **kw) == BAD


def test_orthogonalize_limits():
    size = m.m2rnn_orthogonalize_workspace_size
    assert size(0, 4, 4) == size(1, 0, 4) == size(1, 4, 16385) == size(65536, 4, 4) == 0
    assert 0 < size(1, 4, 4) <= size(3, 4, 4) and size(1, 700, 300) == size(1, 300, 700)
    assert call(m.m2rnn_orthogonalize, ORTHO, cols=16385) == UNSUP
    for kw in (dict(ws=None), dict(ws=S + 8), dict(wsb=size(2, 64, 64) - 1)):
        assert call(m.m2rnn_orthogonalize, ORTHO, **kw) == WS


# ---------------------------------------------------------------------------
# The torch helpers
# ---------------------------------------------------------------------------
def test_helpers_refuse_host_tensors():
    x, c = torch.zeros((2, 3, 8)), torch.zeros(8)
    for f in (lambda: m.residual_norm(x, c), lambda: m.residual_norm_backward(x, c, x), lambda: m.linear_scan(x, x, c),
              lambda: m.linear_scan_backward(x, x, c, None, x), lambda: m.linear_step(x[0], x[0], x[0], c),
              lambda: m.orthogonalize(x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.fixture
def current(monkeypatch):
    """cuda:0 is current; a call of the library fails."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "load", lambda: pytest.fail("the library was called"))
    monkeypatch.setattr(m, "_alloc", lambda like, shape, dtype, stream: On(shape, dtype, like.get_device()))


def test_tensors_of_another_than_the_current_gpu_are_refused(current):
    x, c = On((2, 3, 8), gpu=1), On((8,), gpu=1)
    s = On((3, 8), gpu=1)
    for f in (lambda: m.residual_norm(x, c), lambda: m.residual_norm_backward(x, c, x), lambda: m.linear_scan(x, x, c),
              lambda: m.linear_scan_backward(x, x, c, None, x), lambda: m.linear_step(s, s, s, c),
              lambda: m.orthogonalize(x)):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            f()


def test_helpers_refuse_shapes_and_types(current, monkeypatch):
    called = lambda *a: pytest.fail("the library was called")  # noqa: E731
    lib = {n: (lambda *a: 64) if n.endswith("size") else called for n in m.EXPORTS}
    monkeypatch.setattr(m, "load", lambda: type("Lib", (), lib))
    b, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, c = On((2, 3, 8), b), On((8,))
    wrong = [lambda: m.residual_norm(x, On((7,))), lambda: m.residual_norm(x, On((8,), b)),
             lambda: m.residual_norm(x, c, On((2, 8), b)), lambda: m.residual_norm(x, c, On((2, 3, 8), gpu=1)),
             lambda: m.residual_norm(x, c, dtype=f8, out=dict(scale=On((2, 3, 2)))),
             lambda: m.residual_norm(x, c, out=dict(y=On((2, 3, 8)))),
             lambda: m.residual_norm_backward(x, c, On((2, 8), b)), lambda: m.residual_norm_backward(x, c, x, dh=x),
             lambda: m.linear_scan(x, On((2, 3, 8)), c), lambda: m.linear_scan(x, On((2, 3, 7), b), c),
             lambda: m.linear_scan(x, x, c, H_0=On((2, 8), b)), lambda: m.linear_scan(x, x, c, lengths=On((2,))),
             lambda: m.linear_scan_backward(x, x, c, None, On((2, 3, 8))),
             lambda: m.linear_step(On((3, 8), b), On((3, 8), b), On((3, 8), b), c),
             lambda: m.linear_step(On((3, 8)), On((3, 8), b), On((3, 8), b), c, y=On((3, 8))),
             lambda: m.orthogonalize(On((8,))), lambda: m.orthogonalize(On((4, 8)), out=On((4, 8))),
             lambda: m.orthogonalize(On((4, 8)), workspace=On((64,), torch.uint8, 1))]
    for i, f in enumerate(wrong):
        with pytest.raises(ValueError):
            f()
            pytest.fail(str(i))
    for f in (lambda: m.residual_norm(x, c, dtype=torch.float16), lambda: m.residual_norm(On((2, 8), f8), c),
              lambda: m.linear_scan(On((2, 3, 8), torch.float16), x, c), lambda: m.orthogonalize(On((4, 8), torch.float16))):
        with pytest.raises(TypeError):
            f()


def test_flat_rows():
    """Rows of a column slice: evenly spaced through all leading dimensions, or refused."""
    t = torch.zeros((2, 3, 10))

    class Here:
        def __init__(self, t):
            self.t = t

        def __getattr__(self, n):
            return getattr(self.t, n)

        def get_device(self):
            return 0

    at = lambda t: m._flat_rows(Here(t), "x", torch.float32, 0)[1]  # noqa: E731
    assert at(t) == 10 and at(t[..., :4]) == 10 and at(t[:1, :, :4]) == 10 and at(t[:, :1, :4]) == 30
    assert at(t[0, 0, :4]) == 4 and at(torch.zeros((4, 5))[:, :1]) == 5
    for bad in (t[:, :2, :4], t.mT, t[..., ::2], t.transpose(0, 1)[..., :4]):
        with pytest.raises(ValueError):
            at(bad)
