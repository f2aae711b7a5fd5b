"""Argument checks of the hybrid layer's entry points.  None of these calls
reaches the device, so they run on a host without a GPU."""
import ctypes

import pytest

from matrix_state_non_gb300 import binding as m

P = 1 << 20   # a fake, 16-byte-aligned address: never dereferenced
Q = 1 << 40   # far from the others
BF, F32 = m.M2RNN_BF16, m.M2RNN_F32
BAD, UNSUP, WS = m.M2RNN_ERR_INVALID_ARG, m.M2RNN_ERR_UNSUPPORTED, m.M2RNN_ERR_WORKSPACE


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), kw
    return fn(*dict(defaults, **kw).values())


CONV = dict(x=P, stride=64, w=P, bias=None, x0=None, lengths=None, y=Q, x_T=None, B=2, T=8, C=64, W=4, silu=1, dt=BF,
            stream=None)
CONV_BWD = dict(x=P, stride=64, w=P, bias=None, x0=None, lengths=None, dy=P, dx_T=None, dx=Q, dw=Q, db=None, dx0=None,
                B=2, T=8, C=64, W=4, silu=1, dt=BF, ws=Q, wsb=1 << 30, stream=None)
CONV_STEP = dict(state=P, x=Q, stride=64, w=P, bias=None, y=Q + (1 << 30), B=2, C=64, W=4, silu=1, dt=BF, stream=None)
SSM = dict(q=P, qs=64, k=P, ks=64, v=P, vs=128, d=P, ds=2, A=P, dt_bias=None, w_r=None, H_0=None, lengths=None, y=Q,
           H_T=None, B=1, T=8, N=2, G=1, K=64, V=64, dt=BF, ws=Q, wsb=1 << 40, stream=None)
SSM_BWD = dict(q=P, qs=64, k=P, ks=64, v=P, vs=128, d=P, ds=2, A=P, dt_bias=None, w_r=None, H_0=None, lengths=None,
               dy=P, dH_T=None, dq=Q, dk=Q, dv=Q, ddt=Q, dA=Q, ddt_bias=None, dw_r=None, dH_0=None, B=1, T=8, N=2,
               G=1, K=64, V=64, dt=BF, ws=Q, wsb=1 << 40, stream=None)
SSM_STEP = dict(H=Q, q=P, qs=64, k=P, ks=64, v=P, vs=128, d=P, ds=2, A=P, dt_bias=None, w_r=None, y=Q, B=1, N=2, G=1,
                K=64, V=64, dt=BF, stream=None)

ROWS_BAD = [dict(qs=63), dict(ks=8), dict(vs=127), dict(ds=1), dict(q=None), dict(k=P + 1), dict(v=None), dict(d=None),
            dict(A=None), dict(A=P + 4), dict(dt_bias=P + 8), dict(w_r=P + 2), dict(G=0), dict(G=3), dict(N=0),
            dict(B=0), dict(K=0), dict(V=-1), dict(dt=7)]


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=P + 1), dict(stride=63), dict(w=None), dict(w=P + 2),
                                dict(bias=P + 8), dict(x0=P + 4), dict(y=None), dict(y=Q + 8), dict(x_T=Q + 2),
                                dict(lengths=P + 2), dict(B=0), dict(T=0), dict(C=0), dict(W=0), dict(dt=5),
                                dict(silu=2), dict(y=P + 16), dict(x_T=P), dict(x0=Q), dict(x0=Q, x_T=Q)])
def test_conv_refuses(kw):
    assert call(m.m2rnn_causal_conv, CONV, **kw) == BAD


def test_conv_limits():
    assert call(m.m2rnn_causal_conv, CONV, W=9) == UNSUP
    assert m.m2rnn_causal_conv_backward_workspace_size(1, 8, 64, 9) == 0
    assert m.m2rnn_causal_conv_backward_workspace_size(1, 0, 64, 4) == 0
    assert m.m2rnn_causal_conv_backward_workspace_size(2, 1000, 64, 4) >= 2 * 5 * 64 * 4


@pytest.mark.parametrize("kw", [dict(dy=None), dict(dy=P + 4), dict(dx=None), dict(dw=None), dict(dw=Q + 4),
                                dict(db=Q + 8), dict(dx0=Q + 4), dict(dx_T=P + 8), dict(stride=1), dict(T=0),
                                dict(silu=-1), dict(dx=P), dict(dx_T=Q, dx0=Q)])
def test_conv_backward_refuses(kw):
    assert call(m.m2rnn_causal_conv_backward, CONV_BWD, **kw) == BAD


def test_conv_backward_workspace():
    need = m.m2rnn_causal_conv_backward_workspace_size(2, 8, 64, 4)
    assert call(m.m2rnn_causal_conv_backward, CONV_BWD, ws=None) == WS
    assert call(m.m2rnn_causal_conv_backward, CONV_BWD, wsb=need - 1) == WS
    assert call(m.m2rnn_causal_conv_backward, CONV_BWD, W=12) == UNSUP


@pytest.mark.parametrize("kw", [dict(state=None), dict(state=P + 8), dict(x=None), dict(y=None), dict(y=P), dict(x=P),
                                dict(y=Q), dict(stride=60), dict(B=0), dict(dt=2)])
def test_conv_step_refuses(kw):
    assert call(m.m2rnn_causal_conv_step, CONV_STEP, **kw) == BAD


@pytest.mark.parametrize("kw", ROWS_BAD + [dict(T=0), dict(y=None), dict(y=Q + 4), dict(H_T=Q + 4), dict(H_0=P + 4),
                                           dict(lengths=P + 1), dict(y=P)])
def test_ssm_scan_refuses(kw):
    assert call(m.m2rnn_ssm_scan, SSM, **kw) == BAD


@pytest.mark.parametrize("kw", ROWS_BAD + [dict(T=0), dict(dy=None), dict(dy=P + 2), dict(dq=None), dict(dk=None),
                                           dict(dv=Q + 4), dict(ddt=None), dict(dA=None), dict(ddt_bias=Q + 4),
                                           dict(dw_r=Q + 8), dict(dH_T=P + 8), dict(dH_0=P + 8), dict(dv=P),
                                           dict(dq=P)])
def test_ssm_scan_backward_refuses(kw):
    assert call(m.m2rnn_ssm_scan_backward, SSM_BWD, **kw) == BAD


@pytest.mark.parametrize("kw", ROWS_BAD + [dict(H=None), dict(H=Q + 4), dict(y=None)])
def test_ssm_step_refuses(kw):
    assert call(m.m2rnn_ssm_step, SSM_STEP, **kw) == BAD


@pytest.mark.parametrize("fn,d", [(m.m2rnn_ssm_scan, SSM), (m.m2rnn_ssm_scan_backward, SSM_BWD),
                                  (m.m2rnn_ssm_step, SSM_STEP)])
def test_ssm_limits(fn, d):
    assert call(fn, d, K=129, qs=200, ks=200) == UNSUP
    assert call(fn, d, V=129, vs=400) == UNSUP
    if "ws" in d:
        assert call(fn, d, ws=None) == WS
        assert call(fn, d, ws=Q + 4) == WS
        assert call(fn, d, wsb=16) == WS


def test_ssm_workspace_sizes():
    for size in (m.m2rnn_ssm_workspace_size, m.m2rnn_ssm_backward_workspace_size):
        assert size(1, 8, 4, 3, 64, 64, BF) == 0      # G does not divide N
        assert size(1, 0, 4, 4, 64, 64, BF) == 0
        assert size(1, 8, 4, 4, 200, 64, BF) == 0
        assert size(1, 8, 4, 4, 64, 64, 9) == 0
        for dt in (BF, F32):
            assert 0 < size(1, 8, 4, 4, 64, 64, dt) <= size(2, 800, 4, 4, 64, 64, dt)
    shared = m.m2rnn_ssm_backward_workspace_size(2, 100, 4, 2, 64, 64, BF)
    assert shared >= m.m2rnn_ssm_backward_workspace_size(2, 100, 4, 4, 64, 64, BF) + 2 * 2 * 100 * 4 * 64 * 4


def _plan(ptrs, outs, counts, dtypes, size=None):
    n = len(counts)
    counts = (ctypes.c_int64 * n)(*counts)
    need = m.m2rnn_grad_plan_size(n, counts)
    buf = (ctypes.c_uint8 * max(need, 1))()
    arr = lambda p: None if p is None else (ctypes.c_void_p * n)(*p)  # noqa: E731
    st = m.m2rnn_grad_plan_build(n, arr(ptrs), arr(outs), counts, (ctypes.c_int32 * n)(*dtypes), buf,
                                 need if size is None else size)
    return st, need, bytes(buf)


def test_grad_plan():
    st, need, buf = _plan([P, Q], None, [5, 20000], [F32, BF])
    assert st == m.M2RNN_OK and need % 32 == 0 and need > 32
    pieces = [(int.from_bytes(buf[i:i + 8], "little"), int.from_bytes(buf[i + 8:i + 16], "little"),
               int.from_bytes(buf[i + 16:i + 20], "little"), buf[i + 20]) for i in range(32, need, 32)]
    assert pieces[0] == (P, P, 5, 0)
    assert sum(p[2] for p in pieces[1:]) == 20000 and all(p[3] == 1 for p in pieces[1:])
    at = Q
    for src, dst, count, _ in pieces[1:]:  # consecutive and in place
        assert src == dst == at
        at += 2 * count
    assert m.m2rnn_grad_plan_size(0, None) == 32
    assert _plan([P], None, [0], [F32])[:2] == (m.M2RNN_OK, 32)


@pytest.mark.parametrize("a", [([None], None, [4], [F32]), ([P + 2], None, [4], [F32]), ([P + 1], None, [4], [BF]),
                               ([P], [P + 8], [4], [F32]), ([P], [None], [4], [F32]), ([P], None, [4], [3])])
def test_grad_plan_refuses(a):
    assert _plan(*a)[0] == BAD


def test_grad_plan_sizes():
    assert m.m2rnn_grad_plan_size(-1, None) == 0
    assert m.m2rnn_grad_plan_size(1, None) == 0
    assert m.m2rnn_grad_plan_size(1, (ctypes.c_int64 * 1)(-3)) == 0
    assert _plan([P], None, [4], [F32], size=32)[0] == WS


@pytest.mark.parametrize("max_norm", [0.0, -1.0, float("nan")])
def test_grad_clip_refuses_bounds(max_norm):
    assert m.m2rnn_grad_clip(P, 64, max_norm, P, P, 1 << 20, None) == BAD


def test_grad_calls_refuse():
    assert m.m2rnn_grad_norm(None, 64, P, P, 1 << 20, None) == BAD
    assert m.m2rnn_grad_norm(P, 48, P, P, 1 << 20, None) == BAD
    assert m.m2rnn_grad_norm(P, 0, P, P, 1 << 20, None) == BAD
    assert m.m2rnn_grad_norm(P, 64, None, P, 1 << 20, None) == BAD
    assert m.m2rnn_grad_norm(P, 64, P, None, 1 << 20, None) == WS
    assert m.m2rnn_grad_norm(P, 64, P, P, m.m2rnn_grad_workspace_size() - 1, None) == WS


def test_torch_helpers_refuse_host_tensors():
    import torch
    x, w = torch.zeros((1, 4, 8)), torch.zeros((8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        m.causal_conv(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        m.grad_plan([x])
    with pytest.raises(ValueError, match="no gradients"):
        m.grad_plan([])
    q = torch.zeros((1, 4, 1, 8))
    with pytest.raises(ValueError, match="CUDA"):
        m.ssm_scan(q, q, q, torch.zeros((1, 4, 1)), torch.zeros(1))
