"""The hybrid layer's float64 oracle: its gradients against central
differences, and closed forms."""
import numpy as np
import pytest

from layer_util import SSM_IN, SSM_OPT, conv_inputs, ssm_inputs
from oracle import layer_oracle as o


def _differences(f, args, names, h=1e-6):
    for n in names:
        a = args[n]
        g = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = f()
            a[i] = keep - h
            g[i] = (up - f()) / (2 * h)
            a[i] = keep
        yield n, g


@pytest.mark.parametrize("W,silu,lengths", [(4, True, None), (3, False, (2, 0)), (2, True, (5, 1))])
def test_conv_gradients_are_differences(W, silu, lengths):
    d = conv_inputs(2, 5, 3, W, "f32", seed=W, x0=True)
    kw = dict(lengths=lengths, silu=silu)

    def loss():
        y, x_T = o.causal_conv(d["x"], d["w"], d["bias"], d["x0"], **kw)
        return (y * d["dy"]).sum() + (x_T * d["dx_T"]).sum()

    got = o.causal_conv_backward(d["x"], d["w"], d["bias"], d["dy"], d["x0"], d["dx_T"], **kw)
    names = dict(x="dx", w="dw", bias="db", x0="dx0")
    for n, g in _differences(loss, d, names):
        np.testing.assert_allclose(got[names[n]], g, atol=2e-8, rtol=1e-6)


def test_conv_of_width_one_is_a_gate():
    d = conv_inputs(1, 4, 3, 1, "f32", seed=9)
    y, x_T = o.causal_conv(d["x"], d["w"], d["bias"], silu=False)
    np.testing.assert_allclose(y, d["x"] * d["w"][:, 0] + d["bias"], rtol=1e-15)
    assert x_T.shape == (1, 0, 3)


@pytest.mark.parametrize("N,G,lengths", [(2, 2, None), (4, 2, (4, 1)), (2, 1, (0, 3))])
def test_ssm_gradients_are_differences(N, G, lengths):
    d = ssm_inputs(2, 4, N, G, 3, 2, "f32", seed=N + G)
    d["dt_bias"] += 2.0  # larger steps: every term counts
    d["A"] /= 8.0

    def args():
        return [d[n] for n in SSM_IN], {n: d[n] for n in SSM_OPT}

    def loss():
        a, kw = args()
        y, H = o.ssm_scan(*a, lengths=lengths, **kw)
        return (y * d["dy"]).sum() + (H * d["dH_T"]).sum()

    a, kw = args()
    got = o.ssm_scan_backward(*a, d["dy"], dH_T=d["dH_T"], lengths=lengths, **kw)
    for n, g in _differences(loss, d, SSM_IN + SSM_OPT):
        np.testing.assert_allclose(got["d" + n], g, atol=3e-8, rtol=1e-6, err_msg=n)


def test_ssm_without_decay_is_linear_attention():
    d = ssm_inputs(1, 6, 2, 1, 4, 3, "f32", seed=5, h0=False, decay=0.0)
    y, H = o.ssm_scan(*(d[n] for n in SSM_IN), dt_bias=d["dt_bias"])
    D = np.logaddexp(d["dt"] + d["dt_bias"], 0.0)
    s = np.tril(np.einsum("btk,bsk->bts", d["q"][:, :, 0], d["k"][:, :, 0]))
    np.testing.assert_allclose(y, np.einsum("bts,bsn,bsnv->btnv", s, D, d["v"]), rtol=1e-12)
    np.testing.assert_allclose(H, np.einsum("bsk,bsn,bsnv->bnkv", d["k"][:, :, 0], D, d["v"]), rtol=1e-12)


def test_clip():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    norm, c = o.clip(g, 1.0)
    assert norm == 5.0
    np.testing.assert_allclose(c[1], [[0.8]], rtol=1e-6)
    assert np.array_equal(o.clip(g, 10.0)[1][0], g[0])
