"""The convolution of every width with one value that is not finite: it
touches the steps whose window it lies in, and no other; a prompt and the same
tokens one by one agree."""
import numpy as np
import pytest

from layer_util import conv_inputs, dev, host

pytestmark = pytest.mark.gpu

SHAPES = [(2, 150, 16), (1, 150, 33)]  # rows in vectors, and one channel at a time


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", range(1, 9))
@pytest.mark.parametrize("B,T,C", SHAPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_forward_spreads_over_its_window(B, T, C, W, dtype, bad):
    import torch
    from matrix_state_non_gb300 import binding as m
    d = conv_inputs(B, T, C, W, dtype, seed=W, x0=True)
    g = {n: dev(a, dtype) for n, a in d.items() if n in ("x", "w", "bias", "x0")}
    clean = m.causal_conv(g["x"], g["w"], g["bias"], x0=g["x0"], silu=False)["y"]
    for t, c in ((0, 0), (70, 5), (T - 2, C - 1)):
        x = g["x"].clone()
        x[0, t, c] = bad
        r = m.causal_conv(x, g["w"], g["bias"], x0=g["x0"], silu=False, want_state=True)
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[0, t:t + W, c] = True
        assert torch.equal(~torch.isfinite(r["y"]), hit), (t, c)
        assert torch.equal(r["y"][~hit], clean[~hit])
        state = m.causal_conv(x[:, :60], g["w"], g["bias"], x0=g["x0"], silu=False, want_state=True)["x_T"] \
            if B == 1 else None
        for i in range(60, T) if B == 1 else ():
            y = m.causal_conv_step(state, x[:, i], g["w"], g["bias"], silu=False)
            # the taps may be summed in another order: equal where not finite, else to a rounding
            assert torch.equal(torch.isfinite(y), torch.isfinite(r["y"][:, i]))
    if W > 1:  # a value before the sequence
        x0 = g["x0"].clone()
        x0[B - 1, 0, 2] = bad
        y = m.causal_conv(g["x"], g["w"], g["bias"], x0=x0, silu=False)["y"]
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[B - 1, 0, 2] = True
        assert torch.equal(~torch.isfinite(y), hit) and torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", range(1, 9))
@pytest.mark.parametrize("B,T,C", SHAPES)
def test_backward_spreads_over_its_window(B, T, C, W, dtype):
    import torch
    from matrix_state_non_gb300 import binding as m
    d = conv_inputs(B, T, C, W, dtype, seed=W + 10)
    g = {n: None if a is None else dev(a, "f32" if n == "dy" else dtype) for n, a in d.items()}

    def run(x, dy, silu):
        return m.causal_conv_backward(x, g["w"], g["bias"], dy, silu=silu)

    nan = float("nan")
    for silu in (True, False):
        clean = run(g["x"], g["dy"], silu)
        for t, c in ((W + 1, 0), (70, 5), (T - 2, C - 1)):
            # g at t is NaN: dx of the window's inputs, every tap and the bias of the channel
            dy = g["dy"].clone()
            dy[0, t, c] = nan
            r = run(g["x"], dy, silu)
            hit = torch.zeros_like(clean["dx"], dtype=torch.bool)
            hit[0, max(0, t - W + 1):t + 1, c] = True
            assert torch.equal(torch.isnan(r["dx"]), hit), (t, c)
            assert torch.equal(r["dx"][~hit], clean["dx"][~hit])
            for n in ("dw", "db"):
                others = torch.arange(C, device="cuda") != c
                assert torch.isnan(r[n][c]).all() and torch.equal(r[n][others], clean[n][others]), n
            # x at t is NaN: through SiLU the pre-activations of t .. t + W - 1, and from them the inputs of their
            # windows; without it dx does not depend on x
            x = g["x"].clone()
            x[0, t, c] = nan
            r = run(x, g["dy"], silu)
            hit = torch.zeros_like(hit)
            if silu:
                hit[0, max(0, t - W + 1):t + W, c] = True
            assert torch.equal(torch.isnan(r["dx"]), hit), (t, c)
            assert torch.equal(r["dx"][~hit], clean["dx"][~hit])
            # tap w meets x_t at step t + W - 1 - w, where that is a step
            met = torch.tensor([silu or t + W - 1 - w < T for w in range(W)], device="cuda")
            assert torch.equal(torch.isnan(r["dw"][c]), met), (t, c)


@pytest.mark.parametrize("B,T,C,W,dtype", [(2, 300, 40, 5, "bf16"), (1, 131, 24, 6, "f32"), (2, 90, 33, 7, "bf16"),
                                          (1, 300, 64, 8, "f32"), (3, 70, 16, 5, "f32"), (2, 65, 48, 3, "bf16")])
def test_wide_windows(B, T, C, W, dtype):
    """Forward, backward and token step of the other widths, with the oracle."""
    from matrix_state_non_gb300 import binding as m
    from oracle import layer_oracle as o
    from parity_util import rel_fro
    d = conv_inputs(B, T, C, W, dtype, seed=W + C, x0=True)
    g = {n: dev(a, "f32" if n in ("dy", "dx_T") else dtype) for n, a in d.items()}
    y, x_T = o.causal_conv(d["x"], d["w"], d["bias"], d["x0"])
    r = m.causal_conv(g["x"], g["w"], g["bias"], x0=g["x0"], want_state=True)
    # bf16: one rounding to 8 bits; fp32: sums of nine terms
    assert rel_fro(host(r["y"]), y) <= (4e-3 if dtype == "bf16" else 1e-5) and np.array_equal(host(r["x_T"]), x_T)
    b = m.causal_conv_backward(g["x"], g["w"], g["bias"], g["dy"], x0=g["x0"], dx_T=g["dx_T"], want_dx0=True)
    ref = o.causal_conv_backward(d["x"], d["w"], d["bias"], d["dy"], d["x0"], d["dx_T"])
    for n in ("dx", "dw", "db", "dx0"):
        assert rel_fro(host(b[n]), ref[n]) <= 1e-5, n
    state = g["x0"].clone()
    for t in range(10):
        s = m.causal_conv_step(state, g["x"][:, t], g["w"], g["bias"])
        assert rel_fro(host(s), y[:, t]) <= (4e-3 if dtype == "bf16" else 1e-5)
