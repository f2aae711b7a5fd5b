"""The gates of the gated linear recurrence, value by value.

f = 2^-w, w = alpha softplus(z) log2 e: w is good to about 8 units of 2^-24 of
itself (z, softplus and the product with alpha), which are 8 w ln 2 2^-24 of f,
the power itself to 2^-22, the state's product to 2^-24.  At w up to 40 that is
1.4e-5 of f a step: 2e-5, and t times that behind t steps.
"""
import numpy as np
import pytest

from layer_util import dev, host, round_to
from oracle import around_oracle as o

pytestmark = pytest.mark.gpu

STEP = 2e-5


def inputs(T, C, dtype):
    """States that only decay (x = 0, H_0 = 1), with gates from 1/2 to 2^-40."""
    r = np.random.default_rng(C)
    alpha = round_to(np.full(C, 1.0), "f32")
    beta = round_to(np.log(np.expm1(np.linspace(0.6, 27.0, C))), "f32")
    return np.zeros((2, T, C)), round_to(0.1 * r.normal(size=(2, T, C)), dtype), alpha, beta, np.ones((2, C))


def within(got, ref, t, label):
    """`t` steps' tolerance, of each value (bf16 adds its rounding), down to fp32's smallest normal."""
    got = host(got).astype(np.float64)
    off = np.abs(got - ref) - t * np.abs(ref) - 1e-36
    assert np.all(off <= 0), (label, (np.abs(got - ref) / np.maximum(np.abs(ref), 1e-36)).max())


@pytest.mark.parametrize("dtype,C", [("f32", 40), ("f32", 13), ("bf16", 64), ("bf16", 9), ("bf16", 18)])
def test_small_gates_keep_their_digits(dtype, C):
    from matrix_state_non_gb300 import binding as m
    T = 20
    x, a, alpha, beta, H_0 = inputs(T, C, dtype)
    bf = 2.0 ** -8 if dtype == "bf16" else 0.0
    for n in (1, 2, 3):
        y, H = o.linear_scan(x[:, :n], a[:, :n], alpha, beta, H_0)
        xs, as_ = (dev(np.ascontiguousarray(v[:, :n]), dtype) for v in (x, a))
        got = m.linear_scan(xs, as_, dev(alpha), dev(beta), H_0=dev(H_0))
        within(got["H_T"], H, n * STEP, ("H_T", n))
        within(got["y"], y, n * STEP + bf, ("y", n))
    H = dev(H_0)
    y, ref = o.linear_scan(x[:, :1], a[:, :1], alpha, beta, H_0)
    got = m.linear_step(H, dev(x[:, 0], dtype), dev(a[:, 0], dtype), dev(alpha), dev(beta))
    within(H, ref, STEP, "step H")
    within(got, y[:, 0], STEP + bf, "step y")


@pytest.mark.parametrize("dtype,C", [("f32", 40), ("f32", 13), ("bf16", 64), ("bf16", 9)])
def test_gradients_of_states_that_decayed(dtype, C):
    """The backward differentiates the states that the gates really leave: da of later steps shows them.  The state
    before step t has t steps' tolerance, the gradient behind it 2 more."""
    from matrix_state_non_gb300 import binding as m
    T = 20
    x, a, alpha, beta, H_0 = inputs(T, C, dtype)
    dy = np.ones((2, T, C))
    ref = o.linear_scan_backward(x, a, alpha, beta, dy, H_0)
    got = m.linear_scan_backward(dev(x, dtype), dev(a, dtype), dev(alpha), dev(beta), dev(dy, dtype), H_0=dev(H_0))
    for t in range(T):
        within(got["da"][:, t], ref["da"][:, t], (t + 3) * STEP, ("da", t))
