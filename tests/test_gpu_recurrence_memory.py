"""The gated linear recurrence over memories of hundreds to thousands of steps,
channel by channel.

Tolerance: a state of memory M (1 / (1 - f)) keeps the errors of about M steps.
In each of them f is rounded (2^-25 of the state), the step's multiply-add is
(2^-24) and the products that compose steps are (2^-24): at most 2.5 2^-24 M of
the channel, if all have one sign, as they may where all gates of a channel are
alike; and the gates' own error, 1e-5.  Gradients go through two such sums.
"""
import numpy as np
import pytest

from layer_util import dev, host, round_to
from oracle import around_oracle as o

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("alike", [True, False])
@pytest.mark.parametrize("dtype,C", [("f32", 24), ("bf16", 24), ("bf16", 9)])
def test_long_memories(dtype, C, alike):
    from matrix_state_non_gb300 import binding as m
    T = 8000
    r = np.random.default_rng(C)
    memory = np.geomspace(200.0, 4000.0, C)
    alpha = round_to(np.exp(r.uniform(np.log(0.5), np.log(8.0), C)), "f32")
    beta = round_to(np.log(np.expm1(-np.log1p(-1.0 / memory) / alpha)), "f32")
    x = round_to(0.5 + r.normal(size=(1, T, C)), dtype)
    a = np.zeros((1, T, C)) if alike else round_to(0.3 * r.normal(size=(1, T, C)), dtype)
    dy = round_to(0.5 + r.normal(size=(1, T, C)), dtype)
    H_0 = round_to(r.normal(size=(1, C)), "f32")
    y, H = o.linear_scan(x, a, alpha, beta, H_0)
    ref = o.linear_scan_backward(x, a, alpha, beta, dy, H_0)
    args = (dev(x, dtype), dev(a, dtype), dev(alpha), dev(beta))
    got = m.linear_scan(*args, H_0=dev(H_0))
    bwd = m.linear_scan_backward(*args, dev(dy, dtype), H_0=dev(H_0), want_dH0=True)
    tol = 2.5 * 2.0 ** -24 * memory + 1e-5
    bf = 2.0 ** -8 if dtype == "bf16" else 0.0

    def off(g, w):
        g = host(g)
        axes = tuple(range(g.ndim - 1))
        return np.sqrt(((g - w) ** 2).sum(axes) / (w ** 2).sum(axes))

    assert np.all(off(got["H_T"], H) <= 4 * tol), off(got["H_T"], H) / tol  # (one value: may lie near 0)
    assert np.all(off(got["y"], y) <= tol + bf), off(got["y"], y) / tol
    for k in ("dx", "da"):
        assert np.all(off(bwd[k], ref[k]) <= 2 * tol), (k, off(bwd[k], ref[k]) / tol)
