"""The residual norm at the ends of its range, forward and backward: rows as
small and as large as their sum of squares in fp32 allows.

Tolerance: as elsewhere for gradients, 1e-5 (2-norm of a row); sums of squares
next to fp32's smallest normal number, 1.2e-38, keep at least 20 bits here, half
of which the root leaves: that adds nothing.
"""
import numpy as np
import pytest

from layer_util import dev, host, round_to
from oracle import around_oracle as o

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [40, 1000, 4096, 16384])
@pytest.mark.parametrize("size", [2e-18, 1e-10, 1e10, 5e16])
def test_rows_of_any_size(D, size):
    from matrix_state_non_gb300 import binding as m
    r = np.random.default_rng(D)
    sign = r.choice([-1.0, 1.0], (3, D))
    h = round_to(size * sign * r.uniform(0.6, 1.4, (3, D)), "f32")
    w, dy = round_to(1.0 + 0.2 * r.normal(size=D), "f32"), round_to(r.uniform(0.2, 1.0, (3, D)) * sign, "f32")
    y, _ = o.residual_norm(h, w, None, 0.0)
    got = host(m.residual_norm(dev(h), dev(w), eps=0.0)["y"])
    assert np.linalg.norm(got - y) <= 1e-5 * np.linalg.norm(y)
    dx, dw = o.residual_norm_backward(h, w, dy, None, 0.0)
    b = m.residual_norm_backward(dev(h), dev(w), dev(dy), eps=0.0)
    for got, ref in ((b["dx"].double().cpu().numpy(), dx), (host(b["dw"])[None], dw[None])):
        assert np.isfinite(got).all()
        off, norm = np.linalg.norm(got - ref, axis=-1), np.linalg.norm(ref, axis=-1)
        assert np.all(off <= 1e-5 * norm), off / norm
