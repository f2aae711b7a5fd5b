"""The orthogonalised update of matrices of low rank, over more than its five
usual steps.  Where G has nothing, X has rounding noise, which grows 3.4445-fold
a step, so that the parts X is kept in show there first.

Tolerance: what five steps are held to (5e-3, 2-norm), and the growth of what
X's 22 bits leave: 2^-22 of X at most in each step, 3.4445^n of the first one's
and 1.41 as much for all (a geometric sum), over a result that is 0.67 of a unit
or more for each singular value while X began with a norm of 1, so over
0.67 sqrt(rank): 2.1 2^-22 3.4445^n / sqrt(rank).
"""
import numpy as np
import pytest

from layer_util import dev
from oracle import around_oracle as o

pytestmark = pytest.mark.gpu

A, B, C = o.COEFFICIENTS


def tolerance(steps, rank):
    return 5e-3 + 2.1 * 2.0 ** -22 * A ** steps / rank ** 0.5


def low_rank(n, rows, cols, rank, dtype):
    """bf16: products and sums that bf16 holds, so that the rank is exact (integers below 256)."""
    r = np.random.default_rng(rows + cols + rank)
    if dtype == "bf16":
        return r.integers(-2, 3, (n, rows, rank)).astype(np.float64) @ r.integers(-2, 3, (n, rank, cols)).astype(np.float64)
    return r.normal(size=(n, rows, rank)) @ r.normal(size=(n, rank, cols))


def reference(x, steps):
    """In float64, from the values the library got."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.mT if tall else x
    x = x / (x.norm() + 1e-7)
    for _ in range(steps):
        gram = x @ x.mT
        x = A * x + (B * gram + C * gram @ gram) @ x
    return x.mT if tall else x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rank", [1, 32])
@pytest.mark.parametrize("steps", [5, 6, 7, 8, 10])
@pytest.mark.parametrize("n,rows,cols", [(1, 520, 516), (1, 300, 400), (20, 800, 800), (1, 700, 2000)])
def test_low_rank_over_more_steps(n, rows, cols, steps, rank, dtype):
    from matrix_state_non_gb300 import binding as m
    x = dev(low_rank(n, rows, cols, rank, dtype), dtype)
    got = m.orthogonalize(x, steps=steps)
    for i in {0, n - 1}:
        ref = reference(x[i], steps)
        off = float((got[i].double() - ref).norm() / ref.norm())
        assert off <= tolerance(steps, rank), (i, off, tolerance(steps, rank))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rank", [1, 4])
@pytest.mark.parametrize("steps", [5, 6, 7, 8, 10])
@pytest.mark.parametrize("rows,cols", [(64, 64), (20, 30), (64, 200), (64, 513), (2100, 64), (20, 700), (40, 4000)])
def test_low_rank_over_more_steps_with_a_short_side(rows, cols, steps, rank, dtype):
    """In shared memory, and through m x m matrices in fp32.  Products of so few small integers are all of one size or two,
    which the result's rounding, 2^-8 at most, leaves no average of: that in place of its 1.7e-3 in the mean."""
    from matrix_state_non_gb300 import binding as m
    x = dev(low_rank(1, rows, cols, rank, dtype), dtype)[0]
    ref = reference(x, steps)
    off = float((m.orthogonalize(x, steps=steps).double() - ref).norm() / ref.norm())
    assert off <= tolerance(steps, rank) + 2.0 ** -8 - 1.7e-3, off
