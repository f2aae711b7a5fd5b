"""The orthogonalised update of matrices whose values are all of one size, and of
rank 1 or 2, so that rounding errors add up instead of averaging.

Tolerance: the result's rounding is up to 2^-8 there (all its values are rounded
alike).  Long matrices with a side of up to 64 take their steps in fp32, whose
noise, 2^-24, grows 3.44-fold a step and adds up over up to 64 values of a row:
2e-3.  The others' products take operands in fp16, A and P to 2^-11 at most, all
to one side; a step's polynomial has a slope of up to 4 in what A and P are off
and hands up to 4 times that on, and most of it falls back within [0.67, 1.2]: 12
times 2^-11, 6e-3.
"""
import numpy as np
import pytest

from layer_util import dev
from test_gpu_update_steps import reference

pytestmark = pytest.mark.gpu

THIN, WIDE = 2.0 ** -8 + 2e-3, 2.0 ** -8 + 6e-3


def alike(rows, cols, kind):
    r = np.random.default_rng(rows + cols)
    if kind == "ones":
        return np.ones((rows, cols))
    rank = 1 if kind == "signs" else 2
    return r.choice([-1.0, 1.0], (rows, rank)) @ r.choice([-1.0, 1.0], (rank, cols))


@pytest.mark.parametrize("kind", ["ones", "signs", "sum"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,tol", [(64, 513, THIN), (2100, 64, THIN), (64, 2000, THIN), (33, 4000, THIN), (1, 300, THIN),
                                           (9000, 5, THIN), (64, 64, WIDE), (300, 400, WIDE), (520, 516, WIDE), (700, 2000, WIDE),
                                           (1024, 1024, WIDE)])
def test_values_of_one_size(rows, cols, tol, dtype, kind):
    from matrix_state_non_gb300 import binding as m
    x = dev(alike(rows, cols, kind), dtype)
    for steps in (1, 4, 5):
        ref = reference(x, steps)
        off = float((m.orthogonalize(x, steps=steps).double() - ref).norm() / ref.norm())
        assert off <= tol, (steps, off, tol)
