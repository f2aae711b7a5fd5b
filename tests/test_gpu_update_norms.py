"""The orthogonalised update of matrices whose norm, or its inverse, fp32 cannot
hold: the result does not depend on G's size.  Tolerance: as for other sizes,
5e-3 (2-norm; the result's rounding and its operands')."""
import numpy as np
import pytest

from layer_util import dev, host
from oracle import around_oracle as o
from parity_util import rel_fro

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(40, 60), (30, 500), (140, 150), (150, 140), (520, 516), (1, 1), (2, 9000)])
def test_norms_beyond_fp32(rows, cols, dtype):
    import torch
    from matrix_state_non_gb300 import binding as m
    g = np.random.default_rng(rows).uniform(0.3, 0.9, (rows, cols)) * np.random.default_rng(cols).choice([-1.0, 1.0], (rows, cols))
    x = dev(g, dtype)
    for k in (127, 120, -120, -140):  # 127: a norm beyond the type's largest value; below -126: subnormal values
        if k == -140 and dtype == "bf16":  # (its smallest value is 2^-133)
            y = torch.sign(x) * 2.0 ** -66 * 2.0 ** -67
        else:
            y = x * 2.0 ** (k // 2) * 2.0 ** (k - k // 2)
        assert bool(y.isfinite().all()) and bool((y != 0).all())
        ref = o.orthogonalize(host(y).astype(np.float64), eps=0.0)
        got = host(m.orthogonalize(y, eps=0.0))
        assert np.all(np.isfinite(got)), k
        assert rel_fro(got, ref) <= 5e-3, (k, rel_fro(got, ref))
        if k > 0:  # eps is nothing beside such norms
            assert torch.equal(m.orthogonalize(y), m.orthogonalize(y, eps=0.0))


@pytest.mark.parametrize("rows,cols", [(40, 60), (30, 500), (140, 150)])
def test_zeros_stay_zeros_at_any_eps(rows, cols):
    import torch
    from matrix_state_non_gb300 import binding as m
    z = torch.zeros(rows, cols, device="cuda")
    for eps in (1e-7, 1e-30, 1e-39):
        assert int(m.orthogonalize(z, eps=eps).count_nonzero()) == 0, eps
