"""The batched 64-bit reference of the scan against the plain loops."""
import numpy as np
import pytest
import scan_reference as r

from layer_util import SSM_IN, SSM_OPT, ssm_inputs
from oracle import layer_oracle as o


@pytest.mark.parametrize("lengths", [None, (9, 0, 1)])
@pytest.mark.parametrize("h0", [True, False])
def test_reference_is_the_definition(lengths, h0):
    d = ssm_inputs(3, 9, 4, 2, 5, 3, "f32", seed=3, h0=h0)
    a, kw = [d[n] for n in SSM_IN], {n: d[n] for n in SSM_OPT}
    got = r.scan(d, lengths)
    y, H = o.ssm_scan(*a, lengths=lengths, **kw)
    want = dict(o.ssm_scan_backward(*a, d["dy"], dH_T=d["dH_T"], lengths=lengths, **kw), y=y, H_T=H)
    for n, w in want.items():
        assert np.allclose(got[n].numpy(), w, rtol=1e-11, atol=1e-13), n
    assert np.allclose(got["g"].sum((0, 1)).numpy(), want["dA"], rtol=1e-11, atol=1e-13)


def test_sizes_bound_the_sums():
    d = ssm_inputs(2, 7, 2, 1, 4, 4, "f32", seed=5)
    got, size = r.scan(d), r.sizes(d)
    assert all(bool((got[n].abs() <= size[n] * (1 + 1e-12)).all()) for n in ("y", "H_T", "dq", "dk", "dv", "dH_0", "g"))
