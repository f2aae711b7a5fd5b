"""y of the bf16 scan is the fp32 result rounded once.

With S the sum of the absolute values of all that is added up in an element of
y (state terms, scores, the skip), the kernels' sums before the rounding are off
by at most 2^-16 S for operands in two bf16 parts (each part's rounding leaves
2^-8 of what it rounds) and 2^-16 S for the sums themselves and the decays (up
to 128 + 64 truncating adds of 2^-23 at most, 2^-15.4 in the worst case and a
square root of it in earnest).  Every y then lies within half a unit of bf16
of the float64 value, and 2^-15 S."""
import pytest
import scan_reference as ref

from layer_util import SSM_IN, SSM_OPT, ints, ssm_dev, ssm_inputs

pytestmark = pytest.mark.gpu


def half_unit(y):
    """Half the distance of neighbouring bf16 values at |y| (8 significant bits)."""
    import torch
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(1e-30))) - 8)


# B, T, N, G, K, V, lengths, decay, spike
CASES = [(2, 300, 4, 2, 64, 64, None, None, None), (1, 200, 3, 1, 64, 128, None, None, None),
         (2, 700, 4, 2, 80, 48, (700, 333), None, None), (1, 77, 2, 1, 33, 17, None, None, None),
         (4, 1281, 8, 8, 40, 56, None, None, None), (4, 1300, 8, 1, 64, 64, (1300, 64, 130, 1000), None, None),
         # a step that forgets everything, then small ones: differences of sums of 6e4 and of sums of a few
         (2, 300, 4, 2, 64, 64, None, -1.0, 6e4), (4, 1300, 8, 2, 64, 64, None, -1.0, 6e4),
         (2, 300, 4, 2, 32, 16, None, -1.0, 6e4)]


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("B,T,N,G,K,V,lengths,decay,spike", CASES)
def test_y_is_rounded_once(B, T, N, G, K, V, lengths, decay, spike, h0):
    import torch
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, "bf16", seed=T + K + V, h0=h0, decay=decay)
    d.pop("dy"), d.pop("dH_T")
    g = ssm_dev(d, "bf16")
    if spike is not None:
        g["dt"][:, 5::41] = spike
    r = m.ssm_scan(*(g[n] for n in SSM_IN), lengths=ints(lengths), **{n: g[n] for n in SSM_OPT})
    want, size = ref.scan(g, lengths)["y"], ref.sizes(g, lengths)["y"]
    err = (r["y"].double() - want).abs() - half_unit(want)
    assert bool((err <= 2.0 ** -15 * size).all()), float((err / size.clamp_min(1e-30)).max() * 2 ** 15)
