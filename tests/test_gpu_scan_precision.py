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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,N,G,K,V", [(2, 200, 2, 1, 32, 32), (4, 1200, 8, 2, 64, 64)])
def test_log_decays_beyond_the_fp32_range(B, T, N, G, K, V, dtype):
    """Steps so long that D A leaves the fp32 range (D k does not) forget
    everything before them; what they put into the state decays by the small
    steps after them, 1e6 x 2e-9 each."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, dtype, seed=5, decay=-1e6)
    d.pop("dy"), d.pop("dH_T")
    g = ssm_dev(d, dtype)
    g["dt_bias"] -= 20.0
    g["dt"][:, 3::97] = 1e34
    r = m.ssm_scan(*(g[n] for n in SSM_IN), **{n: g[n] for n in SSM_OPT})
    want = ref.scan(g)
    assert bool(want["y"].abs().max() < 1e38)
    tol = 4e-3 if dtype == "bf16" else 1e-5
    for t0 in range(3, T, 97):  # each step's reign on its own: the first steps after it, while its state lasts
        got, w = r["y"][:, t0:t0 + 8].double(), want["y"][:, t0:t0 + 8]
        assert float((got - w).norm() / w.norm()) <= tol, t0
    got, w = r["H_T"].double(), want["H_T"]
    assert bool(got.isfinite().all()) and float((got - w).norm() / w.norm()) <= 1e-5
