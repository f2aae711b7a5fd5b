"""A value of v that is not finite reaches its own column of its own head, from
its own step on: no step before, on any path, at any place in a chunk, tile or
segment.  Steps before it keep their values (to the rounding of y: their sums
may be formed in another order)."""
import pytest

from layer_util import SSM_IN, SSM_OPT, ints, ssm_dev, ssm_inputs

pytestmark = pytest.mark.gpu


def unit(y, dtype):
    """The distance of neighbouring values of the type at |y|."""
    import torch
    bits = 7 if dtype == "bf16" else 23
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(1e-30))) - bits)


# B, T, N, G, K, V, dtype, lengths, columns that the rows are moved by
CASES = [(2, 200, 2, 1, 32, 32, "bf16", None, 0), (2, 200, 4, 2, 80, 48, "bf16", (200, 131), 0),
         (2, 150, 2, 1, 33, 17, "bf16", None, 0), (1, 200, 3, 1, 64, 128, "bf16", None, 3),
         (1, 130, 1, 1, 5, 100, "bf16", None, 0), (4, 1200, 8, 2, 64, 64, "bf16", (1200, 700, 1, 129), 0),
         (4, 1290, 8, 8, 40, 56, "bf16", None, 0), (3, 1100, 8, 4, 48, 96, "bf16", None, 0),
         (2, 150, 2, 1, 33, 17, "f32", None, 0), (2, 200, 4, 2, 64, 64, "f32", (200, 77), 0)]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("B,T,N,G,K,V,dtype,lengths,off", CASES)
def test_v_reaches_no_earlier_step(B, T, N, G, K, V, dtype, lengths, off, bad):
    import torch
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, dtype, seed=V)
    d.pop("dy"), d.pop("dH_T")
    base = ssm_dev(d, dtype)

    def run(v):
        g = dict(base, v=v)
        if off:
            wide = torch.zeros((B, T, N * V + 2 * off), device="cuda", dtype=v.dtype)
            wide[..., off:-off] = v.flatten(2)
            g["v"] = wide[..., off:-off].unflatten(-1, (N, V))
        r = m.ssm_scan(*(g[n] for n in SSM_IN), lengths=ints(lengths), **{n: g[n] for n in SSM_OPT})
        assert m.sync_status(r["workspace"]) == (m.M2RNN_OK, 0)
        return r["y"]

    clean = run(base["v"])
    assert torch.isfinite(clean).all()
    places = [(0, 0, 0), (0, 77, V - 1), (0, 63, 0), (0, 64, V // 2), (0, min(T, 129) - 1, 1 % V)]
    if T > 1000:
        places += [(0, t, t % V) for t in (127, 128, 640, 1001, T - 1 if lengths is None else lengths[0] - 1)]
    for b, t, c in places:
        for n in {0, N - 1}:
            v = base["v"].clone()
            v[b, t, n, c] = bad
            y = run(v)
            hit = torch.zeros_like(y, dtype=torch.bool)
            end = T if lengths is None else lengths[b]
            hit[b, t:end, n, c] = True
            assert torch.equal(~torch.isfinite(y), hit), (b, t, n, c)
            near = (y - clean).abs().float() <= unit(clean.float(), dtype) * (1 if dtype == "bf16" else 64)
            assert bool(near[~hit].all()), (b, t, n, c)
            other = torch.ones_like(hit)
            other[b, :, n, c] = False
            assert torch.equal(y[other], clean[other])
    v = base["v"].clone()  # a whole step, and another value later
    v[0, 70] = bad
    v[0, 90, 0, 0] = float("nan")
    y = run(v)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[0, 70:T if lengths is None else lengths[0]] = True
    assert torch.equal(~torch.isfinite(y), hit)
