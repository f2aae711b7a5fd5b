"""The scan at sizes where a block walks several chunks of a sequence: many
heads and sequences, so that a segment has more than one chunk (or is all of
the sequence), ragged lengths that end inside a segment and leave whole
segments empty, and both hand-ons of states between segments.

Tolerances (relative Frobenius) as in test_gpu_layer.py: bf16 y one rounding
to 8 bits and operands near it, 4e-3; fp32 results 1e-5; ddt and the sums over
all steps, which cancel, 1e-4."""
import pytest
import scan_reference as ref

from layer_util import SSM_IN, SSM_OPT, ints, ssm_dev, ssm_inputs

pytestmark = pytest.mark.gpu

TOL = {"bf16": 4e-3, "f32": 1e-5}
TOL_GRAD, TOL_STEP = 1e-5, 1e-4


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def spoil(g, lengths):
    """NaN behind each sequence's end: it must not be read."""
    if lengths is not None:
        for n in ("q", "k", "v", "dt", "dy"):
            for b, t in enumerate(lengths):
                g[n][b, t:] = float("nan")


def args(g):
    return [g[n] for n in SSM_IN], {n: g[n] for n in SSM_OPT}


def unspoiled(d, dtype):
    """The reference's inputs: on the GPU, in the values that the kernels get."""
    return ssm_dev(d, dtype)


def off_boundaries(g, off):
    """q, k, v, dt as column slices `off` elements into one wider tensor."""
    import torch
    B, T = g["v"].shape[:2]
    names = ("v", "k", "q", "dt")
    width = sum(g[n][0, 0].numel() for n in names)
    wide = torch.full((B, T, width + 2 * off), float("nan"), device="cuda", dtype=g["v"].dtype)
    at, s = off, dict(g)
    for n in names:
        w = g[n][0, 0].numel()
        wide[..., at:at + w] = g[n].flatten(2) if g[n].dim() == 4 else g[n]
        s[n] = wide[..., at:at + w]
        if g[n].dim() == 4:
            s[n] = s[n].unflatten(-1, g[n].shape[2:])
        at += w
    return s


RAGGED = (700, 0, 1, 64, 65, 333, 449, 640)
# B, T, N, G, K, V, dtype, lengths, columns that the rows are moved by
FORWARD = [(8, 700, 16, 1, 64, 32, "bf16", RAGGED, 0), (8, 700, 16, 4, 128, 128, "bf16", RAGGED, 0),
           (8, 700, 16, 2, 80, 48, "bf16", RAGGED, 0), (8, 700, 16, 16, 16, 16, "bf16", None, 0),
           (8, 700, 16, 1, 24, 100, "bf16", None, 0), (8, 700, 16, 8, 128, 16, "bf16", RAGGED, 0),
           (8, 700, 16, 8, 100, 20, "bf16", RAGGED, 0),
           # wide enough for tiles of 128 steps, but rows that only the walks of single chunks can take
           (8, 700, 16, 2, 64, 64, "bf16", RAGGED, 3), (8, 705, 16, 2, 44, 60, "bf16", RAGGED, 0),
           # tiles, several of them to a segment, and one segment per sequence
           (8, 1100, 16, 2, 64, 64, "bf16", (1100, 0, 1, 128, 129, 500, 999, 640), 0),
           (20, 400, 16, 4, 64, 64, "bf16", (400, 0, 1, 256, 257) * 4, 0),
           (2, 1300, 4, 2, 48, 40, "f32", (1300, 640), 0), (1, 2100, 2, 1, 64, 64, "f32", None, 0)]


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("B,T,N,G,K,V,dtype,lengths,off", FORWARD)
def test_forward_over_many_chunks(B, T, N, G, K, V, dtype, lengths, off, h0):
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, dtype, seed=T + K + V, h0=h0)
    d.pop("dy"), d.pop("dH_T")
    want = ref.scan(unspoiled(d, dtype), lengths)
    g = ssm_dev(dict(d, dy=None), dtype)
    if lengths is not None:
        for n in ("q", "k", "v", "dt"):
            for b, t in enumerate(lengths):
                g[n][b, t:] = float("nan")
    if off:
        g = off_boundaries(g, off)
    a, kw = args(g)
    r = m.ssm_scan(*a, lengths=ints(lengths), **kw)
    assert m.sync_status(r["workspace"]) == (m.M2RNN_OK, 0)
    assert rel(r["y"], want["y"]) <= TOL[dtype]
    assert rel(r["H_T"], want["H_T"]) <= 1e-5
    for b, t in enumerate(lengths or ()):  # behind the end, and each sequence on its own
        assert not r["y"][b, t:].any()
        assert not t or rel(r["y"][b, :t], want["y"][b, :t]) <= TOL[dtype]
        if want["H_T"][b].any():
            assert rel(r["H_T"][b], want["H_T"][b]) <= 1e-5


# Several chunks to a segment and several segments; then one segment per sequence.
BACKWARD = [(4, 1500, 8, 2, 64, 64, "bf16", (1500, 0, 130, 1000), 0), (4, 700, 8, 1, 128, 128, "bf16", (700, 1, 64, 500), 0),
            (8, 300, 32, 8, 64, 64, "bf16", (300, 0, 1, 64, 65, 192, 250, 299), 0), (8, 260, 24, 24, 80, 48, "bf16", None, 0),
            (4, 600, 16, 1, 64, 16, "bf16", (600, 7, 64, 321), 0), (8, 300, 32, 4, 32, 32, "bf16", None, 0),
            (4, 500, 8, 2, 33, 100, "bf16", (500, 3, 64, 129), 0), (4, 700, 8, 2, 64, 64, "bf16", None, 3),
            (2, 700, 4, 2, 48, 40, "f32", (700, 330), 0)]


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("B,T,N,G,K,V,dtype,lengths,off", BACKWARD)
def test_backward_over_many_chunks(B, T, N, G, K, V, dtype, lengths, off, h0):
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, dtype, seed=T + K + V, h0=h0)
    want = ref.scan(unspoiled(d, dtype), lengths)
    g = ssm_dev(d, dtype)
    spoil(g, lengths)
    if off:
        g = off_boundaries(g, off)
    a, kw = args(g)
    r = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], lengths=ints(lengths), want_dH0=True, **kw)
    for n in ("dq", "dk", "dv", "dw_r", "dH_0"):
        assert rel(r[n], want[n]) <= TOL_GRAD, n
    for n in ("ddt", "dA", "ddt_bias"):
        assert rel(r[n], want[n]) <= TOL_STEP, n
    for b, t in enumerate(lengths or ()):
        for n in ("dq", "dk", "dv", "ddt"):
            assert not r[n][b, t:].any(), n
            assert not t or rel(r[n][b, :t], want[n][b, :t]) <= (TOL_STEP if n == "ddt" else TOL_GRAD), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [0.0, -1e-3, -300.0, 0.5])
def test_gradients_of_the_decays_at_extreme_decays(dtype, decay):
    """ddt, dA, ddt_bias: each a sum of terms of both signs, compared at the
    size of the terms.  fp32 sums of up to 64 + 64 terms are off by 128 x 2^-24
    of it at most, the decays (fast exponentials of at most a few hundred, where
    they count a few) and operands in three parts by a few 2^-24: 2^-16."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(2, 150, 2, 1, 32, 32, dtype, seed=7, decay=decay)
    g = ssm_dev(d, dtype)
    a, kw = args(g)
    r = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], **kw)
    want, size = ref.scan(g), ref.sizes(g)
    D = abs(decay) * size["g"]  # |A| D g; times 1 / D below
    step = ref.torch.logaddexp(g["dt"].double() + g["dt_bias"], ref.torch.zeros_like(g["dt"], dtype=ref.torch.float64))
    sg = ref.torch.sigmoid(g["dt"].double() + g["dt_bias"])
    # |ddt| <= (|k R v| + |A g|) sg with every sum of absolute values; size's ddt has A's sign, so both are put together.
    terms = (size["ddt"] / sg - d["A"][0] * size["g"] / step) * sg + D / step * sg
    err = (r["ddt"].double() - want["ddt"]).abs()
    assert bool((err <= 2.0 ** -16 * terms).all()), float((err / terms).max())
    for n, s in (("dA", size["g"].sum((0, 1))), ("ddt_bias", terms.sum((0, 1)))):
        err = (r[n].double() - want[n]).abs()
        assert bool((err <= 2.0 ** -16 * s).all()), (n, float((err / s).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dA_is_not_lost_to_cancellation(dtype):
    """dA is the sum of D_t g_t over all steps, of both signs.  Every term's own
    error is a few times 2^-24 of it; errors of a sum of n of them stay below
    2^-21 of the terms' root sum of squares times a few, here 16."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(2, 500, 6, 2, 64, 48, dtype, seed=19)
    g = ssm_dev(d, dtype)
    a, kw = args(g)
    r = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], want_dH0=True, **kw)
    want = ref.scan(g)
    size = want["g"].square().sum((0, 1)).sqrt()
    err = (r["dA"].double() - want["dA"]).abs()
    assert bool((err <= 16 * 2.0 ** -21 * size).all()), float((err / size).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dA_needs_its_running_sums_in_two_floats(dtype):
    """At 6000 steps a head.  A term D_t g_t is off by the roundings of the row
    products in it, 64 of 2^-24 that add up as their square root: 2^-21 of its
    size; independent over the terms, so dA is off by 2^-21 of the terms' root
    sum of squares, in the mean over the heads; 4 of it are allowed.  (Running
    sums over a chunk in single floats leave 6 to 8.)"""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(4, 1500, 8, 8, 64, 64, dtype, seed=3, h0=False)
    g = ssm_dev(d, dtype)
    a, kw = args(g)
    r = m.ssm_scan_backward(*a, g["dy"], **kw)
    want = ref.scan(g)
    off = (r["dA"].double() - want["dA"]) / want["g"].square().sum((0, 1)).sqrt()
    assert float(off.square().mean().sqrt()) <= 4 * 2.0 ** -21, float(off.square().mean().sqrt()) * 2 ** 21


def test_nan_stays_behind_its_step_in_tiles():
    """A NaN in q touches its own step, one in k or dt the steps from its own
    on; other heads and sequences, and the steps before, stay as they were."""
    import torch
    from matrix_state_non_gb300 import binding as m
    T = 1300
    d = ssm_inputs(4, T, 8, 8, 64, 64, "bf16", seed=71)
    d.pop("dy"), d.pop("dH_T")
    base = ssm_dev(d, "bf16")
    a, kw = args(base)
    y0 = m.ssm_scan(*a, **kw)["y"]
    for n, later in (("q", False), ("k", True), ("dt", True)):
        g = {i: None if x is None else x.clone() for i, x in base.items()}
        g[n][1, 333, 1] = float("nan")
        a, kw = args(g)
        y = m.ssm_scan(*a, **kw)["y"]
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[1, 333:(T if later else 334), 1] = True
        assert torch.equal(torch.isnan(y), bad), n
        assert torch.equal(y[~bad], y0[~bad]), n


@pytest.mark.parametrize("B,T,N,G,K,V,dtype", [(2, 200, 4, 2, 80, 48, "bf16"), (4, 1200, 8, 1, 64, 64, "bf16"),
                                              (2, 200, 4, 2, 48, 40, "f32")])
def test_calls_in_a_graph_and_on_two_streams(B, T, N, G, K, V, dtype):
    """A captured forward, backward and token step replayed on other inputs, and
    two forwards at once on two streams, give the bits of plain calls."""
    import torch
    from matrix_state_non_gb300 import binding as m
    sets = [ssm_dev(ssm_inputs(B, T, N, G, K, V, dtype, seed=s), dtype) for s in (1, 2)]
    buf = {n: None if x is None else x.clone() for n, x in sets[0].items()}

    def run(g):
        a, kw = args(g)
        f = m.ssm_scan(*a, **kw)
        H = f["H_T"].clone()
        opts = dict(dt_bias=kw["dt_bias"], w_r=kw["w_r"])
        y = m.ssm_step(H, *(g[n][:, 0] for n in ("q", "k", "v", "dt")), g["A"], **opts)
        b = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], want_dH0=True, **kw)
        b.pop("workspace")
        return dict(b, y=f["y"], H_T=f["H_T"], H=H, step=y)

    want = [run(g) for g in sets]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(buf)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run(buf)
    for g, w in zip(sets[::-1], want[::-1]):
        for n, x in g.items():
            if x is not None:
                buf[n].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for n in w:
            assert torch.equal(out[n], w[n]), n
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for g, st in zip(sets, streams):
            a, kw = args(g)
            got.append(m.ssm_scan(*a, stream=st, **kw))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert torch.equal(r["y"], want[i % 2]["y"]) and torch.equal(r["H_T"], want[i % 2]["H_T"])
