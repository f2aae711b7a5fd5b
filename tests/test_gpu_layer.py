"""GPU parity of the hybrid layer's operators (short causal convolution,
selective state space scan, gradient clipping) with the float64 oracle.

Tolerances (relative Frobenius), from the arithmetic:
 - bf16 outputs: one rounding to 8 bits (at most 2^-9 of a value, 1.7e-3 in the
   mean) and, in the scan, operands of the readout rounded the same way: 4e-3;
 - fp32 outputs: every product exact or split to 24 bits, sums of at most a few
   hundred fp32 roundings of 6e-8: 1e-5;
 - ddt and the sums dA, ddt_bias: differences of such sums over up to 64 steps,
   which cancel by up to about 30: 1e-4.
"""
import numpy as np
import pytest

from layer_util import SSM_IN, SSM_OPT, conv_inputs, dev, host, ints, round_to, ssm_dev, ssm_inputs
from oracle import layer_oracle as o
from parity_util import rel_fro

pytestmark = pytest.mark.gpu

TOL = {"bf16": 4e-3, "f32": 1e-5}
TOL_GRAD, TOL_STEP = 1e-5, 1e-4


def close(got, ref, tol, label):
    got = host(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), label
    r = rel_fro(got, ref)
    assert r <= tol, (label, r)


# ---------------------------------------------------------------------------
# Convolution
# ---------------------------------------------------------------------------
# B, T, C, W, dtype, lengths, x0, bias, wide (extra columns of the projection x is a slice of)
CONV = [(1, 1, 8, 4, "bf16", None, False, True, 0), (2, 37, 64, 4, "bf16", None, True, True, 8),
        (3, 70, 24, 3, "bf16", (70, 1, 0), True, True, 5), (2, 130, 33, 4, "bf16", (2, 129), False, True, 0),
        (2, 65, 40, 2, "f32", (64, 65), True, False, 4), (4, 19, 13, 4, "f32", (0, 1, 3, 19), True, True, 1),
        (1, 300, 136, 4, "f32", None, False, True, 0), (1, 5, 7, 1, "f32", None, False, True, 0),
        (2, 9, 16, 8, "bf16", (1, 9), True, True, 0), (1, 2, 4, 4, "f32", None, True, False, 0),
        (2, 1025, 256, 4, "bf16", (1025, 700), True, True, 16)]


def _conv_dev(d, dtype, wide):
    import torch
    g = {n: dev(a, "f32" if n in ("dy", "dx_T") else dtype) for n, a in d.items()}
    if wide:
        full = torch.full(g["x"].shape[:2] + (g["x"].shape[2] + wide,), float("nan"), device="cuda", dtype=g["x"].dtype)
        full[..., :-wide] = g["x"]
        g["x"] = full[..., :-wide]
    return g


def _spoil(x, lengths):
    """NaN behind each sequence's end: it must not be read."""
    if lengths is not None:
        for b, n in enumerate(lengths):
            x[b, n:] = float("nan")


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("B,T,C,W,dtype,lengths,x0,bias,wide", CONV)
def test_causal_conv(B, T, C, W, dtype, lengths, x0, bias, wide, silu):
    from matrix_state_non_gb300 import binding as m
    d = conv_inputs(B, T, C, W, dtype, seed=T + C, x0=x0, bias=bias)
    g = _conv_dev(d, dtype, wide)
    _spoil(g["x"], lengths)
    r = m.causal_conv(g["x"], g["w"], g["bias"], x0=g["x0"], lengths=ints(lengths), silu=silu, want_state=True)
    y, x_T = o.causal_conv(d["x"], d["w"], d["bias"], d["x0"], lengths, silu)
    close(r["y"], y, TOL[dtype], "y")
    assert np.array_equal(host(r["x_T"]), x_T)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("B,T,C,W,dtype,lengths,x0,bias,wide", CONV)
def test_causal_conv_backward(B, T, C, W, dtype, lengths, x0, bias, wide, silu):
    from matrix_state_non_gb300 import binding as m
    d = conv_inputs(B, T, C, W, dtype, seed=T + C, x0=x0, bias=bias)
    g = _conv_dev(d, dtype, wide)
    _spoil(g["x"], lengths)
    _spoil(g["dy"], lengths)
    r = m.causal_conv_backward(g["x"], g["w"], g["bias"], g["dy"], x0=g["x0"], dx_T=g["dx_T"], lengths=ints(lengths),
                               silu=silu, want_dx0=True)
    ref = o.causal_conv_backward(d["x"], d["w"], d["bias"], d["dy"], d["x0"], d["dx_T"], lengths, silu)
    for n in ("dx", "dw", "dx0") + (("db",) if bias else ()):
        close(r[n], ref[n], TOL_GRAD, n)


def test_causal_conv_gradient_is_a_difference():
    """The kernel's gradient along a random direction against the oracle's
    forward: (L(x + h e) - L(x - h e)) / 2h in 64 bits, off by O(h^2)."""
    from matrix_state_non_gb300 import binding as m
    d = conv_inputs(2, 40, 12, 4, "f32", seed=3, x0=True)
    g = _conv_dev(d, "f32", 0)
    r = m.causal_conv_backward(g["x"], g["w"], g["bias"], g["dy"], x0=g["x0"], dx_T=g["dx_T"], want_dx0=True)
    rng, h = np.random.default_rng(4), 1e-5
    for n, gn in dict(x="dx", w="dw", bias="db", x0="dx0").items():
        e = rng.normal(size=d[n].shape)

        def loss(s):
            a = dict(d, **{n: d[n] + s * e})
            y, x_T = o.causal_conv(a["x"], a["w"], a["bias"], a["x0"])
            return (y * d["dy"]).sum() + (x_T * d["dx_T"]).sum()

        want = (loss(h) - loss(-h)) / (2 * h)
        got = host(r[gn])
        # fp32 gradients: each entry off by 1e-6 of the largest at most, in random directions
        assert abs((got * e).sum() - want) <= 1e-5 * np.linalg.norm(got) * np.linalg.norm(e)


@pytest.mark.parametrize("B,C,W,dtype,wide", [(1, 8, 4, "bf16", 0), (3, 33, 4, "bf16", 7), (5, 64, 2, "f32", 0),
                                             (2, 100, 3, "f32", 4), (32, 136, 4, "bf16", 8), (2, 5, 1, "f32", 0)])
def test_causal_conv_step_continues_the_prompt(B, C, W, dtype, wide):
    from matrix_state_non_gb300 import binding as m
    T = 9
    d = conv_inputs(B, T, C, W, dtype, seed=B + C, x0=True)
    g = _conv_dev(d, dtype, wide)
    state = m.causal_conv(g["x"][:, :5].contiguous(), g["w"], g["bias"], x0=g["x0"], want_state=True)["x_T"]
    y, x_T = o.causal_conv(d["x"], d["w"], d["bias"], d["x0"])
    for t in range(5, T):
        close(m.causal_conv_step(state, g["x"][:, t], g["w"], g["bias"]), y[:, t], TOL[dtype], t)
    assert np.array_equal(host(state), x_T)


# ---------------------------------------------------------------------------
# Scan
# ---------------------------------------------------------------------------
# B, T, N, G, K, V, dtype, lengths
SSM = [(1, 1, 1, 1, 16, 16, "bf16", None), (2, 63, 2, 2, 64, 64, "bf16", None), (1, 64, 2, 1, 64, 64, "bf16", None),
       (2, 65, 4, 2, 32, 64, "bf16", (65, 64)), (3, 130, 2, 1, 128, 64, "bf16", (130, 1, 0)),
       (1, 200, 3, 1, 64, 128, "bf16", None), (1, 129, 1, 1, 128, 128, "bf16", None),
       (2, 100, 2, 2, 80, 48, "bf16", (31, 100)), (1, 77, 2, 1, 33, 17, "bf16", None),
       (2, 70, 2, 1, 16, 16, "bf16", (2, 69)), (1, 90, 2, 2, 5, 100, "bf16", None), (1, 33, 1, 1, 1, 1, "bf16", None),
       (1, 1, 2, 1, 8, 8, "f32", None), (2, 33, 2, 1, 16, 24, "f32", (33, 5)), (1, 100, 3, 3, 33, 17, "f32", None),
       (2, 64, 2, 2, 64, 64, "f32", (0, 64)), (1, 40, 1, 1, 128, 128, "f32", None), (1, 31, 1, 1, 1, 3, "f32", None),
       (2, 130, 2, 1, 64, 16, "bf16", (130, 7)), (1, 100, 4, 2, 100, 12, "bf16", None),
       (1, 700, 2, 1, 128, 16, "bf16", None), (1, 66, 1, 1, 40, 1, "bf16", None)]


def _scan_args(g):
    return [g[n] for n in SSM_IN], {n: g[n] for n in SSM_OPT}


def _spoil_ssm(g, lengths):
    for n in ("q", "k", "v", "dt", "dy"):
        _spoil(g[n], lengths)


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("B,T,N,G,K,V,dtype,lengths", SSM)
def test_ssm_scan(B, T, N, G, K, V, dtype, lengths, h0):
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, dtype, seed=T + K + V, h0=h0)
    g = ssm_dev(d, dtype)
    _spoil_ssm(g, lengths)
    a, kw = _scan_args(g)
    r = m.ssm_scan(*a, lengths=ints(lengths), **kw)
    ra, rkw = _scan_args(d)
    y, H = o.ssm_scan(*ra, lengths=lengths, **rkw)
    close(r["y"], y, TOL[dtype], "y")
    close(r["H_T"], H, 1e-5, "H_T")


# Enough heads and steps for the tcgen05 outputs (tiles of 128 steps).
TILES = [(4, 1200, 8, 1, 64, 64, None), (5, 1300, 8, 2, 64, 64, (1300, 0, 1, 129, 640)), (4, 1281, 8, 8, 40, 56, None),
         (3, 1100, 8, 4, 48, 96, (1100, 64, 1000)), (1, 5000, 8, 1, 64, 40, None), (40, 128, 8, 1, 64, 64, None)]


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("B,T,N,G,K,V,lengths", TILES)
def test_ssm_scan_in_tiles(B, T, N, G, K, V, lengths, h0):
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, "bf16", seed=T + K + V, h0=h0)
    g = ssm_dev(d, "bf16")
    _spoil_ssm(g, lengths)
    a, kw = _scan_args(g)
    if not h0:
        kw["w_r"] = None
    r = m.ssm_scan(*a, lengths=ints(lengths), **kw)
    assert m.sync_status(r["workspace"]) == (m.M2RNN_OK, 0)
    ra, rkw = _scan_args(d)
    if not h0:
        rkw["w_r"] = None
    y, H = o.ssm_scan(*ra, lengths=lengths, **rkw)
    close(r["y"], y, TOL["bf16"], "y")
    close(r["H_T"], H, 1e-5, "H_T")


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("B,T,N,G,K,V,dtype,lengths", SSM)
def test_ssm_scan_backward(B, T, N, G, K, V, dtype, lengths, h0):
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(B, T, N, G, K, V, dtype, seed=T + K + V, h0=h0)
    g = ssm_dev(d, dtype)
    _spoil_ssm(g, lengths)
    a, kw = _scan_args(g)
    r = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], lengths=ints(lengths), want_dH0=True, **kw)
    ra, rkw = _scan_args(d)
    ref = o.ssm_scan_backward(*ra, d["dy"], dH_T=d["dH_T"], lengths=lengths, **rkw)
    for n in ("dq", "dk", "dv", "dw_r", "dH_0"):
        close(r[n], ref[n], TOL_GRAD, n)
    for n in ("ddt", "dA", "ddt_bias"):
        close(r[n], ref[n], TOL_STEP, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_gradient_is_a_difference(dtype):
    """The kernel's gradient along a random direction against the oracle's
    forward in 64 bits: (L(x + h e) - L(x - h e)) / 2h, off by O(h^2)."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(2, 70, 4, 2, 16, 32, dtype, seed=61)
    g = ssm_dev(d, dtype)
    a, kw = _scan_args(g)
    r = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], want_dH0=True, **kw)
    rng, h = np.random.default_rng(62), 1e-5
    for n in SSM_IN + SSM_OPT:
        e = rng.normal(size=d[n].shape)

        def loss(s):
            p = dict(d, **{n: d[n] + s * e})
            y, H = o.ssm_scan(*(p[i] for i in SSM_IN), **{i: p[i] for i in SSM_OPT})
            return (y * d["dy"]).sum() + (H * d["dH_T"]).sum()

        want, got = (loss(h) - loss(-h)) / (2 * h), host(r["d" + n])
        tol = TOL_STEP if n in ("dt", "A", "dt_bias") else TOL_GRAD
        assert abs((got * e).sum() - want) <= tol * np.linalg.norm(got) * np.linalg.norm(e), n


def test_ssm_nan_stays_behind_its_step():
    """A NaN in q touches its own step, one in k or dt the steps from its own
    on; earlier steps and other heads and sequences stay as they were."""
    import torch
    from matrix_state_non_gb300 import binding as m
    for dtype in ("bf16", "f32"):
        d = ssm_inputs(2, 150, 2, 2, 32, 32, dtype, seed=71)
        base = ssm_dev(d, dtype)
        a, kw = _scan_args(base)
        ref = m.ssm_scan(*a, **kw)["y"]
        for n, later in (("q", False), ("k", True), ("dt", True)):
            g = {i: None if x is None else x.clone() for i, x in base.items()}
            g[n][1, 77, 1] = float("nan")
            a, kw = _scan_args(g)
            y = m.ssm_scan(*a, **kw)["y"]
            bad = torch.zeros_like(y, dtype=torch.bool)
            bad[1, 77:(150 if later else 78), 1] = True
            assert torch.equal(torch.isnan(y), bad), (dtype, n)
            assert torch.equal(y[~bad], ref[~bad]), (dtype, n)


def test_offsets_beyond_32_bits():
    """Rows 2^20 elements apart: the last tokens lie beyond 2^32 elements."""
    import torch
    from matrix_state_non_gb300 import binding as m
    T, wide = 4200, 1 << 20
    d = ssm_inputs(1, T, 1, 1, 16, 16, "bf16", seed=81, h0=False)
    g = ssm_dev(d, "bf16")
    big = torch.empty((1, T, wide), dtype=torch.bfloat16, device="cuda")
    s, at = {}, wide - 64
    for n, w in (("v", 16), ("k", 16), ("q", 16), ("dt", 1)):
        big[..., at:at + w] = g[n].flatten(2)
        s[n] = big[..., at:at + w].unflatten(-1, g[n].shape[2:])
        at += w
    want, got = m.ssm_scan(*(g[n] for n in SSM_IN)), m.ssm_scan(s["q"], s["k"], s["v"], s["dt"], g["A"])
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["H_T"], want["H_T"])
    a = m.ssm_scan_backward(*(g[n] for n in SSM_IN), g["dy"])
    b = m.ssm_scan_backward(s["q"], s["k"], s["v"], s["dt"], g["A"], g["dy"])
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dv", "ddt", "dA"))
    c = conv_inputs(1, T, 16, 4, "bf16", seed=82)
    w, bias, dy = dev(c["w"], "bf16"), dev(c["bias"], "bf16"), dev(c["dy"])
    x = big[..., wide - 64:wide - 48]
    assert torch.equal(m.causal_conv(x, w, bias)["y"], m.causal_conv(x.contiguous(), w, bias)["y"])
    p, q = m.causal_conv_backward(x, w, bias, dy), m.causal_conv_backward(x.contiguous(), w, bias, dy)
    assert all(torch.equal(p[n], q[n]) for n in p)
    del big
    # More than 2^31 elements in one dense tensor.
    x = torch.empty((1, 70000, 32768), dtype=torch.bfloat16, device="cuda")
    x[:, :100] = 1.0
    x[:, -100:] = torch.randn((1, 100, 32768), device="cuda")
    w = torch.randn((32768, 4), device="cuda").bfloat16()
    y = m.causal_conv(x, w, silu=False)["y"]
    assert torch.equal(y[:, -90:], m.causal_conv(x[:, -100:].contiguous(), w, silu=False)["y"][:, 10:])


def test_torch_helpers_refuse():
    import torch
    from matrix_state_non_gb300 import binding as m
    g = ssm_dev(ssm_inputs(2, 8, 2, 1, 16, 16, "bf16", seed=91), "bf16")
    a, kw = _scan_args(g)
    with pytest.raises(ValueError, match="k: expected"):
        m.ssm_scan(a[0], a[1].float(), *a[2:])
    with pytest.raises(ValueError, match="A: expected"):
        m.ssm_scan(*a[:4], a[4].bfloat16())
    with pytest.raises(ValueError, match="dense"):
        m.ssm_scan(*a[:2], a[2].transpose(2, 3).contiguous().transpose(2, 3), *a[3:])
    with pytest.raises(ValueError, match="T rows apart"):
        m.ssm_scan(*a[:2], torch.cat([a[2], a[2]], 1)[:, :8], *a[3:])
    with pytest.raises(ValueError, match="contiguous"):
        m.ssm_scan(*a, H_0=g["H_0"].transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError, match="lengths"):
        m.ssm_scan(*a, lengths=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="unsupported"):
        m.ssm_scan(*(x.half() for x in a[:4]), a[4])
    with pytest.raises(m.M2RNNError, match="unsupported"):
        wide = torch.zeros((1, 2, 1, 130), dtype=torch.bfloat16, device="cuda")
        m.ssm_scan(wide, wide, wide, wide[..., 0], torch.zeros(1, device="cuda"))
    with pytest.raises(m.M2RNNError):
        m.grad_clip(m.grad_plan([a[4]]), -1.0)
    x = torch.zeros((1, 4, 8), device="cuda")
    with pytest.raises(m.M2RNNError, match="invalid"):
        m.causal_conv(x, torch.zeros((8, 4), device="cuda"), out=dict(y=x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [0.0, -1e-3, -300.0, 0.5])
def test_ssm_scan_extreme_decays(dtype, decay):
    """No decay, almost none, states forgotten within a step, growing states."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(1, 150, 2, 1, 32, 32, dtype, seed=7, decay=decay)
    g = ssm_dev(d, dtype)
    a, kw = _scan_args(g)
    ra, rkw = _scan_args(d)
    r = m.ssm_scan(*a, **kw)
    y, H = o.ssm_scan(*ra, **rkw)
    close(r["y"], y, TOL[dtype], "y")
    close(r["H_T"], H, 1e-5, "H_T")
    r = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], want_dH0=True, **kw)
    ref = o.ssm_scan_backward(*ra, d["dy"], dH_T=d["dH_T"], **rkw)
    for n in ("dq", "dk", "dv", "dw_r"):
        close(r[n], ref[n], TOL_GRAD, n)
    if np.linalg.norm(ref["dH_0"]) > 1e-30:
        close(r["dH_0"], ref["dH_0"], TOL_GRAD, "dH_0")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_scan_large_and_small_steps(dtype):
    """dt far on both sides of softplus: steps of 60 and steps of e^-60."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(1, 100, 2, 2, 16, 32, dtype, seed=11, decay=-0.05)
    d["dt"][:, ::7] = 60.0
    d["dt"][:, 3::7] = -60.0
    g = ssm_dev(d, dtype)
    a, kw = _scan_args(g)
    ra, rkw = _scan_args(d)
    y, H = o.ssm_scan(*ra, **rkw)
    r = m.ssm_scan(*a, **kw)
    close(r["y"], y, TOL[dtype], "y")
    close(r["H_T"], H, 1e-5, "H_T")


@pytest.mark.parametrize("decay", [0.0, -1e-3, -300.0])
def test_ssm_scan_in_tiles_extreme_decays(decay):
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(4, 1160, 8, 2, 64, 64, "bf16", seed=9, decay=decay)
    d["dt"][:, 5::41] = 60.0
    g = ssm_dev(d, "bf16")
    a, kw = _scan_args(g)
    ra, rkw = _scan_args(d)
    r = m.ssm_scan(*a, **kw)
    y, H = o.ssm_scan(*ra, **rkw)
    close(r["y"], y, TOL["bf16"], "y")
    close(r["H_T"], H, 1e-5, "H_T")
    assert m.sync_status(r["workspace"]) == (m.M2RNN_OK, 0)


def test_ssm_sums_over_all_steps_are_not_lost_to_cancellation():
    """dA and ddt_bias are sums of per-step gradients of both signs.  Every
    term's own error is a few times 2^-24 of it; errors of a sum of n of them
    stay below 2^-21 of the terms' root sum of squares times a few, here 16."""
    from matrix_state_non_gb300 import binding as m
    for dtype in ("bf16", "f32"):
        d = ssm_inputs(2, 500, 6, 2, 64, 48, dtype, seed=19)
        g = ssm_dev(d, dtype)
        a, kw = _scan_args(g)
        ra, rkw = _scan_args(d)
        r = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], want_dH0=True, **kw)
        ref = o.ssm_scan_backward(*ra, d["dy"], dH_T=d["dH_T"], **rkw)
        size = np.sqrt((ref["ddt"] ** 2).sum((0, 1)))
        err = np.abs(r["ddt_bias"].double().cpu().numpy() - ref["ddt_bias"])
        assert (err <= 16 * 2.0 ** -21 * size).all(), (dtype, err / size)


def test_ssm_scan_on_column_slices_another_stream_and_without_options():
    import torch
    from matrix_state_non_gb300 import binding as m
    B, T, N, G, K, V = 2, 90, 2, 1, 64, 64
    d = ssm_inputs(B, T, N, G, K, V, "bf16", seed=21)
    g = ssm_dev(d, "bf16")
    for off in (8, 3):  # 16-byte aligned rows, and not
        wide = torch.full((B, T, N * V + 2 * G * K + N + 2 * off), float("nan"), device="cuda", dtype=torch.bfloat16)
        at = off
        s = {}
        for n, w in (("v", N * V), ("k", G * K), ("q", G * K), ("dt", N)):
            wide[..., at:at + w] = g[n].flatten(2)
            s[n] = wide[..., at:at + w].unflatten(-1, g[n].shape[2:])
            at += w
        ref = m.ssm_scan(*(g[n] for n in SSM_IN))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        r = m.ssm_scan(s["q"], s["k"], s["v"], s["dt"], g["A"], stream=stream)
        gr = m.ssm_scan_backward(s["q"], s["k"], s["v"], s["dt"], g["A"], g["dy"], stream=stream)
        stream.synchronize()
        assert torch.equal(r["y"], ref["y"]) and torch.equal(r["H_T"], ref["H_T"])
        want = m.ssm_scan_backward(*(g[n] for n in SSM_IN), g["dy"])
        assert set(gr) == {"dq", "dk", "dv", "ddt", "dA", "workspace"}
        for n in ("dq", "dk", "dv", "ddt", "dA"):
            assert torch.equal(gr[n], want[n]), n
    y, H = o.ssm_scan(*(d[n] for n in SSM_IN))
    close(ref["y"], y, TOL["bf16"], "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_pieces_compose(dtype):
    """Two pieces, the state handed on in place, against one call; gradients
    handed back through dH_0 -> dH_T."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(2, 150, 2, 1, 64, 32, dtype, seed=31)
    g = ssm_dev(d, dtype)
    a, kw = _scan_args(g)
    whole = m.ssm_scan(*a, **kw)
    cut = {n: (g[n][:, :70].contiguous(), g[n][:, 70:].contiguous()) for n in ("q", "k", "v", "dt", "dy")}
    H = g["H_0"].clone()
    opts = dict(dt_bias=g["dt_bias"], w_r=g["w_r"])
    ys, starts = [], []
    for i in range(2):
        starts.append(H.clone())
        r = m.ssm_scan(*(cut[n][i] for n in ("q", "k", "v", "dt")), g["A"], H_0=H, out=dict(H_T=H), **opts)
        ys.append(host(r["y"]))
    ref_y, ref_H = host(whole["y"]), host(whole["H_T"])
    assert rel_fro(np.concatenate(ys, 1), ref_y) <= TOL[dtype] and rel_fro(host(H), ref_H) <= 1e-5
    grads = m.ssm_scan_backward(*a, g["dy"], dH_T=g["dH_T"], want_dH0=True, **kw)
    back = g["dH_T"]
    for i in (1, 0):
        r = m.ssm_scan_backward(*(cut[n][i] for n in ("q", "k", "v", "dt")), g["A"], cut["dy"][i], H_0=starts[i],
                                dH_T=back, want_dH0=True, **opts)
        back = r["dH_0"]
        sl = slice(0, 70) if i == 0 else slice(70, None)
        for n in ("dq", "dk", "dv"):
            assert rel_fro(host(r[n]), host(grads[n])[:, sl]) <= TOL_GRAD, n
    assert rel_fro(host(back), host(grads["dH_0"])) <= TOL_GRAD


@pytest.mark.parametrize("B,N,G,K,V,dtype", [(1, 1, 1, 64, 64, "bf16"), (4, 8, 1, 64, 64, "bf16"),
                                            (3, 4, 2, 128, 128, "bf16"), (2, 2, 2, 80, 48, "bf16"),
                                            (2, 3, 1, 33, 17, "bf16"), (1, 2, 1, 1, 1, "bf16"),
                                            (2, 2, 1, 16, 100, "f32"), (2, 4, 4, 5, 128, "f32"),
                                            (1, 2, 1, 128, 3, "f32")])
def test_ssm_step_continues_the_prompt(B, N, G, K, V, dtype):
    from matrix_state_non_gb300 import binding as m
    T, T0 = 40, 35
    d = ssm_inputs(B, T, N, G, K, V, dtype, seed=K + V)
    g = ssm_dev(d, dtype)
    opts = dict(dt_bias=g["dt_bias"], w_r=g["w_r"])
    H = m.ssm_scan(*(g[n][:, :T0].contiguous() for n in ("q", "k", "v", "dt")), g["A"], H_0=g["H_0"], **opts)["H_T"]
    ra, rkw = _scan_args(d)
    y, H_ref = o.ssm_scan(*ra, **rkw)
    for t in range(T0, T):
        close(m.ssm_step(H, *(g[n][:, t] for n in ("q", "k", "v", "dt")), g["A"], **opts), y[:, t], TOL[dtype], t)
    close(H, H_ref, 1e-5, "H")


def test_layer_is_deterministic():
    import torch
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(2, 300, 4, 1, 64, 64, "bf16", seed=41)
    g = ssm_dev(d, "bf16")
    a, kw = _scan_args(g)
    runs = [(m.ssm_scan(*a, **kw), m.ssm_scan_backward(*a, g["dy"], **kw)) for _ in range(2)]
    for x, y in zip(*runs):
        for n in x:
            assert n == "workspace" or torch.equal(x[n], y[n]), n
    c = _conv_dev(conv_inputs(2, 500, 72, 4, "bf16", seed=42), "bf16", 0)
    x, y = (m.causal_conv_backward(c["x"], c["w"], c["bias"], c["dy"]) for _ in range(2))
    for n in x:
        assert torch.equal(x[n], y[n]), n


def test_ssm_long_prompt():
    """4096 steps of four heads: the chunks' hand-on over a long sequence."""
    from matrix_state_non_gb300 import binding as m
    d = ssm_inputs(1, 4096, 4, 1, 64, 64, "bf16", seed=51)
    g = ssm_dev(d, "bf16")
    a, kw = _scan_args(g)
    r = m.ssm_scan(*a, **kw)
    y, H = o.ssm_scan(*(d[n] for n in SSM_IN), **{n: d[n] for n in SSM_OPT})
    close(r["y"], y, TOL["bf16"], "y")
    close(r["H_T"], H, 1e-5, "H_T")


# ---------------------------------------------------------------------------
# Clipping
# ---------------------------------------------------------------------------
def _grads(shapes, dtypes, seed, scale=1.0, odd=False):
    import torch
    r = np.random.default_rng(seed)
    ref, got = [], []
    for sh, dt in zip(shapes, dtypes):
        x = round_to(scale * r.normal(size=sh), dt)
        t = dev(x, dt)
        if odd:  # one element off a 16-byte boundary
            b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            b[1:] = t.flatten()
            t = b[1:].view(sh)
        ref.append(x)
        got.append(t)
    return ref, got


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("odd", [True, False])
@pytest.mark.parametrize("shapes,dtypes,max_norm", [
    ([(1,)], ["f32"], 1.0), ([(7,)], ["bf16"], 0.5), ([(16384,), (16385,), (3, 5)], ["f32", "bf16", "f32"], 1.0),
    ([(0,), (100, 100), (1,)], ["f32", "bf16", "bf16"], 2.0), ([(200000,), (40000,)], ["bf16", "f32"], 1e9),
    ([(5,)] * 70, ["f32", "bf16"] * 35, 1.0)])
def test_grad_clip(shapes, dtypes, max_norm, odd, in_place):
    import torch
    from matrix_state_non_gb300 import binding as m
    ref, got = _grads(shapes, dtypes, seed=len(shapes), odd=odd)
    outs = got if in_place else [torch.full_like(t, 7.0) for t in got]
    plan = m.grad_plan(got, None if in_place else outs)
    keep = [t.clone() for t in got]
    norm, clipped = o.clip(ref, max_norm)
    assert abs(float(m.grad_norm(plan)) - norm) <= 1e-6 * norm
    n = m.grad_clip(plan, max_norm)
    assert n.shape == () and abs(float(n) - norm) <= 1e-6 * norm
    for a, b, dt in zip(outs, clipped, dtypes):
        # one product in fp32, one rounding
        close(a, b, 2e-6 if dt == "f32" else 3e-3 if a.numel() > 100 else 4e-3, dt)
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(got, keep))
    if max_norm > norm:
        assert all(torch.equal(a, b) for a, b in zip(outs, keep))


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-19, 1e18, 1e20, 1e30])
def test_grad_norm_over_the_fp32_range(scale):
    from matrix_state_non_gb300 import binding as m
    ref, got = _grads([(50000,), (33,)], ["f32", "f32"], seed=5, scale=scale)
    norm, _ = o.clip(ref, 1.0)
    assert abs(float(m.grad_norm(m.grad_plan(got))) - norm) <= 2e-6 * norm


@pytest.mark.parametrize("bad,norm_is,out_is", [(float("nan"), np.isnan, np.isnan), (float("inf"), np.isinf, None)])
def test_grad_clip_of_values_that_are_not_finite(bad, norm_is, out_is):
    """NaN reaches every output; an infinity makes the factor 0 (and 0 x inf NaN)."""
    from matrix_state_non_gb300 import binding as m
    _, got = _grads([(40000,), (10,)], ["f32", "bf16"], seed=6)
    got[0][39999] = bad
    n = m.grad_clip(m.grad_plan(got), 1.0)
    assert norm_is(float(n))
    a, b = host(got[0]), host(got[1])
    if out_is is not None:
        assert np.all(out_is(a)) and np.all(out_is(b))
    else:
        assert np.isnan(a[39999]) and np.all(a[:39999] == 0) and np.all(b == 0)


def test_grad_clip_many_times_is_the_same():
    import torch
    from matrix_state_non_gb300 import binding as m
    _, got = _grads([(300000,), (70001,), (5, 5)], ["bf16", "f32", "f32"], seed=8)
    outs = [[torch.empty_like(t) for t in got] for _ in range(2)]
    norms = [m.grad_clip(m.grad_plan(got, w), 1.0) for w in outs]
    assert torch.equal(*norms)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
