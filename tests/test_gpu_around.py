"""GPU parity of the residual norm, the gated linear recurrence and the
orthogonalised update with the float64 oracle.

Tolerances, from the arithmetic:
 - bf16 outputs: one rounding of an fp32 result, at most 2^-8 of the value;
 - the norm in fp32: the sum of squares keeps 16384 terms of one sign, added in
   at most 64 steps per thread and a tree, so at most about 80 roundings of
   2^-24, half of which the root leaves; with the products behind it 50 2^-24 =
   3e-6 of the value;  its gradients cancel by a few: 1e-5 (2-norm);
 - 8-bit outputs: half a step of the format, 2^-4 of the value or 2^-10 of the
   scale, and the scale's own error as above;
 - the recurrence: a step's rounding of about 2^-23 of the state decays with the
   state, so that over a memory of up to about 60 steps (the decays below) up to
   60 of them add up, 7e-6: 1e-5 (2-norm) for states and gradients;
 - the orthogonalised update: bf16 rounding, 2^-8 at most and 1.7e-3 in the mean,
   and operands of its products in 11 bits and more, 1.5e-3 of the result (found
   by simulation in float64 over spectra from flat to rank one): 5e-3 (2-norm).
"""
import numpy as np
import pytest

from layer_util import dev, host, ints, round_to
from oracle import around_oracle as o
from parity_util import rel_fro

pytestmark = pytest.mark.gpu

TOL = 1e-5
BF16_HALF, NORM_TOL = 2.0 ** -8, 3e-6


def close(got, ref, tol, label):
    got = host(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), label
    r = rel_fro(got, ref)
    assert r <= tol, (label, r)


def near(got, ref, tol, label, floor=0.0):
    """Every value within tol of its own size (and floor)."""
    got = host(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    off = np.abs(got - ref) - tol * np.abs(ref) - floor
    assert np.all(off <= 0), (label, off.max(), np.argmax(off))


def slice_of(x, dtype, wide):
    """x on the device as a column slice of a tensor `wide` columns wider, NaN in the others."""
    import torch
    t = dev(x, dtype)
    if not wide:
        return t
    full = torch.full(t.shape[:-1] + (t.shape[-1] + wide,), float("nan"), device="cuda", dtype=t.dtype)
    full[..., :-wide] = t
    return full[..., :-wide]


# ---------------------------------------------------------------------------
# Residual norm
# ---------------------------------------------------------------------------
ROWS = [((1, 1), 0), ((1, 8), 0), ((3, 7), 5), ((2, 5, 64), 8), ((5, 128), 0), ((9, 129), 0), ((4, 250), 6), ((33, 256), 0),
        ((7, 1000), 24), ((2, 3, 1024), 0), ((3, 1027), 1), ((130, 384), 0), ((2, 2048), 16), ((5, 4096), 0), ((3, 4100), 0),
        ((2, 5003), 3), ((2, 8192), 0), ((3, 16384), 0), ((2, 16381), 0), ((700, 96), 0), ((4100, 40), 0)]


def norm_inputs(shape, xt, ht, seed):
    r = np.random.default_rng(seed)
    size = np.exp(r.normal(size=shape[-1]))
    return dict(x=round_to(r.normal(size=shape), xt), residual=round_to(r.normal(size=shape) * size, ht),
                w=round_to(1 + 0.3 * r.normal(size=shape[-1]), "f32"))


def check_norm(r, d, ht, yt, eps, label=""):
    import torch
    y, h = o.residual_norm(d["x"], d["w"], d.get("residual"), eps)
    if "residual" in d:
        near(r["h"], h, BF16_HALF if ht == "bf16" else 2.0 ** -23, label + "h")
    if yt != "e4m3":
        # the fp32 sum h has 24 bits of its larger part, which counts where x and the residual cancel
        floor = 2.0 ** -23 * np.abs(y / np.where(h == 0, 1, h)) * (np.abs(d["x"]) + np.abs(d.get("residual", 0)))
        near(r["y"], y, NORM_TOL + (BF16_HALF if yt == "bf16" else 0), label + "y", floor)
        return
    assert r["y"].dtype is torch.float8_e4m3fn
    _, scale = o.quantize(y)
    near(r["scale"], scale, 2 * NORM_TOL, label + "scale", 2.0 ** -149)
    wide = np.repeat(scale, 128, -1)[..., :y.shape[-1]]
    near(_dequantised(r), y, 2.0 ** -4 + 1e-5, label + "q", 2.0 ** -10 * wide * (1 + 1e-5))


def _dequantised(r):
    q, scale = r["y"].float(), r["scale"]
    return q * scale.repeat_interleave(128, -1)[..., :q.shape[-1]]


@pytest.mark.parametrize("yt", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("xt,ht", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shape,wide", ROWS)
def test_norm(shape, wide, xt, ht, yt):
    import torch
    from matrix_state_non_gb300 import binding as m
    types = dict(bf16=torch.bfloat16, f32=torch.float32, e4m3=torch.float8_e4m3fn)
    d = norm_inputs(shape, xt, ht, sum(shape))
    w = dev(d["w"])
    r = m.residual_norm(slice_of(d["x"], xt, wide), w, dev(d["residual"], ht), eps=1e-5, dtype=types[yt])
    check_norm(r, d, ht, yt, 1e-5)
    first = dict(x=d["x"], w=d["w"])
    r = m.residual_norm(slice_of(d["x"], xt, wide), w, eps=1e-5, dtype=types[yt])
    assert "h" not in r
    check_norm(r, first, ht, yt, 1e-5, "first ")


@pytest.mark.parametrize("shape", [(5, 1000), (3, 403), (2, 6000)])
def test_norm_in_place(shape):
    """h may be the residual; outputs may be given."""
    import torch
    from matrix_state_non_gb300 import binding as m
    d = norm_inputs(shape, "bf16", "f32", 3)
    x, w, res = dev(d["x"], "bf16"), dev(d["w"]), dev(d["residual"])
    want = m.residual_norm(x, w, res)
    y = torch.empty_like(x)
    got = m.residual_norm(x, w, res, out=dict(h=res, y=y))
    assert got["h"] is res and got["y"] is y and torch.equal(res, want["h"]) and torch.equal(y, want["y"])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("ht", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [True, False])
@pytest.mark.parametrize("shape", [s for s, _ in ROWS])
def test_norm_backward(shape, dh, ht, dt):
    from matrix_state_non_gb300 import binding as m
    r = np.random.default_rng(sum(shape) + 1)
    h, dy = round_to(r.normal(size=shape) * np.exp(r.normal(size=shape[-1])), ht), round_to(r.normal(size=shape), dt)
    w, up = round_to(1 + 0.3 * r.normal(size=shape[-1]), "f32"), round_to(r.normal(size=shape), "f32") if dh else None
    dx, dw = o.residual_norm_backward(h, w, dy, up, 1e-3)
    got = m.residual_norm_backward(dev(h, ht), dev(w), dev(dy, dt), dh=dev(up), eps=1e-3)
    # a row of one value has a gradient near 0: of the size of its two terms
    s = 1 / np.sqrt(np.mean(h * h, -1, keepdims=True) + 1e-3)
    size = np.linalg.norm(s * w * dy) / max(np.linalg.norm(dx), 1e-300)
    close(got["dx"], dx, TOL * max(1, size), "dx")
    close(got["dw"], dw, TOL * max(1, np.linalg.norm(np.sqrt(((dy * h * s) ** 2).reshape(-1, shape[-1]).sum(0)))
                                   / np.linalg.norm(dw)), "dw")


def test_norm_backward_in_place():
    import torch
    from matrix_state_non_gb300 import binding as m
    h, dy, dh, w = (torch.randn(s, device="cuda") for s in ((40, 1000), (40, 1000), (40, 1000), (1000,)))
    want = m.residual_norm_backward(h, w, dy, dh=dh)
    got = m.residual_norm_backward(h, w, dy, dh=dh, out=dict(dx=dh))
    assert got["dx"] is dh and torch.equal(dh, want["dx"]) and torch.equal(got["dw"], want["dw"])


def test_norm_of_rows_that_are_zero_or_not_finite():
    """A row of zeros gives zeros; a NaN or an infinity spoils its own row alone."""
    import torch
    from matrix_state_non_gb300 import binding as m
    w = torch.ones(300, device="cuda")
    x = torch.randn(6, 300, device="cuda")
    x[1], x[3, 7], x[4, 290] = 0, float("nan"), float("inf")
    for ty in (torch.bfloat16, torch.float32, torch.float8_e4m3fn):
        r = m.residual_norm(x, w, torch.zeros_like(x), dtype=ty)
        y = r["y"].float()
        assert torch.equal(y[1], torch.zeros_like(y[1])) and y[3].isnan().all() and y[4, 290].isnan()
        assert y[[0, 1, 2, 5]].isfinite().all() and torch.equal(y[4, :290], torch.zeros_like(y[4, :290]))
        if "scale" in r:
            assert bool((r["scale"][1] == 2.0 ** -126).all())


def test_norm_of_small_and_large_rows():
    """Values near 1e-15 (where eps rules) and 1e15 keep their digits."""
    from matrix_state_non_gb300 import binding as m
    d = norm_inputs((4, 520), "f32", "f32", 9)
    for size in (1e-15, 1e15):
        x, res = round_to(d["x"] * size, "f32"), round_to(d["residual"] * size, "f32")
        y, h = o.residual_norm(x, d["w"], res, 1e-6)
        r = m.residual_norm(dev(x), dev(d["w"]), dev(res), eps=1e-6)
        close(r["y"], y, TOL, "y")
        close(r["h"], h, TOL, "h")


# ---------------------------------------------------------------------------
# Gated linear recurrence
# ---------------------------------------------------------------------------
# B, T, C, dtype, lengths, H_0, wide
SCAN = [(1, 1, 1, "f32", None, False, 0), (1, 1, 64, "bf16", None, True, 0), (2, 5, 8, "bf16", (5, 1), True, 8),
        (3, 70, 24, "f32", (70, 1, 0), True, 5), (2, 63, 33, "bf16", None, False, 0), (2, 129, 66, "bf16", (2, 128), True, 4),
        (4, 19, 13, "f32", (0, 1, 3, 19), False, 1), (1, 1000, 40, "f32", None, True, 0), (1, 2100, 130, "bf16", None, True, 2),
        (2, 1025, 256, "bf16", (1025, 700), True, 16), (5, 257, 403, "f32", (257, 256, 0, 31, 33), True, 17),
        (1, 4099, 64, "bf16", None, False, 0), (2, 300, 1024, "bf16", None, True, 0), (40, 17, 72, "bf16", None, True, 0),
        (1, 515, 2050, "f32", None, False, 0), (3, 16, 127, "f32", (17, -3, 16), True, 0)]


def scan_inputs(B, T, C, dtype, seed, h0, memory=60.0):
    """Decays with memories of one step to about `memory` steps."""
    r = np.random.default_rng(seed)
    d = dict(x=round_to(r.normal(size=(B, T, C)), dtype), a=round_to(r.normal(size=(B, T, C)), dtype),
             dy=round_to(r.normal(size=(B, T, C)), dtype))
    d["alpha"] = round_to(np.exp(r.uniform(np.log(0.5), np.log(8.0), C)), "f32")
    d["beta"] = round_to(np.log(np.expm1(np.exp(r.uniform(np.log(1 / memory), np.log(1.5), C)) / d["alpha"])), "f32")
    d["H_0"] = round_to(r.normal(size=(B, C)), "f32") if h0 else None
    d["dH_T"] = round_to(r.normal(size=(B, C)), "f32") if h0 else None
    return d


def scan_dev(d, dtype, wide, lengths):
    g = {n: (slice_of(v, dtype, wide) if n in ("x", "a") else dev(v, dtype if n == "dy" else "f32")) for n, v in d.items()}
    if lengths is not None:
        for b, n in enumerate(lengths):  # what lies behind a sequence's end must not be read
            for k in ("x", "a", "dy"):
                g[k][b, max(n, 0):] = float("nan")
    return g


def clamped(lengths, T):
    return None if lengths is None else [min(max(n, 0), T) for n in lengths]


@pytest.mark.parametrize("B,T,C,dtype,lengths,h0,wide", SCAN)
def test_linear_scan(B, T, C, dtype, lengths, h0, wide):
    from matrix_state_non_gb300 import binding as m
    d = scan_inputs(B, T, C, dtype, T + C, h0)
    g = scan_dev(d, dtype, wide, lengths)
    y, H = o.linear_scan(d["x"], d["a"], d["alpha"], d["beta"], d["H_0"], clamped(lengths, T))
    r = m.linear_scan(g["x"], g["a"], g["alpha"], g["beta"], H_0=g["H_0"], lengths=ints(lengths))
    close(r["H_T"], H, TOL, "H_T")
    near(r["y"], y, (BF16_HALF if dtype == "bf16" else 0) + TOL, "y", TOL * np.abs(y).max())
    if lengths is not None:
        for b, n in enumerate(clamped(lengths, T)):
            assert np.all(host(r["y"])[b, n:] == 0.0)
    assert "H_T" not in m.linear_scan(g["x"], g["a"], g["alpha"], g["beta"], lengths=ints(lengths), want_state=False)


@pytest.mark.parametrize("B,T,C,dtype,lengths,h0,wide", SCAN)
def test_linear_scan_backward(B, T, C, dtype, lengths, h0, wide):
    import torch
    from matrix_state_non_gb300 import binding as m
    d = scan_inputs(B, T, C, dtype, T + C, h0)
    g = scan_dev(d, dtype, wide, lengths)
    ref = o.linear_scan_backward(d["x"], d["a"], d["alpha"], d["beta"], d["dy"], d["H_0"], d["dH_T"], clamped(lengths, T))
    call = lambda: m.linear_scan_backward(g["x"], g["a"], g["alpha"], g["beta"], g["dy"], H_0=g["H_0"],  # noqa: E731
                                          dH_T=g["dH_T"], lengths=ints(lengths), want_dH0=True)
    got = call()
    n = B * T
    for k in ("dx", "da", "dH_0"):
        close(got[k], ref[k], TOL, k)
    for k in ("dalpha", "dbeta"):  # sums of n terms of both signs, each as good as the above
        close(got[k], ref[k], TOL * 4 if n > 1 else TOL, k)
    again = call()
    for k in ref:
        assert torch.equal(got[k], again[k]), k
    if lengths is not None:
        for b, e in enumerate(clamped(lengths, T)):
            assert np.all(host(got["dx"])[b, e:] == 0.0) and np.all(host(got["da"])[b, e:] == 0.0)


@pytest.mark.parametrize("B", [36, 37, 44, 56, 70, 90, 100, 150, 200, 230])
@pytest.mark.parametrize("C,dtype", [(16, "bf16"), (9, "f32")])
def test_linear_scan_of_many_sequences(B, C, dtype):
    """One to eight blocks share a sequence, by the number of sequences."""
    from matrix_state_non_gb300 import binding as m
    T = 1030
    d = scan_inputs(B, T, C, dtype, B, True)
    lengths = [int(n) for n in np.random.default_rng(B).integers(-3, T + 5, B)]
    lengths[:4] = [T, 0, 1, T - 1]
    g = scan_dev(d, dtype, 0, lengths)
    y, H = o.linear_scan(d["x"], d["a"], d["alpha"], d["beta"], d["H_0"], clamped(lengths, T))
    r = m.linear_scan(g["x"], g["a"], g["alpha"], g["beta"], H_0=g["H_0"], lengths=ints(lengths))
    close(r["H_T"], H, TOL, "H_T")
    near(r["y"], y, (BF16_HALF if dtype == "bf16" else 0) + TOL, "y", TOL * np.abs(y).max())
    ref = o.linear_scan_backward(d["x"], d["a"], d["alpha"], d["beta"], d["dy"], d["H_0"], d["dH_T"], clamped(lengths, T))
    got = m.linear_scan_backward(g["x"], g["a"], g["alpha"], g["beta"], g["dy"], H_0=g["H_0"], dH_T=g["dH_T"],
                                 lengths=ints(lengths), want_dH0=True)
    for k in ref:
        close(got[k], ref[k], 4 * TOL if k in ("dalpha", "dbeta") else TOL, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_scan_without_beta(dtype):
    from matrix_state_non_gb300 import binding as m
    d = scan_inputs(2, 50, 20, dtype, 5, True)
    g = scan_dev(d, dtype, 0, None)
    y, H = o.linear_scan(d["x"], d["a"], d["alpha"], None, d["H_0"])
    close(m.linear_scan(g["x"], g["a"], g["alpha"], H_0=g["H_0"])["H_T"], H, TOL, "H_T")
    ref = o.linear_scan_backward(d["x"], d["a"], d["alpha"], None, d["dy"], d["H_0"])
    got = m.linear_scan_backward(g["x"], g["a"], g["alpha"], None, g["dy"], H_0=g["H_0"])
    assert "dbeta" not in got and "dH_0" not in got
    for k in ("dx", "da", "dalpha"):
        close(got[k], ref[k], TOL, k)


def test_state_in_place():
    """H_T may be H_0, dH_0 may be dH_T."""
    import torch
    from matrix_state_non_gb300 import binding as m
    d = scan_inputs(2, 700, 100, "bf16", 6, True)
    g = scan_dev(d, "bf16", 0, None)
    want = m.linear_scan(g["x"], g["a"], g["alpha"], g["beta"], H_0=g["H_0"])
    H = g["H_0"].clone()
    got = m.linear_scan(g["x"], g["a"], g["alpha"], g["beta"], H_0=H, out=dict(H_T=H))
    assert got["H_T"] is H and torch.equal(H, want["H_T"]) and torch.equal(got["y"], want["y"])
    call = lambda dH, **kw: m.linear_scan_backward(g["x"], g["a"], g["alpha"], g["beta"], g["dy"], H_0=g["H_0"],  # noqa: E731
                                                   dH_T=dH, want_dH0=True, **kw)
    want = call(g["dH_T"])
    dH = g["dH_T"].clone()
    got = call(dH, out=dict(dH_0=dH))
    assert got["dH_0"] is dH and torch.equal(dH, want["dH_0"]) and torch.equal(got["dx"], want["dx"])


@pytest.mark.parametrize("B,C,dtype,wide", [(1, 1, "f32", 0), (3, 7, "bf16", 3), (32, 1024, "bf16", 0), (70000, 8, "bf16", 0),
                                            (5, 403, "f32", 2), (2, 2050, "bf16", 0), (9, 66, "bf16", 2)])
def test_linear_step(B, C, dtype, wide):
    from matrix_state_non_gb300 import binding as m
    d = scan_inputs(B, 1, C, dtype, B + C, True)
    x, a = d["x"][:, 0], d["a"][:, 0]
    H = dev(d["H_0"])
    y = m.linear_step(H, slice_of(x, dtype, wide), slice_of(a, dtype, wide), dev(d["alpha"]), dev(d["beta"]))
    ref, _ = o.linear_scan(d["x"], d["a"], d["alpha"], d["beta"], d["H_0"])
    close(H, ref[:, 0], TOL, "H")
    near(y, ref[:, 0], (BF16_HALF if dtype == "bf16" else 0) + TOL, "y", TOL * np.abs(ref).max())


def test_extreme_gates():
    """Decays of 0 and 1 to the last bit, softplus far on both sides, alpha of 0."""
    from matrix_state_non_gb300 import binding as m
    T, C = 200, 12
    r = np.random.default_rng(8)
    x = round_to(r.normal(size=(1, T, C)), "f32")
    a = round_to(r.normal(size=(1, T, C)), "f32")
    alpha = np.array([0.0, 1e-6, 1e-3, 1.0, 50.0, 1e6, 1.0, 1.0, 1.0, 1.0, 30.0, 1e-20])
    beta = np.array([0.0, 0.0, 3.0, 0.0, 0.0, 0.0, -100.0, 100.0, -15.0, 30.0, -12.0, 80.0])
    alpha, beta = round_to(alpha, "f32"), round_to(beta, "f32")
    H_0, dH, dy = (round_to(r.normal(size=s), "f32") for s in ((1, C), (1, C), (1, T, C)))
    y, H = o.linear_scan(x, a, alpha, beta, H_0)
    got = m.linear_scan(dev(x), dev(a), dev(alpha), dev(beta), H_0=dev(H_0))
    ref = o.linear_scan_backward(x, a, alpha, beta, dy, H_0, dH)
    bwd = m.linear_scan_backward(dev(x), dev(a), dev(alpha), dev(beta), dev(dy), H_0=dev(H_0), dH_T=dev(dH), want_dH0=True)
    # channel by channel: softplus loses up to |z| 2^-24 of itself far below 0, and 200 steps add up: 200 * 100 * 6e-8 at
    # most, of what the gate moves; 1e-4 of the channel's own size
    for c in range(C):
        close(got["y"][..., c], y[..., c], 1e-4, ("y", c))
        for k in ("dx", "da"):
            size = np.linalg.norm(ref[k][..., c])
            off = np.linalg.norm(host(bwd[k])[..., c] - ref[k][..., c])
            assert off <= 1e-4 * size + 1e-37, (k, c, off, size)
        assert abs(host(bwd["dH_0"])[0, c] - ref["dH_0"][0, c]) <= 1e-4 * abs(ref["dH_0"][0, c]) + 1e-37


@pytest.mark.parametrize("dtype,C", [("f32", 12), ("bf16", 64), ("bf16", 9)])
def test_gates_at_the_ends_of_their_type(dtype, C):
    """a of the type's largest and lowest value and of either infinity: the state is x, or stays (alpha of 0: stays)."""
    import torch
    from matrix_state_non_gb300 import binding as m
    T = 300
    d = scan_inputs(2, T, C, dtype, 11, True)
    limit = torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16)
    opened, shut = (40, 133, 134, 299), (0, 77, 78, 200)
    ref_a = np.array(d["a"])
    for n in (opened, shut):
        ref_a[:, list(n)] = 1e30 if n is opened else -1e30  # (f is 0 or 1, softplus finite)
    alpha = np.array(d["alpha"])
    alpha[1] = 0.0
    ref_y, ref_H = o.linear_scan(d["x"], ref_a, alpha, d["beta"], d["H_0"])
    dy = round_to(np.random.default_rng(12).normal(size=(2, T, C)), dtype)
    ref = o.linear_scan_backward(d["x"], ref_a, alpha, d["beta"], dy, d["H_0"])
    live = np.arange(C) != 1  # (where alpha is 0, dalpha is as large as softplus)
    some = torch.from_numpy(live).cuda()
    for high, low in ((limit.max, limit.min), (float("inf"), float("-inf"))):
        a = dev(d["a"], dtype)
        a[:, list(opened)], a[:, list(shut)] = high, low
        if high == float("inf"):  # (0 times infinity where alpha is 0)
            a[:, list(opened), 1] = 1.0
        args = (dev(d["x"], dtype), a, dev(alpha), dev(d["beta"]))
        got = m.linear_scan(*args, H_0=dev(d["H_0"]))
        close(got["H_T"], ref_H, TOL, "H_T")
        near(got["y"], ref_y, (BF16_HALF if dtype == "bf16" else 0) + TOL, "y", TOL * np.abs(ref_y).max())
        bwd = m.linear_scan_backward(*args, dev(dy, dtype), H_0=dev(d["H_0"]))
        for k in ("dx", "da"):
            close(bwd[k], ref[k], TOL, k)
        for k in ("dalpha", "dbeta"):
            close(bwd[k][some], ref[k][live], 4 * TOL, k)
        H = dev(d["H_0"]).clone()
        y = m.linear_step(H, args[0][:, 40].contiguous(), a[:, 40].contiguous(), args[2], args[3])
        assert torch.equal(y[:, some], args[0][:, 40][:, some]) and torch.equal(H[:, 1], dev(d["H_0"])[:, 1])


def test_scan_values_that_are_not_finite():
    """They reach their own channel from their own step on, and no other sequence."""
    import torch
    from matrix_state_non_gb300 import binding as m
    d = scan_inputs(2, 600, 70, "f32", 9, True)
    clean = m.linear_scan(*(dev(d[n]) for n in ("x", "a", "alpha", "beta")), H_0=dev(d["H_0"]))["y"]
    for t, value in ((0, float("nan")), (130, float("inf")), (599, float("nan"))):
        x = dev(d["x"])
        x[1, t, 33] = value
        y = m.linear_scan(x, dev(d["a"]), dev(d["alpha"]), dev(d["beta"]), H_0=dev(d["H_0"]))["y"]
        assert not y[1, t:, 33].isfinite().any()
        y[1, t:, 33] = clean[1, t:, 33]
        assert torch.equal(y, clean)


# ---------------------------------------------------------------------------
# Orthogonalised update
# ---------------------------------------------------------------------------
ORTHO_TOL = 5e-3


def spectrum(rows, cols, kind, seed):
    r = np.random.default_rng(seed)
    g = r.normal(size=(rows, cols))
    few = min(rows, cols)
    if kind == "gauss":
        return g
    if kind == "decay":
        u, _, v = np.linalg.svd(g, full_matrices=False)
        return (u * np.arange(1, few + 1.0) ** -1.0) @ v
    if kind == "floor":
        k = max(1, few // 16)
        return r.normal(size=(rows, k)) @ r.normal(size=(k, cols)) + 1e-2 * g
    return r.normal(size=(rows, 1)) @ r.normal(size=(1, cols))


ORTHO = [(1, 1, 1), (1, 1, 9), (1, 9, 1), (2, 3, 5), (3, 16, 16), (1, 17, 40), (2, 64, 64), (5, 64, 48), (2, 33, 64), (1, 65, 64),
         (2, 64, 200), (2, 100, 100), (1, 128, 128), (1, 130, 70), (2, 128, 384), (1, 200, 513), (1, 333, 1000),
         (2, 257, 256), (1, 512, 512), (3, 640, 130)]


@pytest.mark.parametrize("kind", ["gauss", "decay", "floor", "rank1"])
@pytest.mark.parametrize("n,rows,cols", ORTHO)
def test_orthogonalize(n, rows, cols, kind):
    import torch
    from matrix_state_non_gb300 import binding as m
    g = np.stack([spectrum(rows, cols, kind, 10 * rows + cols + i) for i in range(n)])
    for dtype in ("bf16", "f32"):
        x = round_to(g, dtype)
        got = m.orthogonalize(dev(x, dtype))
        assert got.dtype is torch.bfloat16
        # singular values of the rounded matrix that stand for noise of its own are in it, and are brought up like others
        ref = o.orthogonalize(x)
        for i in range(n):
            close(got[i], ref[i], ORTHO_TOL, (dtype, i))


@pytest.mark.parametrize("kind", ["gauss", "decay", "floor", "rank1"])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 300), (2, 3, 1000), (1, 700, 17), (3, 40, 257), (2, 64, 513), (1, 2100, 64), (2, 33, 4099),
                                         (1, 9000, 5), (1, 65, 300), (2, 257, 65)])
def test_orthogonalize_thin(n, rows, cols, kind):
    """One side short, the other long; few rows average least over the errors of an entry."""
    from matrix_state_non_gb300 import binding as m
    g = np.stack([spectrum(rows, cols, kind, 7 * rows + cols + i) for i in range(n)])
    for dtype in ("bf16", "f32"):
        x = round_to(g, dtype)
        got = m.orthogonalize(dev(x, dtype))
        ref = o.orthogonalize(x)
        for i in range(n):
            close(got[i], ref[i], ORTHO_TOL, (dtype, i))


@pytest.mark.parametrize("kind", ["gauss", "floor"])
@pytest.mark.parametrize("steps", [1, 2, 6, 11, 32])
@pytest.mark.parametrize("rows,cols", [(24, 32), (20, 300), (400, 48), (100, 130)])
def test_orthogonalize_few_and_many_steps(rows, cols, steps, kind):
    """The polynomial maps [0.67, 1.21] into itself, where its slope of up to 4
    makes the places of singular values unpredictable after many steps; but there
    they stay, and after eleven all of these are there."""
    import torch
    from matrix_state_non_gb300 import binding as m
    x = round_to(spectrum(rows, cols, kind, 5), "f32")
    got = m.orthogonalize(dev(x), steps=steps)
    if steps <= 2:
        close(got, o.orthogonalize(x, steps), ORTHO_TOL, steps)
        return
    s = torch.linalg.svdvals(got.double())
    assert float(s.max()) <= 1.25, s
    assert steps < 11 or float(s.min()) >= 0.6, s


@pytest.mark.parametrize("n,rows,cols", [(27, 512, 520), (8, 1000, 1025), (13, 1030, 777), (76, 513, 512)])
def test_orthogonalize_stacks(n, rows, cols):
    """Stacks that fill the GPU, whose matrices share tiles of 256 x 256."""
    import torch
    from matrix_state_non_gb300 import binding as m
    gen = torch.Generator(device="cuda").manual_seed(n)
    g = torch.randn((n, rows, cols), generator=gen, device="cuda")
    got = m.orthogonalize(g)
    a, b, c = o.COEFFICIENTS
    for i in (0, 1, n // 2, n - 1):
        x = g[i].double()
        x = x / (x.norm() + 1e-7)
        for _ in range(5):
            gram = x @ x.mT
            x = a * x + (b * gram + c * gram @ gram) @ x
        assert float((got[i].double() - x).norm() / x.norm()) <= ORTHO_TOL, i
    assert torch.equal(got, m.orthogonalize(g))


@pytest.mark.parametrize("rows,cols", [(48, 64), (200, 136)])
@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_orthogonalize_steps(rows, cols, steps):
    from matrix_state_non_gb300 import binding as m
    x = round_to(spectrum(rows, cols, "gauss", 3), "f32")
    close(m.orthogonalize(dev(x), steps=steps), o.orthogonalize(x, steps), ORTHO_TOL, steps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(520, 516), (20, 700), (600, 904), (130, 200)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_orthogonalize_early_steps(rows, cols, steps, dtype):
    """Whichever step is the last: what X is kept in depends on it."""
    from matrix_state_non_gb300 import binding as m
    for kind in ("gauss", "rank1"):
        x = round_to(spectrum(rows, cols, kind, 13), dtype)
        close(m.orthogonalize(dev(x, dtype), steps=steps), o.orthogonalize(x, steps), ORTHO_TOL, (steps, kind))


@pytest.mark.parametrize("rows,cols", [(40, 60), (140, 150)])
def test_orthogonalize_sizes_of_values(rows, cols):
    """The result does not depend on the size of G, over the fp32 range; eps counts where G is small; zeros stay zeros."""
    import torch
    from matrix_state_non_gb300 import binding as m
    x = round_to(spectrum(rows, cols, "gauss", 4), "f32")
    for size in (2.0 ** -100, 2.0 ** -40, 2.0 ** 40, 2.0 ** 100):
        close(m.orthogonalize(dev(x * size), eps=0.0), o.orthogonalize(x, eps=0.0), ORTHO_TOL, size)
    small = round_to(x * 1e-9, "f32")
    close(m.orthogonalize(dev(small), eps=1e-7), o.orthogonalize(small, eps=1e-7), ORTHO_TOL, "eps")
    z = torch.zeros((2, rows, cols), device="cuda")
    z[1] = dev(x)
    got = m.orthogonalize(z)
    assert torch.equal(got[0], torch.zeros_like(got[0])) and torch.equal(got[1], m.orthogonalize(z[1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(40, 60), (30, 500), (140, 150), (150, 140), (520, 516)])
def test_orthogonalize_sizes_at_the_ends(rows, cols, dtype):
    """Powers of two leave the result as it is, up to norms whose inverse is no normal fp32 number; so does eps = 0."""
    import torch
    from matrix_state_non_gb300 import binding as m
    x = dev(spectrum(rows, cols, "gauss", 6), dtype)
    want = m.orthogonalize(x, eps=0.0)
    close(want, o.orthogonalize(host(x).astype(np.float64), eps=0.0), ORTHO_TOL, "1")
    up = 126 - int(np.floor(np.log2(float(x.double().norm()))))
    for k in (-90, 60, up, up + 1):
        y = x * 2.0 ** (k // 2) * 2.0 ** (k - k // 2)
        assert bool(y.isfinite().all())
        # factors of fp32 with and without all their bits: an operand's last place may differ
        close(m.orthogonalize(y, eps=0.0), host(want).astype(np.float64), ORTHO_TOL, k)
    z = torch.zeros_like(x)
    assert torch.equal(m.orthogonalize(z), z.bfloat16())


@pytest.mark.parametrize("kind", ["gauss", "decay", "floor", "rank1"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,cols", [(1, 520, 700), (2, 1100, 600), (1, 800, 8200), (30, 515, 512), (20, 800, 800),
                                         (20, 904, 800)])
def test_orthogonalize_long_sides(n, rows, cols, dtype, kind):
    """Matrices whose last step takes X in one part: 3.4445 2^-12 of it, 1.2 / 0.67 at most of the result's size: 1.5e-3."""
    import torch
    from matrix_state_non_gb300 import binding as m
    x = torch.stack([dev(spectrum(rows, cols, kind, 3 * rows + i), dtype) for i in range(min(n, 2))])
    x = x.repeat((n + 1) // 2, 1, 1)[:n].contiguous()
    got = m.orthogonalize(x)
    a, b, c = o.COEFFICIENTS
    for i in {0, n - 1}:
        v = x[i].double()
        v = v if rows <= cols else v.mT
        v = v / (v.norm() + 1e-7)
        for _ in range(5):
            gram = v @ v.mT
            v = a * v + (b * gram + c * gram @ gram) @ v
        v = v if rows <= cols else v.mT
        off = float((got[i].double() - v).norm() / v.norm())
        assert off <= ORTHO_TOL, (i, off)


@pytest.mark.parametrize("rows,cols", [(64, 64), (150, 140)])
def test_orthogonalize_not_finite(rows, cols):
    """A NaN spoils its own matrix and no other of the stack."""
    import torch
    from matrix_state_non_gb300 import binding as m
    g = torch.randn((3, rows, cols), device="cuda")
    clean = m.orthogonalize(g)
    g[1, 5, 7] = float("nan")
    got = m.orthogonalize(g)
    assert got[1].isnan().all() and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


def test_orthogonalize_in_place_and_workspace():
    import torch
    from matrix_state_non_gb300 import binding as m
    for shape in ((2, 3, 64, 40), (150, 200), (300, 160)):
        g = torch.randn(shape, device="cuda").bfloat16()
        want = m.orthogonalize(g)
        ws = torch.empty(m.m2rnn_orthogonalize_workspace_size(g.numel() // (shape[-1] * shape[-2]), *shape[-2:]),
                         dtype=torch.uint8, device="cuda")
        assert torch.equal(m.orthogonalize(g.clone(), workspace=ws), want)
        assert m.sync_status(ws)[0] == m.M2RNN_OK
        assert m.orthogonalize(g, out=g) is g and torch.equal(g, want)


@pytest.mark.parametrize("shape", [(20, 400), (700, 33), (2, 5, 300), (65, 70), (3, 128, 257)])
def test_orthogonalize_in_place_elsewhere(shape):
    import torch
    from matrix_state_non_gb300 import binding as m
    g = torch.randn(shape, device="cuda").bfloat16()
    want = m.orthogonalize(g, steps=7)
    assert m.orthogonalize(g, steps=7, out=g) is g and torch.equal(g, want)


def test_orthogonalize_stacks_are_matrices_on_their_own():
    """Each matrix of a stack gets what it would get in a stack of as many others."""
    import torch
    from matrix_state_non_gb300 import binding as m
    for n, rows, cols in ((5, 40, 64), (4, 30, 900), (3, 200, 136), (30, 300, 300)):
        g = torch.randn((n, rows, cols), device="cuda")
        got = m.orthogonalize(g)
        turned = m.orthogonalize(g.flip(0).contiguous()).flip(0)
        assert torch.equal(got, turned)
        zeros = torch.zeros_like(g)
        zeros[n // 2] = g[n // 2]
        alone = m.orthogonalize(zeros)
        assert torch.equal(alone[n // 2], got[n // 2]) and int(alone[:n // 2].count_nonzero()) == 0


# ---------------------------------------------------------------------------
# Calls in graphs and on two streams
# ---------------------------------------------------------------------------
def _all_calls(g):
    from matrix_state_non_gb300 import binding as m
    import torch
    f = m.residual_norm(g["x"], g["w"], g["r"], dtype=torch.float8_e4m3fn)
    y = m.residual_norm(g["x"], g["w"], g["r"])["y"]
    b = m.residual_norm_backward(f["h"], g["w"], g["dy"], dh=g["dh"])
    s = m.linear_scan(y, g["r"], g["alpha"], g["beta"], H_0=g["H_0"])
    H = s["H_T"].clone()
    t = m.linear_step(H, y[:, 0].contiguous(), g["x"][:, 0].contiguous(), g["alpha"], g["beta"])
    d = m.linear_scan_backward(y, g["r"], g["alpha"], g["beta"], g["dy"], H_0=g["H_0"], dH_T=g["H_0"], want_dH0=True)
    small, large = m.orthogonalize(g["small"]), m.orthogonalize(g["large"])
    thin = m.orthogonalize(g["thin"])
    return [thin, f["y"].float(), f["scale"], f["h"], y, b["dx"], b["dw"], s["y"], s["H_T"], H, t, d["dx"], d["da"], d["dalpha"],
            d["dbeta"], d["dH_0"], small, large]


def _graph_inputs(seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=r(2, 700, 264).bfloat16(), r=r(2, 700, 264).bfloat16(), w=r(264), dy=r(2, 700, 264).bfloat16(),
                dh=r(2, 700, 264), alpha=r(264).exp(), beta=r(264), H_0=r(2, 264), small=r(3, 40, 64),
                large=r(2, 200, 136).bfloat16(), thin=r(2, 30, 600))


def test_calls_in_a_graph():
    import torch
    from test_gpu_layer_graphs import capture
    sets = [_graph_inputs(s) for s in (1, 2)]
    want = [_all_calls(g) for g in sets]
    buf = {n: t.clone() for n, t in sets[0].items()}
    graph, out = capture(lambda: _all_calls(buf))
    for g, w in zip(sets[::-1], want[::-1]):
        for n, t in g.items():
            buf[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, w)):
            assert torch.equal(a, b), i


def test_calls_on_two_streams():
    import torch
    sets = [_graph_inputs(s) for s in (3, 4)]
    want = [_all_calls(g) for g in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _all_calls(sets[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for i, (x, y) in enumerate(zip(a, b)):
            assert torch.equal(x, y), i
