"""The operators around the scans as they are measured: the residual RMS norm
(with an 8-bit output), the gated linear recurrence and the orthogonalised
update of a weight matrix.

Each case runs one pass of one operator.  With ``own`` false the pass is the
operator's plain form in elementary torch operations, in 32 bits, rounded once
at the end; with ``own`` true it is the call that a user makes of the library.
``exact`` is the operator's definition in 64 bits.

Layouts (the library's): activations [B,T,D] or [B,D] of one token, the
recurrence's state [B,C], stacks of weight gradients [n,rows,columns].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
BLOCK = 128  # values that share a scale
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # The residual stream of the repository's training workload (B=4, T=4096) at the hidden size of the gradient
        # lists, normalised for the next layer's projection.
        dict(name="norm_prompt_4k", op="norm_forward", rows=16384, D=1024, x="bf16", h="bf16", y="bf16", wide=0,
             first=False),
        # Serving in 8 bits: prompts of odd lengths and an odd width, the branch a column slice of a fused product, the
        # residual stream in fp32.
        dict(name="norm_prompt_fp8", op="norm_forward", rows=3063, D=1000, x="bf16", h="f32", y="e4m3", wide=24,
             first=False),
        # The training step's backward of the first case.
        dict(name="norm_train_4k", op="norm_backward", rows=16384, D=1024, h="bf16", dy="bf16", dh=True),
        # One token for 32 sequences, in 8 bits: a latency.
        dict(name="norm_step_32", op="norm_forward", rows=32, D=1024, x="bf16", h="bf16", y="e4m3", wide=0, first=False),
        # The repository's 16K workload (B=2, 16 heads of 64) as channels of a vector recurrence: a long prompt.
        dict(name="linear_prompt_16k", op="linear_forward", B=2, T=16384, C=1024, dtype="bf16", wide=0, ragged=False,
             h0=False),
        # A ragged batch (lengths 0 and 1 among them) that continues from kept states, odd sizes, in fp32.
        dict(name="linear_prompt_odd", op="linear_forward", B=5, T=1021, C=403, dtype="f32", wide=17, ragged=True,
             h0=True),
        # The training workload's B=4, T=4096: all gradients.
        dict(name="linear_train_4k", op="linear_backward", B=4, T=4096, C=1024, dtype="bf16", wide=0, ragged=False,
             h0=False),
        # One token for 32 sequences: a latency.
        dict(name="linear_step_32", op="linear_step", B=32, C=1024, dtype="bf16"),
        # The gradients of the recurrence's W, 64 x 64 for 8 heads, of 24 layers.
        dict(name="ortho_heads", op="ortho", n=192, rows=64, cols=64, dtype="f32"),
        # One square projection of the hidden size.
        dict(name="ortho_layer", op="ortho", n=1, rows=1024, cols=1024, dtype="f32"),
        # The wide projections of 24 layers.
        dict(name="ortho_24_wide", op="ortho", n=24, rows=1024, cols=4096, dtype="bf16"),
        # Tall matrices of odd sizes.
        dict(name="ortho_odd_tall", op="ortho", n=2, rows=1000, cols=333, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_forward", "norm_backward", "linear_forward", "linear_backward", "linear_step",
                     "ortho", "ortho"])
    if op.startswith("norm"):
        D = _log_int(rng, 48, 8192)
        D = D if rng.random() < 0.4 else -(-D // 64) * 64
        rows = _log_int(rng, 1, 16384)
        while rows * D > 16384 * 1024:
            rows = rows // 2 + 1
        if op == "norm_backward":
            return dict(op=op, rows=rows, D=D, h=rng.choice(["bf16", "f32"]), dy=rng.choice(["bf16", "f32"]),
                        dh=rng.random() < 0.7)
        return dict(op=op, rows=rows, D=D, x=rng.choice(["bf16", "bf16", "f32"]), h=rng.choice(["bf16", "f32"]),
                    y=rng.choice(["bf16", "f32", "e4m3", "e4m3"]), wide=rng.choice([0, 0, 24, 17]),
                    first=rng.random() < 0.2)
    if op == "ortho":
        m, n = _log_int(rng, 16, 2048), _log_int(rng, 16, 4096)
        if rng.random() < 0.6:
            m, n = -(-m // 16) * 16, -(-n // 16) * 16
        if rng.random() < 0.3:
            m, n = n, m
        few = min(m, n)
        most = max(1, min(64, int(24 * 1024 * 1024 * 4096 / (few * m * n))))
        return dict(op=op, n=_log_int(rng, 1, most), rows=m, cols=n, dtype=rng.choice(["bf16", "f32"]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    C = _log_int(rng, 48, 2560)
    C = C if rng.random() < 0.4 else -(-C // 8) * 8
    if op == "linear_step":
        return dict(op=op, B=_log_int(rng, 1, 512), C=C, dtype=dtype)
    T, B = _log_int(rng, 1, 16384), _log_int(rng, 1, 8)
    while B * T * C > 2 * 16384 * 1024 or (op == "linear_backward" and B * T * C > 4 * 4096 * 1024):
        T = T // 2 + 1
    return dict(op=op, B=B, T=T, C=C, dtype=dtype, wide=rng.choice([0, 8, 17]), ragged=rng.random() < 0.5,
                h0=rng.random() < 0.5)


def _lengths(case):
    """The lengths of a ragged batch: full, one, none, then spread out."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [(T, 1, 0)[b] if b < 3 else T * (b - 2) // (B - 1) for b in range(B)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _rand(gen, shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * scale if scale != 1.0 else x).to(dtype)


def _prepare_norm(case, gen):
    rows, D = case["rows"], case["D"]
    # a residual stream has channels of very different size
    size = torch.exp(0.7 * torch.randn((D,), generator=gen, device="cuda"))
    s = dict(w=1.0 + 0.2 * torch.randn((D,), generator=gen, device="cuda"))
    h = (torch.randn((rows, D), generator=gen, device="cuda") * size).to(DTYPES[case["h"]])
    if case["op"] == "norm_backward":
        return dict(s, h=h, dy=_rand(gen, (rows, D), DTYPES[case["dy"]]),
                    dh=_rand(gen, (rows, D)) if case["dh"] else None)
    x = _rand(gen, (rows, D + case["wide"]), DTYPES[case["x"]])[:, :D]
    return dict(s, x=x, residual=None if case["first"] else h, y=DTYPES[case["y"]])


def _prepare_linear(case, gen):
    dt = DTYPES[case["dtype"]]
    B, C = case["B"], case["C"]
    # decays from a few steps to thousands, as the recurrences' gates are initialised
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((C,), generator=gen, device="cuda"))
    s = dict(alpha=1.0 + 15.0 * torch.rand((C,), generator=gen, device="cuda"), beta=torch.log(torch.expm1(step)))
    if case["op"] == "linear_step":
        return dict(s, x=_rand(gen, (B, C), dt), a=_rand(gen, (B, C), dt), H=_rand(gen, (B, C), scale=0.5),
                    y=torch.empty((B, C), device="cuda", dtype=dt))
    T = case["T"]
    z = _rand(gen, (B, T, 2 * C + case["wide"]), dt)  # x | a side by side, as one projection makes them
    s.update(x=z[..., :C], a=z[..., C:2 * C])
    s["H_0"] = _rand(gen, (B, C), scale=0.5) if case["h0"] else None
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"] == "linear_backward":
        s["dy"] = _rand(gen, (B, T, C), dt)
        s["dH_T"] = _rand(gen, (B, C)) if case["h0"] else None
    return s


def _prepare_ortho(case, gen):
    n, rows, cols = case["n"], case["rows"], case["cols"]
    # momentum of a gradient: a few strong directions over a wide floor, rows of different size
    rank = max(1, min(rows, cols) // 16)
    strong = _rand(gen, (n, rows, rank)) @ _rand(gen, (n, rank, cols)) * rank ** -0.5
    g = strong + _rand(gen, (n, rows, cols), scale=0.3)
    return dict(g=(1e-3 * g * torch.exp(0.5 * torch.randn((n, rows, 1), generator=gen, device="cuda"))).to(
        DTYPES[case["dtype"]]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["op"].split("_")[0]
    made = {"norm": _prepare_norm, "linear": _prepare_linear, "ortho": _prepare_ortho}[kind](case, gen)
    return dict(made, op=case["op"])


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _norm_forward(s):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["h"] = h.to(s["residual"].dtype)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"]
    if s["y"] is not torch.float8_e4m3fn:
        return dict(out, y=y.to(s["y"]))
    rows, D = y.shape
    blocks = torch.cat([y, y.new_zeros((rows, -D % BLOCK))], 1).unflatten(1, (-1, BLOCK))
    scale = torch.clamp(blocks.abs().amax(-1) / 448.0, min=torch.finfo(torch.float32).tiny)
    q = (blocks / scale[..., None]).flatten(1)[:, :D].to(torch.float8_e4m3fn)
    return dict(out, y=q.contiguous(), scale=scale)


def _norm_backward(s):
    h, dy = s["h"].float(), s["dy"].float()
    D = h.shape[-1]
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    p = dy * s["w"]
    dx = r * p - h * (r * r * r * (p * h).sum(-1, keepdim=True) / D)
    return dict(dx=dx if s["dh"] is None else dx + s["dh"], dw=(dy * h * r).sum(0))


def _keep(x, valid, other):
    return x if valid is None else torch.where(valid[..., None], x, other)


def _gate(s, valid):
    z = s["a"].float() + s["beta"]
    soft = torch.logaddexp(z, torch.zeros_like(z))
    u = _keep(s["alpha"] * soft, valid, 0.0)
    return z, soft, torch.exp(-u), -torch.expm1(-u)


def _scan(f, b):
    """h_t = f_t h_{t-1} + b_t from zero, in steps of doubled length."""
    shift = 1
    while shift < f.shape[1]:
        b = torch.cat([b[:, :shift], b[:, shift:] + f[:, shift:] * b[:, :-shift]], 1)
        f = torch.cat([f[:, :shift], f[:, shift:] * f[:, :-shift]], 1)
        shift *= 2
    return b


def _linear_states(s):
    B, T, C = s["x"].shape
    valid = None if s["lengths"] is None else torch.arange(T, device="cuda") < s["lengths"][:, None]
    z, soft, f, e = _gate(s, valid)
    x = _keep(s["x"].float(), valid, 0.0)
    H_0 = s["H_0"] if s["H_0"] is not None else x.new_zeros((B, C))
    b = e * x
    b = torch.cat([b[:, :1] + f[:, :1] * H_0[:, None], b[:, 1:]], 1)
    return valid, z, soft, f, e, x, H_0, _scan(f, b)


def _linear_forward(s):
    valid, z, soft, f, e, x, H_0, h = _linear_states(s)
    return dict(y=_keep(h, valid, 0.0).to(s["x"].dtype), H_T=h[:, -1].contiguous())


def _linear_backward(s):
    valid, z, soft, f, e, x, H_0, h = _linear_states(s)
    dy = _keep(s["dy"].float(), valid, 0.0)
    if s["dH_T"] is not None:
        dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dH_T"][:, None]], 1)
    ahead = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1)
    dh = _scan(ahead.flip(1), dy.flip(1)).flip(1)
    g = _keep(dh * f * (torch.cat([H_0[:, None], h[:, :-1]], 1) - x), valid, 0.0)
    da = -s["alpha"] * g / (1.0 + torch.exp(-z))
    out = dict(dx=_keep(dh * e, valid, 0.0), da=da, dalpha=-(g * soft).sum((0, 1)), dbeta=da.sum((0, 1)))
    return dict(out, dH_0=f[:, 0] * dh[:, 0]) if s["H_0"] is not None else out


def _linear_step(s):
    z, soft, f, e = _gate(s, None)
    s["H"].mul_(f).add_(e * s["x"].float())
    s["y"].copy_(s["H"])
    return dict(y=s["y"], H=s["H"])


def _ortho(s):
    a, b, c = COEFFICIENTS
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.mT if tall else x).contiguous().bfloat16()


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s):
    from matrix_state_non_gb300 import binding as m
    op = s["op"]
    if op == "norm_forward":
        return m.residual_norm(s["x"], s["w"], s["residual"], eps=EPS, dtype=s["y"])
    if op == "norm_backward":
        r = m.residual_norm_backward(s["h"], s["w"], s["dy"], dh=s["dh"], eps=EPS)
        return dict(dx=r["dx"], dw=r["dw"])
    if op == "linear_forward":
        r = m.linear_scan(s["x"], s["a"], s["alpha"], s["beta"], H_0=s["H_0"], lengths=s["lengths"])
        return dict(y=r["y"], H_T=r["H_T"])
    if op == "linear_backward":
        r = m.linear_scan_backward(s["x"], s["a"], s["alpha"], s["beta"], s["dy"], H_0=s["H_0"], dH_T=s["dH_T"],
                                   lengths=s["lengths"], want_dH0=s["H_0"] is not None)
        return {n: r[n] for n in ("dx", "da", "dalpha", "dbeta", "dH_0") if n in r}
    if op == "linear_step":
        y = m.linear_step(s["H"], s["x"], s["a"], s["alpha"], s["beta"], y=s["y"])
        return dict(y=y, H=s["H"])
    return m.orthogonalize(s["g"], steps=STEPS)


PLAIN = dict(norm_forward=_norm_forward, norm_backward=_norm_backward, linear_forward=_linear_forward,
             linear_backward=_linear_backward, linear_step=_linear_step, ortho=_ortho)


@torch.no_grad()
def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
SIZES = {"bf16": 2, "f32": 4, "e4m3": 1}


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, D = case["rows"] * case["D"], case["D"]
        if op == "norm_backward":
            return dict(bytes=n * (SIZES[case["h"]] + SIZES[case["dy"]] + 4 + 4 * case["dh"]) + 8 * D, flops=11 * n)
        scales = 4 * case["rows"] * -(-D // BLOCK) if case["y"] == "e4m3" else 0
        stream = 0 if case["first"] else 2 * SIZES[case["h"]]
        return dict(bytes=n * (SIZES[case["x"]] + SIZES[case["y"]] + stream) + scales + 4 * D, flops=6 * n)
    if op == "ortho":
        m, n = sorted((case["rows"], case["cols"]))
        # the products of a matrix with its own transpose, and of a symmetric one with itself, need one half
        return dict(bytes=case["n"] * m * n * (SIZES[case["dtype"]] + 2),
                    flops=case["n"] * STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n))
    B, C, e = case["B"], case["C"], SIZES[case["dtype"]]
    if op == "linear_step":
        return dict(bytes=B * C * (3 * e + 8) + 8 * C, flops=12 * B * C)
    live, all_ = sum(_lengths(case)) * C, B * case["T"] * C
    state = 4 * B * C
    if op == "linear_forward":
        return dict(bytes=e * (2 * live + all_) + state * (2 if case["h0"] else 1) + 8 * C, flops=12 * live)
    return dict(bytes=3 * e * live + 8 * all_ + 3 * state * case["h0"] + 16 * C, flops=24 * live)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _e4m3(v):
    """The nearest value of the format: 3 bits behind the leading one, exponents from -6, up to 448."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(exponent - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_norm(s):
    if s["op"] == "norm_forward":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = s["w"].double() * h / (h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt()
        out = dict(y=y) if s["residual"] is None else dict(h=h, y=y)
        if s["y"] is torch.float8_e4m3fn:
            parts = [p for p in y.split(BLOCK, 1)]
            scales = [(p.abs().max(1).values / 448.0).clamp(min=2.0 ** -126) for p in parts]
            out.update(y=torch.cat([_e4m3(p / c[:, None]) for p, c in zip(parts, scales)], 1), scale=torch.stack(scales, 1))
        return out
    h, w = s["h"].double().requires_grad_(), s["w"].double().requires_grad_()
    y = w * h / (h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt()
    loss = (y * s["dy"].double()).sum() + (0.0 if s["dh"] is None else (h * s["dh"].double()).sum())
    dx, dw = torch.autograd.grad(loss, [h, w])
    return dict(dx=dx, dw=dw)


def _exact_linear(s):
    """h_t = f_t h_{t-1} + (1 - f_t) x_t with f_t = exp(-alpha softplus(a_t + beta)), one step after another."""
    train = s["op"] == "linear_backward"
    names = ("x", "a", "alpha", "beta")
    p = {n: s[n].double().detach().requires_grad_(train) for n in names}
    if s["op"] == "linear_step":
        decay = -p["alpha"] * torch.nn.functional.softplus(p["a"] + p["beta"], threshold=40.0)
        H = torch.exp(decay) * s["H"].double() - torch.expm1(decay) * p["x"]
        return dict(y=H, H=H)
    B, T, C = s["x"].shape
    lens = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"]
    live = (torch.arange(T, device="cuda")[:, None] < lens)[..., None]  # [T,B,1]
    H_0 = s["H_0"].double() if s["H_0"] is not None else torch.zeros((B, C), dtype=torch.float64, device="cuda")
    H_0 = H_0.detach().requires_grad_(train)
    with torch.set_grad_enabled(train):
        decay = -p["alpha"] * torch.nn.functional.softplus(p["a"] + p["beta"], threshold=40.0)
        f, b = torch.exp(decay).unbind(1), (-torch.expm1(decay) * p["x"]).unbind(1)
        H, ys = H_0, []
        for t in range(T):
            H = torch.where(live[t], f[t] * H + b[t], H)
            ys.append(torch.where(live[t], H, 0.0))
        y = torch.stack(ys, 1)
        if not train:
            return dict(y=y, H_T=H)
        loss = (y * s["dy"].double()).sum() + (0.0 if s["dH_T"] is None else (H * s["dH_T"].double()).sum())
        g = torch.autograd.grad(loss, [p[n] for n in names] + [H_0])
    out = {"d" + n: v for n, v in zip(names, g)}
    return dict(out, dH_0=g[4]) if s["H_0"] is not None else out


def _exact_ortho(s):
    """The odd polynomial a t + b t^3 + c t^5 of a matrix over its norm, again and again."""
    a, b, c = COEFFICIENTS
    x = s["g"].double()
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + 1e-7)
    for _ in range(STEPS):
        if x.shape[1] <= x.shape[2]:
            xxx = torch.bmm(torch.bmm(x, x.mT), x)
            x = a * x + b * xxx + c * torch.bmm(torch.bmm(x, x.mT), xxx)
        else:
            xxx = torch.bmm(x, torch.bmm(x.mT, x))
            x = a * x + b * xxx + c * torch.bmm(xxx, torch.bmm(x.mT, x))
    return x


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["op"].split("_")[0]
    return {"norm": _exact_norm, "linear": _exact_linear, "ortho": _exact_ortho}[kind](s)
