"""The hybrid layer's operators as they are measured: the short causal
convolution, the selective state space scan and gradient clipping.

Each case runs one pass of one operator.  With ``own`` false the pass is the
operator's plain form in elementary torch operations, in 32 bits, rounded once
at the end; with ``own`` true it is the call that a user makes of the library.
``exact`` is the operator's definition in 64 bits.

Layouts (the library's): x [B,T,C]; q, k [B,T,G,K] with G heads that divide
the N value heads; v, y [B,T,N,V]; dt [B,T,N]; states [B,N,K,V] and [B,W-1,C].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # steps per chunk of the plain scan


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # The q | k | v channels of a layer of 8 heads of 64 (the repository's training workload, B=4, T=4096),
        # convolved in one call on a column slice of the fused projection.
        dict(name="conv_prompt_4k", op="conv_forward", B=4, T=4096, C=1536, W=4, dtype="bf16", wide=520, ragged=False,
             x0=False),
        # A ragged batch of prompts that continue from a kept state, odd sizes, all in fp32.
        dict(name="conv_prompt_odd", op="conv_forward", B=5, T=1021, C=403, W=3, dtype="f32", wide=17, ragged=True,
             x0=True),
        # The training step's backward of the first case.
        dict(name="conv_train_4k", op="conv_backward", B=4, T=4096, C=1536, W=4, dtype="bf16", wide=520, ragged=False,
             x0=False),
        # One token for 32 sequences: a latency.
        dict(name="conv_step_32", op="conv_step", B=32, C=1536, W=4, dtype="bf16"),
        # The repository's 16K workload (B=2, 16 heads, 64 x 64 states) with one q and k shared by the heads: a long
        # prompt on few chains.
        dict(name="ssm_prompt_16k", op="ssm_forward", B=2, T=16384, N=16, G=1, K=64, V=64, dtype="bf16", ragged=False,
             h0=False),
        # Serving: a ragged batch (lengths 0 and 1 among them) with grouped heads of odd widths, from kept states.
        dict(name="ssm_prompt_ragged", op="ssm_forward", B=6, T=777, N=10, G=2, K=80, V=48, dtype="bf16", ragged=True,
             h0=True),
        # The repository's training workload's shape, one q and k per head.
        dict(name="ssm_train_4k", op="ssm_backward", B=4, T=4096, N=8, G=8, K=64, V=64, dtype="bf16", ragged=False,
             h0=False),
        # A small fp32 training run, as for a numerical check of a model: odd in every size.
        dict(name="ssm_train_odd", op="ssm_backward", B=2, T=301, N=3, G=1, K=33, V=17, dtype="f32", ragged=True,
             h0=True),
        # One token for the repository's 32 decoding states of 64 x 64: a latency.
        dict(name="ssm_step_32", op="ssm_step", B=4, N=8, G=1, K=64, V=64, dtype="bf16"),
        # One token for a large serving batch of wide heads: the states stream through.
        dict(name="ssm_step_2048", op="ssm_step", B=128, N=16, G=1, K=128, V=128, dtype="bf16"),
        # The gradients of one layer: a handful of tensors of both types, at odd offsets of one bucket.
        dict(name="clip_layer", op="clip", hidden=1024, layers=1, vocab=0, mixed=True, max_norm=1.0),
        # The gradients of a 410M dense model in fp32.
        dict(name="clip_410m", op="clip", hidden=1024, layers=24, vocab=32000, mixed=False, max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_forward", "conv_backward", "conv_step", "ssm_forward", "ssm_backward", "ssm_step", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip":
        return dict(op=op, hidden=16 * rng.randint(4, 40) + rng.choice([0, 0, 1, 7]), layers=_log_int(rng, 1, 24), vocab=rng.choice([0, 1000, 32000]),
                    mixed=rng.random() < 0.5, max_norm=rng.choice([0.5, 1.0, 1e9]))
    if op.startswith("conv"):
        C = _log_int(rng, 48, 2560)
        C = C if rng.random() < 0.4 else -(-C // 8) * 8
        W = rng.choice([2, 3, 4, 4])
        if op == "conv_step":
            return dict(op=op, B=_log_int(rng, 1, 512), C=C, W=W, dtype=dtype)
        T = _log_int(rng, 16, 16384)
        B = _log_int(rng, 1, 8)
        while B * T * C > 4 * 4096 * 1536:
            T = T // 2 + 1
        return dict(op=op, B=B, T=T, C=C, W=W, dtype=dtype, wide=rng.choice([0, 8, 520, 17]), ragged=rng.random() < 0.5,
                    x0=rng.random() < 0.5)
    N = rng.choice([1, 2, 4, 6, 8, 16])
    G = rng.choice([g for g in (1, 2, 4, 8, 16) if N % g == 0])
    if rng.random() < 0.6:
        K, V = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
    else:
        K, V = rng.randint(8, 128), rng.randint(8, 128)
    if op == "ssm_step":
        return dict(op=op, B=_log_int(rng, 1, 128), N=N, G=G, K=K, V=V, dtype=dtype)
    T = _log_int(rng, 16, 16384)
    B = _log_int(rng, 1, 8)
    most = (2 * 16 * 16384 * 64) if op == "ssm_forward" else (4 * 8 * 4096 * 64)
    while B * T * N * max(K, V) > most or (op == "ssm_backward" and T > 4096):
        T = T // 2 + 1
    return dict(op=op, B=B, T=T, N=N, G=G, K=K, V=V, dtype=dtype, ragged=rng.random() < 0.5, h0=rng.random() < 0.5)


def _lengths(case):
    """The lengths of a ragged batch: full, one, none, then spread out."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [(T, 1, 0)[b] if b < 3 else T * (b - 2) // (B - 1) for b in range(B)]


def _clip_shapes(case):
    h, f = case["hidden"], 4 * case["hidden"]
    shapes = [(case["vocab"], h)] if case["vocab"] else []
    for _ in range(case["layers"]):
        shapes += [(h,), (2 * h, h), (2 * h, 4), (2 * h,), (16,), (h // 16, h), (h, h), (h,), (2 * f, h), (h, f)]
    return shapes + [(h,)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _rand(gen, shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * scale if scale != 1.0 else x).to(dtype)


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _prepare_conv(case, gen):
    dt = DTYPES[case["dtype"]]
    B, C, W = case["B"], case["C"], case["W"]
    s = dict(w=_rand(gen, (C, W), dt, W ** -0.5), b=_rand(gen, (C,), dt, 0.1))
    if case["op"] == "conv_step":
        return dict(s, state=_rand(gen, (B, W - 1, C), dt), x=_rand(gen, (B, C), dt),
                    y=torch.empty((B, C), device="cuda", dtype=dt))
    T = case["T"]
    s["x"] = _rand(gen, (B, T, C + case["wide"]), dt)[..., :C]  # a column slice of a wider projection
    s["x0"] = _rand(gen, (B, W - 1, C), dt) if case["x0"] else None
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"] == "conv_backward":
        s["dy"] = _rand(gen, (B, T, C))
        s["dx_T"] = _rand(gen, (B, W - 1, C)) if case["x0"] else None
    return s


def _prepare_ssm(case, gen):
    dt = DTYPES[case["dtype"]]
    B, N, G, K, V = (case[n] for n in ("B", "N", "G", "K", "V"))
    A = -(1.0 + 15.0 * torch.rand((N,), generator=gen, device="cuda"))
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((N,), generator=gen, device="cuda"))
    s = dict(A=A, dt_bias=torch.log(torch.expm1(step)), w_r=_rand(gen, (N, V), dt))
    rows = (B,) if case["op"] == "ssm_step" else (B, case["T"])
    # v | k | q side by side, as the convolution leaves them
    z = _silu(_rand(gen, rows + (N * V + 2 * G * K,))).to(dt)
    s["v"] = z[..., :N * V].unflatten(-1, (N, V))
    s["k"] = z[..., N * V:N * V + G * K].unflatten(-1, (G, K))
    s["q"] = z[..., N * V + G * K:].unflatten(-1, (G, K))
    s["dt"] = _rand(gen, rows + (N,), dt)
    if case["op"] == "ssm_step":
        return dict(s, H=_rand(gen, (B, N, K, V), scale=0.5), y=torch.empty((B, N, V), device="cuda", dtype=dt))
    s["H_0"] = _rand(gen, (B, N, K, V), scale=0.5) if case["h0"] else None
    s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"] == "ssm_backward":
        s["dy"] = _rand(gen, (B, case["T"], N, V), dt)
        s["dH_T"] = _rand(gen, (B, N, K, V)) if case["h0"] else None
    return s


def _prepare_clip(case, gen):
    shapes = _clip_shapes(case)
    # Gradients lie one after another in a bucket of each type, the clipped ones in another.
    kinds = [torch.bfloat16 if case["mixed"] and len(sh) == 2 and sh[1] > 4 else torch.float32 for sh in shapes]
    flat, clipped, at = {}, {}, {}
    for kind in sorted(set(kinds), key=str):
        n = sum(math.prod(sh) for sh, k in zip(shapes, kinds) if k == kind)
        flat[kind] = _rand(gen, (n,), kind, 0.01)
        clipped[kind] = torch.empty(n, device="cuda", dtype=kind)
        at[kind] = 0
    grads, outs = [], []
    for sh, kind in zip(shapes, kinds):
        n, o = math.prod(sh), at[kind]
        grads.append(flat[kind][o:o + n].view(sh))
        outs.append(clipped[kind][o:o + n].view(sh))
        at[kind] = o + n
    s = dict(grads=grads, buckets={str(k): v for k, v in flat.items()}, clipped={str(k): v for k, v in clipped.items()},
             max_norm=case["max_norm"])
    if own:  # the handle that a program keeps for its gradient buffers
        from matrix_state_non_gb300 import binding
        s["plan"] = binding.grad_plan(grads, out=outs)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["op"].split("_")[0]
    return dict({"conv": _prepare_conv, "ssm": _prepare_ssm, "clip": _prepare_clip}[kind](case, gen), op=case["op"])


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _valid(lengths, T):
    """[B,T]: whether a step lies in its sequence; None = all do."""
    return None if lengths is None else torch.arange(T, device="cuda") < lengths[:, None]


def _keep(x, valid):
    return x if valid is None else torch.where(valid.reshape(valid.shape + (1,) * (x.dim() - 2)), x, 0.0)


def _conv_pre(s):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    B, T, C = x.shape
    W = w.shape[1]
    valid = _valid(s["lengths"], T)
    x0 = s["x0"].float() if s["x0"] is not None else x.new_zeros((B, W - 1, C))
    xs = torch.cat([x0, _keep(x, valid)], 1)
    pre = (xs.unfold(1, W, 1) * w).sum(-1) + b
    last = T if s["lengths"] is None else s["lengths"].long()[:, None]
    at = (last + torch.arange(W - 1, device="cuda")).expand(B, W - 1)[..., None].expand(B, W - 1, C)
    return xs, pre, valid, at


def _conv_forward(s):
    xs, pre, valid, at = _conv_pre(s)
    return dict(y=_keep(_silu(pre), valid).to(s["x"].dtype), x_T=xs.gather(1, at).to(s["x"].dtype))


def _conv_backward(s):
    xs, pre, valid, at = _conv_pre(s)
    w = s["w"].float()
    W = w.shape[1]
    sg = 1.0 / (1.0 + torch.exp(-pre))
    g = _keep(s["dy"] * sg * (1.0 + pre * (1.0 - sg)), valid)
    edge = g.new_zeros((g.shape[0], W - 1, g.shape[2]))
    dxs = (torch.cat([edge, g, edge], 1).unfold(1, W, 1) * w.flip(1)).sum(-1)
    if s["dx_T"] is not None:
        dxs = dxs.scatter_add(1, at, s["dx_T"])
    out = dict(dx=dxs[:, W - 1:], dw=(xs.unfold(1, W, 1) * g[..., None]).sum((0, 1)), db=g.sum((0, 1)))
    if s["x0"] is not None:
        out["dx0"] = dxs[:, :W - 1]
    return out


def _conv_step(s):
    xs = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (xs.float() * s["w"].float().t()).sum(1) + s["b"].float()
    s["state"].copy_(xs[:, 1:])
    return dict(y=_silu(pre).to(s["x"].dtype), state=s["state"])


def _segsum(x):
    """E[..., i, j] = exp(sum of x[j+1..i]) for i >= j, else 0: sums of differences only, so nothing cancels."""
    n = x.shape[-1]
    low = torch.ones((n, n), dtype=torch.bool, device=x.device).tril(-1)
    d = torch.where(low, x[..., :, None], 0.0).cumsum(-2)
    return torch.where(low | torch.eye(n, dtype=torch.bool, device=x.device), torch.exp(d), 0.0)


def _chunked(x, N, nc):
    """[B,T,heads,...] -> [B,N,nc,CHUNK,...] in fp32, heads repeated to N, the steps padded with zeros."""
    x = x.float()
    if x.dim() == 4:
        x = x.repeat_interleave(N // x.shape[2], 2)
    pad = nc * CHUNK - x.shape[1]
    x = torch.cat([x, x.new_zeros((x.shape[0], pad) + x.shape[2:])], 1) if pad else x
    return x.unflatten(1, (nc, CHUNK)).movedim(3, 1)


def _scan_parts(s):
    """The pieces that the scan and its backward share, a chunk of CHUNK steps at a time."""
    B, T, N, V = s["v"].shape
    nc = -(-T // CHUNK)
    valid = _valid(s["lengths"], T)
    x = s["dt"].float() + s["dt_bias"]
    D = _chunked(_keep(torch.logaddexp(x, torch.zeros_like(x)), valid), N, nc)        # [B,N,nc,L]
    q, k, v = (_chunked(_keep(s[n].float(), valid), N, nc) for n in ("q", "k", "v"))
    la = D * s["A"][:, None, None]
    E = _segsum(la)
    first = torch.exp(la.cumsum(-1))                                                  # chunk start -> step
    last = E[..., -1, :]                                                              # step -> chunk end
    K = q.shape[-1]
    H_0 = s["H_0"] if s["H_0"] is not None else v.new_zeros((B, N, K, V))
    U = (k * (last * D)[..., None]).transpose(-1, -2) @ v                             # [B,N,nc,K,V]
    tot = la.sum(-1)
    Ec = _segsum(torch.cat([torch.zeros_like(tot[..., :1]), tot], -1))                # [B,N,nc+1,nc+1]
    states = (Ec @ torch.cat([H_0[:, :, None], U], 2).flatten(-2)).unflatten(-1, (K, V))
    return x, valid, D, q, k, v, E, first, last, Ec, states


def _steps(x, T):
    """[B,N,nc,L,...] -> [B,T,N,...]"""
    return x.movedim(1, 3).flatten(1, 2)[:, :T]


def _ssm_forward(s):
    T = s["v"].shape[1]
    x, valid, D, q, k, v, E, first, last, Ec, states = _scan_parts(s)
    P = (q @ k.transpose(-1, -2)) * E * D[..., None, :]
    y = P @ v + first[..., None] * (q @ states[:, :, :-1]) + s["w_r"].float()[:, None, None] * v
    return dict(y=_keep(_steps(y, T), valid).to(s["v"].dtype), H_T=states[:, :, -1].contiguous())


def _ssm_backward(s):
    B, T, N, V = s["v"].shape
    G = s["q"].shape[2]
    x, valid, D, q, k, v, E, first, last, Ec, states = _scan_parts(s)
    u = _chunked(_keep(s["dy"].float(), valid), N, states.shape[2] - 1)
    S, K = states[:, :, :-1], q.shape[-1]
    # Gradients of the states at the chunk boundaries, from the later chunks and dH_T.
    Ru = (q * first[..., None]).transpose(-1, -2) @ u
    dH_T = s["dH_T"] if s["dH_T"] is not None else v.new_zeros((B, N, K, V))
    R = (Ec.transpose(-1, -2) @ torch.cat([Ru, dH_T[:, :, None]], 2).flatten(-2)).unflatten(-1, (K, V))
    Rn = R[:, :, 1:]
    P = (q @ k.transpose(-1, -2)) * E
    dP = (u @ v.transpose(-1, -2)) * E
    dq = (dP * D[..., None, :]) @ k + first[..., None] * (u @ S.transpose(-1, -2))
    zk = dP.transpose(-1, -2) @ q + last[..., None] * (v @ Rn.transpose(-1, -2))
    zv = P.transpose(-1, -2) @ u + last[..., None] * (k @ Rn)
    dk, dv = D[..., None] * zk, D[..., None] * zv + s["w_r"].float()[:, None, None] * u
    # g_t, the gradient of log a_t: everything that crosses from steps < t to steps >= t.
    c = (k * zk).sum(-1)
    end = (R[:, :, 1:] * states[:, :, 1:]).sum((-1, -2))
    g = ((q * dq).sum(-1) - D * c).flip(-1).cumsum(-1).flip(-1) + end[..., None]
    dD, g, D = (_keep(_steps(z, T), valid) for z in (c + s["A"][:, None, None] * g, g, D))
    ddt = dD / (1.0 + torch.exp(-x))
    group = lambda z: _steps(z, T).unflatten(2, (G, N // G)).sum(3)  # noqa: E731
    out = dict(dq=group(dq), dk=group(dk), dv=_steps(dv, T).contiguous(), ddt=ddt, dA=(D * g).sum((0, 1)),
               ddt_bias=ddt.sum((0, 1)), dw_r=(u * v).sum((0, 2, 3)))
    if s["H_0"] is not None:
        out["dH_0"] = R[:, :, 0].contiguous()
    return out


def _ssm_step(s):
    N, G = s["v"].shape[1], s["q"].shape[1]
    x = s["dt"].float() + s["dt_bias"]
    D = torch.logaddexp(x, torch.zeros_like(x))
    q, k = (s[n].float().repeat_interleave(N // G, 1) for n in ("q", "k"))
    v, H = s["v"].float(), s["H"]
    H.mul_(torch.exp(D * s["A"])[..., None, None]).add_((D[..., None] * k)[..., None] * v[..., None, :])
    y = (H * q[..., None]).sum(2) + s["w_r"].float() * v
    return dict(y=y.to(s["v"].dtype), H=H)


def _clip(s):
    # on the buckets that the tensors lie in, one after another: few and large operations
    norm = sum(g.float().square().sum() for g in s["buckets"].values()).sqrt()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return dict(norm=norm, clipped={n: s["clipped"][n].copy_(g.float() * coef) for n, g in s["buckets"].items()})


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(s):
    from matrix_state_non_gb300 import binding as m
    op = s["op"]
    if op == "conv_forward":
        r = m.causal_conv(s["x"], s["w"], s["b"], x0=s["x0"], lengths=s["lengths"], want_state=True)
        return dict(y=r["y"], x_T=r["x_T"])
    if op == "conv_backward":
        r = m.causal_conv_backward(s["x"], s["w"], s["b"], s["dy"], x0=s["x0"], dx_T=s["dx_T"], lengths=s["lengths"],
                                   want_dx0=s["x0"] is not None)
        return {n: r[n] for n in ("dx", "dw", "db", "dx0") if n in r}
    if op == "conv_step":
        return dict(y=m.causal_conv_step(s["state"], s["x"], s["w"], s["b"], y=s["y"]), state=s["state"])
    if op == "ssm_forward":
        r = m.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], w_r=s["w_r"], H_0=s["H_0"],
                       lengths=s["lengths"])
        return dict(y=r["y"], H_T=r["H_T"])
    if op == "ssm_backward":
        r = m.ssm_scan_backward(s["q"], s["k"], s["v"], s["dt"], s["A"], s["dy"], dt_bias=s["dt_bias"], w_r=s["w_r"],
                                H_0=s["H_0"], dH_T=s["dH_T"], lengths=s["lengths"], want_dH0=s["H_0"] is not None)
        return {n: r[n] for n in ("dq", "dk", "dv", "ddt", "dA", "ddt_bias", "dw_r", "dH_0") if n in r}
    if op == "ssm_step":
        y = m.ssm_step(s["H"], s["q"], s["k"], s["v"], s["dt"], s["A"], dt_bias=s["dt_bias"], w_r=s["w_r"], y=s["y"])
        return dict(y=y, H=s["H"])
    return dict(norm=m.grad_clip(s["plan"], s["max_norm"]), clipped=s["clipped"])


PLAIN = dict(conv_forward=_conv_forward, conv_backward=_conv_backward, conv_step=_conv_step, ssm_forward=_ssm_forward,
             ssm_backward=_ssm_backward, ssm_step=_ssm_step, clip=_clip)


@torch.no_grad()
def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "clip":
        n = [(math.prod(sh), 2 if case["mixed"] and len(sh) == 2 and sh[1] > 4 else 4) for sh in _clip_shapes(case)]
        return dict(bytes=sum(2 * a * e for a, e in n), flops=sum(3 * a for a, _ in n))
    B, e = case["B"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        weights, state = C * (W + 1), B * (W - 1) * C
        if op == "conv_step":
            return dict(bytes=e * (2 * B * C + 2 * state + weights), flops=B * C * (2 * W + 4))
        live, rows = sum(_lengths(case)) * C, B * case["T"] * C
        states = (2 if case["x0"] else 1) * state
        if op == "conv_forward":
            return dict(bytes=e * (live + rows + states + weights), flops=live * (2 * W + 4))
        return dict(bytes=live * (e + 4) + 4 * rows + e * weights + 4 * weights + (e + 8) * state * case["x0"],
                    flops=live * (6 * W + 10))
    N, G, K, V = (case[n] for n in ("N", "G", "K", "V"))
    token, state = 2 * G * K + 2 * N * V + N, 4 * B * N * K * V
    if op == "ssm_step":
        return dict(bytes=e * (B * token + N * V) + 2 * state + 8 * N, flops=5 * B * N * K * V)
    live, rows = sum(_lengths(case)), B * case["T"]
    if op == "ssm_forward":
        return dict(bytes=e * (live * (2 * G * K + N * V + N) + rows * N * V + N * V) + 8 * N
                    + state * (2 if case["h0"] else 1), flops=4 * live * N * K * V)
    grads = 4 * (rows * (2 * G * K + N * V + N) + N * V + 2 * N)
    return dict(bytes=e * live * token + grads + e * N * V + 8 * N + 3 * state * case["h0"], flops=10 * live * N * K * V)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_conv(s):
    """y_t = silu(b + sum over w of w[:, w] x_{t - W + 1 + w}), step by step on each sequence."""
    x, w, b = (s[n].double().detach().requires_grad_() for n in ("x", "w", "b"))
    B, T, C = x.shape
    W = w.shape[1]
    x0 = (s["x0"].double() if s["x0"] is not None else x.new_zeros((B, W - 1, C))).detach().requires_grad_()
    lens = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    ys, ends = [], []
    for i in range(B):
        xs = torch.cat([x0[i], x[i, :lens[i]]])
        pre = b.expand(lens[i], C)
        for j in range(W):
            pre = pre + xs[j:j + lens[i]] * w[:, j]
        ys.append(torch.cat([pre * torch.sigmoid(pre), x.new_zeros((T - lens[i], C))]))
        ends.append(xs[lens[i]:])
    y, x_T = torch.stack(ys), torch.stack(ends)
    if s["op"] == "conv_forward":
        return dict(y=y.detach(), x_T=x_T.detach())
    loss = (y * s["dy"].double()).sum() + ((x_T * s["dx_T"].double()).sum() if s["dx_T"] is not None else 0.0)
    g = torch.autograd.grad(loss, [x, w, b, x0])
    out = dict(dx=g[0], dw=g[1], db=g[2])
    return dict(out, dx0=g[3]) if s["x0"] is not None else out


def _exact_recurrence(q, k, v, D, A, w_r, H, live):
    """H_t = exp(D_t A) H_{t-1} + D_t k_t v_t^T and y_t = H_t^T q_t + w_r v_t, one step after another."""
    ys = []
    for t in range(v.shape[1]):
        a = torch.exp(D[:, t] * A)[..., None, None]
        new = a * H + (D[:, t, :, None] * k[:, t])[..., None] * v[:, t, :, None, :]
        H = torch.where(live[:, t, None, None, None], new, H)
        y = (q[:, t, :, None, :] @ H).squeeze(-2) + w_r * v[:, t]
        ys.append(torch.where(live[:, t, None, None], y, 0.0))
    return torch.stack(ys, 1), H


def _exact_ssm(s):
    B, T, N, V = s["v"].shape
    K, G = s["q"].shape[-1], s["q"].shape[2]
    train = s["op"] == "ssm_backward"
    live = torch.arange(T, device="cuda") < (s["lengths"][:, None] if s["lengths"] is not None
                                             else torch.full((B, 1), T, device="cuda"))
    if train and T * B * N * K * V * 8 * 5 > 60e9:
        return None
    names = ("q", "k", "v", "dt", "A", "dt_bias", "w_r")
    p = {n: s[n].double().detach().requires_grad_(train) for n in names}
    H_0 = s["H_0"].double() if s["H_0"] is not None else torch.zeros((B, N, K, V), dtype=torch.float64, device="cuda")
    H_0 = H_0.detach().requires_grad_(train)
    with torch.set_grad_enabled(train):
        D = torch.nn.functional.softplus(p["dt"] + p["dt_bias"], threshold=40.0)
        q, k = (p[n].repeat_interleave(N // G, 2) for n in ("q", "k"))
        y, H = _exact_recurrence(q, k, p["v"], D, p["A"], p["w_r"], H_0, live)
        if not train:
            return dict(y=y, H_T=H)
        loss = (y * s["dy"].double()).sum() + ((H * s["dH_T"].double()).sum() if s["dH_T"] is not None else 0.0)
        g = dict(zip(names + ("H_0",), torch.autograd.grad(loss, [p[n] for n in names] + [H_0])))
    return {"d" + n: g[n] for n in names + (("H_0",) if s["H_0"] is not None else ())}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(sum(float(g.double().square().sum()) for g in s["grads"]))
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        flat = {}
        for g in s["grads"]:
            flat.setdefault(str(g.dtype), []).append(g.flatten().double() * c)
        return dict(norm=torch.tensor(norm, dtype=torch.float64, device="cuda"),
                    clipped={n: torch.cat(v) for n, v in flat.items()})
    if op == "conv_step":
        xs = torch.cat([s["state"].double(), s["x"].double()[:, None]], 1)
        pre = torch.einsum("bwc,cw->bc", xs, s["w"].double()) + s["b"].double()
        return dict(y=pre * torch.sigmoid(pre), state=xs[:, 1:])
    if op.startswith("conv"):
        return _exact_conv(s)
    if op == "ssm_step":
        D = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=40.0)
        r = s["v"].shape[1] // s["q"].shape[1]
        live = torch.ones((case["B"], 1), dtype=torch.bool, device="cuda")
        y, H = _exact_recurrence(*(s[n].double().repeat_interleave(r, 1)[:, None] for n in ("q", "k")),
                                 s["v"].double()[:, None], D[:, None], s["A"].double(), s["w_r"].double(),
                                 s["H"].double(), live)
        return dict(y=y[:, 0], H=H)
    return _exact_ssm(s)
