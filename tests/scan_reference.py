"""The selective state space scan and its gradients in 64 bits, one step after
another over all sequences and heads at once (torch, on whatever device the
inputs are on), and the sizes of the sums that they are made of."""
import torch

NAMES = ("q", "k", "v", "dt", "A", "dt_bias", "w_r", "H_0", "dy", "dH_T")


def scan(d, lengths=None):
    """d: arrays by name, None where there is none.  Returns y, H_T and, where
    d has dy, the gradients, with g [B,T,N], the gradient of log a_t times D_t
    (dA summed over nothing)."""
    p = {n: None if d.get(n) is None else torch.as_tensor(d[n]).double() for n in NAMES}
    B, T, N, V = p["v"].shape
    G, K = p["q"].shape[2:]
    q, k = (p[n].repeat_interleave(N // G, 2) for n in ("q", "k"))
    v, dev = p["v"], p["v"].device
    x = p["dt"] if p["dt_bias"] is None else p["dt"] + p["dt_bias"]
    D = torch.logaddexp(x, torch.zeros_like(x))
    a = torch.exp(D * p["A"])
    wr = torch.zeros((N, V), dtype=torch.float64, device=dev) if p["w_r"] is None else p["w_r"]
    live = torch.ones((B, T), dtype=torch.bool, device=dev) if lengths is None else \
        torch.arange(T, device=dev) < torch.as_tensor(list(lengths), device=dev)[:, None]
    H = torch.zeros((B, N, K, V), dtype=torch.float64, device=dev) if p["H_0"] is None else p["H_0"].clone()
    on = lambda t, n: live[:, t].reshape((B,) + (1,) * n)  # noqa: E731
    states, y = [H], torch.zeros_like(v)
    for t in range(T):
        new = a[:, t, :, None, None] * H + (D[:, t, :, None] * k[:, t])[..., None] * v[:, t, :, None, :]
        H = torch.where(on(t, 3), new, H)
        y[:, t] = torch.where(on(t, 2), (q[:, t, :, None] @ H)[:, :, 0] + wr * v[:, t], 0.0)
        if p["dy"] is not None:
            states.append(H)
    out = dict(y=y, H_T=H)
    if p["dy"] is None:
        return out
    R = torch.zeros_like(H) if p["dH_T"] is None else p["dH_T"].clone()
    dq, dk, dv, ddt, g = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(D), torch.zeros_like(D)
    u, sg = p["dy"], torch.sigmoid(x)
    for t in range(T - 1, -1, -1):
        new = R + q[:, t, ..., None] * u[:, t, :, None, :]
        Rv, kR = (new @ v[:, t, ..., None])[..., 0], (k[:, t, :, None] @ new)[:, :, 0]
        gt = a[:, t] * (new * states[t]).sum((2, 3))
        dq[:, t] = torch.where(on(t, 2), (states[t + 1] @ u[:, t, ..., None])[..., 0], 0.0)
        dk[:, t] = torch.where(on(t, 2), D[:, t, :, None] * Rv, 0.0)
        dv[:, t] = torch.where(on(t, 2), D[:, t, :, None] * kR + wr * u[:, t], 0.0)
        ddt[:, t] = torch.where(on(t, 1), ((k[:, t] * Rv).sum(2) + p["A"] * gt) * sg[:, t], 0.0)
        g[:, t] = torch.where(on(t, 1), D[:, t] * gt, 0.0)
        R = torch.where(on(t, 3), a[:, t, :, None, None] * new, R)
    heads = lambda z: z.unflatten(2, (G, N // G)).sum(3)  # noqa: E731
    dwr = (torch.where(live[..., None, None], u * v, 0.0)).sum((0, 1))
    return dict(out, dq=heads(dq), dk=heads(dk), dv=dv, ddt=ddt, dA=g.sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dw_r=dwr,
                dH_0=R, g=g)


def sizes(d, lengths=None):
    """The same of the absolute values: the sums of the absolute values of
    everything that is added up (with A's sign kept where it is a decay)."""
    keep = ("dt", "A", "dt_bias")
    return scan({n: x if x is None or n in keep else torch.as_tensor(x).abs() for n, x in d.items()}, lengths)
