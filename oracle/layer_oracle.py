"""Float64 oracle of the hybrid layer's operators: plain loops over time, no
chunks, no fusion.  Test infrastructure only; shares no code with the CUDA
path.

  causal_conv       y_t = act(bias + sum_w w[:, w] xs[t + w]), xs = [x0 | x]
  ssm_scan          H_t = exp(D_t A) H_{t-1} + D_t k_t v_t^T,
                    y_t = H_t^T q_t + w_r v_t,  D_t = softplus(dt_t + dt_bias)
  clip              out = x min(1, max_norm / (norm + 1e-6))
and the backward of the first two from the chain rule.
"""
import numpy as np


def _sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def causal_conv(x, w, bias=None, x0=None, lengths=None, silu=True):
    """Returns y [B,T,C], x_T [B,W-1,C]."""
    B, T, C = x.shape
    W = w.shape[1]
    y, x_T = np.zeros((B, T, C)), np.zeros((B, W - 1, C))
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        xs = np.concatenate([np.zeros((W - 1, C)) if x0 is None else x0[b], x[b, :n]])
        for t in range(n):
            p = (w.T * xs[t:t + W]).sum(0) + (0.0 if bias is None else bias)
            y[b, t] = p * _sigmoid(p) if silu else p
        x_T[b] = xs[n:]
    return y, x_T


def causal_conv_backward(x, w, bias, dy, x0=None, dx_T=None, lengths=None, silu=True):
    """Returns dict(dx, dw, db, dx0) of sum(dy * y) + sum(dx_T * x_T)."""
    B, T, C = x.shape
    W = w.shape[1]
    out = dict(dx=np.zeros((B, T, C)), dw=np.zeros((C, W)), db=np.zeros(C), dx0=np.zeros((B, W - 1, C)))
    for b in range(B):
        n = T if lengths is None else int(lengths[b])
        xs = np.concatenate([np.zeros((W - 1, C)) if x0 is None else x0[b], x[b, :n]])
        d = np.zeros_like(xs)
        for t in range(n):
            g = dy[b, t]
            if silu:
                p = (w.T * xs[t:t + W]).sum(0) + (0.0 if bias is None else bias)
                s = _sigmoid(p)
                g = g * s * (1.0 + p * (1.0 - s))
            d[t:t + W] += w.T * g
            out["dw"] += (xs[t:t + W] * g).T
            out["db"] += g
        if dx_T is not None:
            d[n:] += dx_T[b]
        out["dx0"][b], out["dx"][b, :n] = d[:W - 1], d[W - 1:]
    return out


def _steps(dt, A, dt_bias):
    x = dt + (0.0 if dt_bias is None else dt_bias)
    D = np.logaddexp(x, 0.0)
    return D, np.exp(D * A), _sigmoid(x)


def ssm_scan(q, k, v, dt, A, dt_bias=None, w_r=None, H_0=None, lengths=None, all_states=False):
    """Returns y [B,T,N,V], H_T [B,N,K,V] (and H after every step)."""
    B, T, N, V = v.shape
    r = N // q.shape[2]
    q, k = np.repeat(q, r, 2), np.repeat(k, r, 2)
    D, a, _ = _steps(dt, A, dt_bias)
    H = np.zeros((B, N, q.shape[3], V)) if H_0 is None else np.array(H_0, np.float64)
    y, Hs = np.zeros((B, T, N, V)), [H.copy()]
    for t in range(T):
        for b in range(B):
            if lengths is not None and t >= lengths[b]:
                continue
            H[b] = a[b, t][:, None, None] * H[b] + D[b, t][:, None, None] * k[b, t][:, :, None] * v[b, t][:, None, :]
            y[b, t] = np.einsum("nk,nkv->nv", q[b, t], H[b]) + (0.0 if w_r is None else w_r * v[b, t])
        if all_states:
            Hs.append(H.copy())
    return (y, H, Hs) if all_states else (y, H)


def ssm_scan_backward(q, k, v, dt, A, dy, dt_bias=None, w_r=None, H_0=None, dH_T=None, lengths=None):
    """Gradients of sum(dy * y) + <dH_T, H_T>."""
    B, T, N, V = v.shape
    G, K = q.shape[2:]
    r = N // G
    _, _, Hs = ssm_scan(q, k, v, dt, A, dt_bias, w_r, H_0, lengths, all_states=True)
    qn, kn = np.repeat(q, r, 2), np.repeat(k, r, 2)
    D, a, sg = _steps(dt, A, dt_bias)
    dq, dk, dv, ddt = np.zeros((B, T, N, K)), np.zeros((B, T, N, K)), np.zeros((B, T, N, V)), np.zeros((B, T, N))
    dA, dwr = np.zeros(N), np.zeros((N, V))
    R = np.zeros((B, N, K, V)) if dH_T is None else np.array(dH_T, np.float64)
    for t in range(T - 1, -1, -1):
        for b in range(B):
            if lengths is not None and t >= lengths[b]:
                continue
            u = dy[b, t]
            R[b] += qn[b, t][:, :, None] * u[:, None, :]
            dq[b, t] = np.einsum("nkv,nv->nk", Hs[t + 1][b], u)
            Rv, kR = np.einsum("nkv,nv->nk", R[b], v[b, t]), np.einsum("nkv,nk->nv", R[b], kn[b, t])
            dk[b, t] = D[b, t][:, None] * Rv
            dv[b, t] = D[b, t][:, None] * kR + (0.0 if w_r is None else w_r * u)
            g = a[b, t] * np.einsum("nkv,nkv->n", R[b], Hs[t][b])
            ddt[b, t] = ((kn[b, t] * Rv).sum(1) + A * g) * sg[b, t]
            dA += D[b, t] * g
            dwr += u * v[b, t]
            R[b] *= a[b, t][:, None, None]
    return dict(dq=dq.reshape(B, T, G, r, K).sum(3), dk=dk.reshape(B, T, G, r, K).sum(3), dv=dv, ddt=ddt, dA=dA,
                ddt_bias=ddt.sum((0, 1)), dw_r=dwr, dH_0=R)


def clip(grads, max_norm):
    """Returns (norm, clipped gradients)."""
    norm = np.sqrt(sum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [np.asarray(g, np.float64) * c for g in grads]
