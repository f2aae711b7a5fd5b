"""Float64 oracle of the operators around the layers: plain formulas, a loop
over time.  Test infrastructure only; shares no code with the CUDA path.

  residual_norm   h = x + r,  y = w h / sqrt(mean(h^2) + eps)
  linear_scan     h_t = f_t h_{t-1} + (1 - f_t) x_t,  f_t = exp(-alpha softplus(a_t + beta))
  orthogonalize   X = G / (|G| + eps),  X <- a X + (b A + c A A) X,  A = X X^T
and the backward of the first two from the chain rule.
"""
import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def residual_norm(x, w, residual=None, eps=1e-6):
    """Returns y, h."""
    h = x if residual is None else x + residual
    return w * h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps), h


def residual_norm_backward(h, w, dy, dh=None, eps=1e-6):
    """Gradients dx, dw of sum(dy * y) + sum(dh * h)."""
    s = 1.0 / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    p = w * dy
    dx = s * p - h * s ** 3 * np.mean(p * h, -1, keepdims=True) + (0.0 if dh is None else dh)
    return dx, (dy * h * s).reshape(-1, h.shape[-1]).sum(0)


def e4m3(v):
    """The nearest 8-bit value (3 bits behind the leading one, exponents from -6, at most 448), ties to even."""
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -20))), -6.0) - 3.0)
    return np.clip(np.round(v / step) * step, -448.0, 448.0)


def quantize(y, block=128):
    """Returns the stored values and their scales, one for each `block` of the last axis."""
    parts = [y[..., i:i + block] for i in range(0, y.shape[-1], block)]
    scale = np.stack([np.maximum(np.abs(p).max(-1) / 448.0, 2.0 ** -126) for p in parts], -1)
    return np.concatenate([e4m3(p / scale[..., i:i + 1]) for i, p in enumerate(parts)], -1), scale


def _gate(a, alpha, beta):
    z = a + (0.0 if beta is None else beta)
    soft = np.logaddexp(z, 0.0)
    return soft, np.exp(-alpha * soft), -np.expm1(-alpha * soft), 0.5 * (1.0 + np.tanh(0.5 * z))


def linear_scan(x, a, alpha, beta=None, H_0=None, lengths=None, all_states=False):
    """Returns y [B,T,C], H_T [B,C] (and the states before the first and after every step)."""
    B, T, C = x.shape
    _, f, e, _ = _gate(a, alpha, beta)
    H = np.zeros((B, C)) if H_0 is None else np.array(H_0, np.float64)
    y, states = np.zeros((B, T, C)), [H.copy()]
    for t in range(T):
        live = np.full((B, 1), True) if lengths is None else (t < np.asarray(lengths))[:, None]
        H = np.where(live, f[:, t] * H + e[:, t] * x[:, t], H)
        y[:, t] = np.where(live, H, 0.0)
        states.append(H.copy())
    return (y, H, states) if all_states else (y, H)


def linear_scan_backward(x, a, alpha, beta, dy, H_0=None, dH_T=None, lengths=None):
    """Gradients of sum(dy * y) + <dH_T, H_T>."""
    B, T, C = x.shape
    _, _, states = linear_scan(x, a, alpha, beta, H_0, lengths, all_states=True)
    soft, f, e, sig = _gate(a, alpha, beta)
    carry = np.zeros((B, C)) if dH_T is None else np.array(dH_T, np.float64)
    dx, da, dalpha = np.zeros((B, T, C)), np.zeros((B, T, C)), np.zeros(C)
    for t in range(T - 1, -1, -1):
        live = np.full((B, 1), True) if lengths is None else (t < np.asarray(lengths))[:, None]
        dh = np.where(live, dy[:, t] + carry, 0.0)
        g = dh * f[:, t] * (states[t] - x[:, t])
        dx[:, t], da[:, t] = e[:, t] * dh, -alpha * sig[:, t] * g
        dalpha -= (soft[:, t] * g).sum(0)
        carry = np.where(live, f[:, t] * dh, carry)
    return dict(dx=dx, da=da, dalpha=dalpha, dbeta=da.sum((0, 1)), dH_0=carry)


def orthogonalize(g, steps=5, eps=1e-7):
    """g [..., rows, columns], from the singular values: each goes through the polynomial on its own."""
    a, b, c = COEFFICIENTS
    g = np.asarray(g, np.float64)
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((g * g).sum((-2, -1), keepdims=True))[..., 0] + eps)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return (u * s[..., None, :]) @ v
