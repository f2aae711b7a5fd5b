"""Inputs and comparisons of the hybrid layer's tests: seeded numpy arrays that
are exact in the type they are uploaded in."""
import numpy as np


def round_to(x, dtype):
    """float64 -> the float64 values that `dtype` ("bf16" | "f32") holds."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).float()
    return (t.bfloat16() if dtype == "bf16" else t).double().numpy()


def dev(x, dtype="f32"):
    import torch
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).float()
    return (t.bfloat16() if dtype == "bf16" else t).cuda()


def ints(x):
    import torch
    return None if x is None else torch.tensor(list(x), dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def conv_inputs(B, T, C, W, dtype, seed, x0=False, bias=True):
    r = np.random.default_rng(seed)
    d = dict(x=r.normal(size=(B, T, C)), w=r.normal(size=(C, W)) / np.sqrt(W))
    d["bias"] = 0.3 * r.normal(size=C) if bias else None
    d["x0"] = r.normal(size=(B, W - 1, C)) if x0 else None
    d = {n: None if a is None else round_to(a, dtype) for n, a in d.items()}
    d["dy"], d["dx_T"] = round_to(r.normal(size=(B, T, C)), "f32"), round_to(r.normal(size=(B, W - 1, C)), "f32")
    return d


def ssm_inputs(B, T, N, G, K, V, dtype, seed, h0=True, decay=None):
    """q, k, v positive on average, as after SiLU; steps between 1e-3 and 0.1
    around which dt moves; A in [-16, -1] (or `decay`)."""
    r = np.random.default_rng(seed)

    def silu(*shape):
        x = r.normal(size=shape)
        return x / (1.0 + np.exp(-x))

    d = dict(q=silu(B, T, G, K), k=silu(B, T, G, K), v=silu(B, T, N, V), dt=r.normal(size=(B, T, N)),
             w_r=r.normal(size=(N, V)), dy=r.normal(size=(B, T, N, V)))
    d = {n: round_to(a, dtype) for n, a in d.items()}
    d["A"] = round_to(-r.uniform(1, 16, N) if decay is None else np.full(N, decay), "f32")
    d["dt_bias"] = round_to(np.log(np.expm1(np.exp(r.uniform(np.log(1e-3), np.log(0.1), N)))), "f32")
    d["H_0"] = round_to(0.5 * r.normal(size=(B, N, K, V)), "f32") if h0 else None
    d["dH_T"] = round_to(r.normal(size=(B, N, K, V)), "f32") if h0 else None
    return d


SSM_IN = ("q", "k", "v", "dt", "A")
SSM_OPT = ("dt_bias", "w_r", "H_0")
SSM_TYPED = ("q", "k", "v", "dt", "w_r", "dy")


def ssm_dev(d, dtype):
    return {n: dev(a, dtype if n in SSM_TYPED else "f32") for n, a in d.items()}
