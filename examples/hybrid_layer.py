"""A hybrid layer trained and served with the library's operators.

One residual layer of a language model's mixer, as in hybrid models that
put selective state space layers beside the matrix-state recurrence:

    in-projection -> short causal convolution + SiLU -> selective state space
    scan -> gated RMS norm -> out-projection -> residual

``train`` runs steps on a synthetic task (forward, backward, global gradient
clipping, SGD); ``serve`` takes a ragged batch of prompts through the layer and
continues each one token at a time from the states the prompts left.  The
projections are plain matrix products; everything between them, and the
clipping, runs in the library's kernels.

    python examples/hybrid_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from matrix_state_non_gb300 import binding as m  # noqa: E402


class HybridLayer:
    """Weights of one layer: D channels, N value heads of V, G shared q/k heads
    of K, convolution width W.  bf16 weights, fp32 gate parameters."""

    def __init__(self, D=256, N=8, G=1, K=64, V=64, W=4, seed=0, device="cuda"):
        self.D, self.N, self.G, self.K, self.V, self.W = D, N, G, K, V, W
        self.C = N * V + 2 * G * K  # v | k | q, convolved together
        gen = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, scale):
            return (scale * torch.randn(shape, generator=gen, device=device)).bfloat16()

        step = torch.logspace(-3, -1, N, device=device)
        self.p = dict(
            w_in=rand(D, self.C + N * V + N, scale=D ** -0.5), w_out=rand(N * V, D, scale=(N * V) ** -0.5),
            conv_w=rand(self.C, W, scale=W ** -0.5), conv_b=rand(self.C, scale=0.1), w_r=rand(N, V, scale=1.0),
            A=-torch.linspace(1, 16, N, device=device), dt_bias=torch.log(torch.expm1(step)),
            norm_w=torch.ones((N, V), device=device))

    def _split(self, z, h):
        """Projection -> gate, dt; convolved channels -> q, k, v (views)."""
        N, G, K, V, C = self.N, self.G, self.K, self.V, self.C
        v, k, q = h[..., :N * V], h[..., N * V:N * V + G * K], h[..., N * V + G * K:]
        gate, dt = z[..., C:C + N * V].unflatten(-1, (N, V)), z[..., C + N * V:]
        return q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (N, V)), dt, gate.contiguous()

    def forward(self, x, lengths=None, conv_state=None, H=None):
        """x [B,T,D] bf16.  Returns the layer's output and what the backward and
        the next piece of the sequences need."""
        p = self.p
        z = x @ p["w_in"]
        c = m.causal_conv(z[..., :self.C], p["conv_w"], p["conv_b"], x0=conv_state, lengths=lengths, want_state=True)
        q, k, v, dt, gate = self._split(z, c["y"])
        s = m.ssm_scan(q, k, v, dt, p["A"], dt_bias=p["dt_bias"], w_r=p["w_r"], H_0=H, lengths=lengths)
        y = s["y"].float()
        o = m.output_norm(y, gate, p["norm_w"])
        out = x + o.flatten(2).bfloat16() @ p["w_out"]
        return out, dict(x=x, z=z, h=c["y"], y=y, o=o, conv_state=c["x_T"], H=s["H_T"])

    def backward(self, saved, dout):
        """Gradients of every weight, given the output's gradient [B,T,D]."""
        p, N, V = self.p, self.N, self.V
        q, k, v, dt, gate = self._split(saved["z"], saved["h"])
        flat = lambda t: t.flatten(0, 1)  # noqa: E731
        g = dict(w_out=flat(saved["o"].flatten(2).bfloat16()).t() @ flat(dout))
        do = (dout @ p["w_out"].t()).float().unflatten(-1, (N, V))
        n = m.output_norm_backward(saved["y"], gate, p["norm_w"], do)
        g["norm_w"] = n["dw"]
        s = m.ssm_scan_backward(q, k, v, dt, p["A"], n["dy"].bfloat16(), dt_bias=p["dt_bias"], w_r=p["w_r"])
        g.update(A=s["dA"], dt_bias=s["ddt_bias"], w_r=s["dw_r"])
        dh = torch.cat([s[i].flatten(2) for i in ("dv", "dk", "dq")], -1)
        c = m.causal_conv_backward(saved["z"][..., :self.C], p["conv_w"], p["conv_b"], dh)
        g.update(conv_w=c["dw"], conv_b=c["db"])
        dz = torch.cat([c["dx"], n["dg"].flatten(2), s["ddt"]], -1).bfloat16()
        g["w_in"] = flat(saved["x"]).t() @ flat(dz)
        return g

    def step(self, x, conv_state, H):
        """One token for every sequence: x [B,D]; both states advance in place."""
        p = self.p
        z = x @ p["w_in"]
        h = m.causal_conv_step(conv_state, z[:, :self.C], p["conv_w"], p["conv_b"])
        q, k, v, dt, gate = self._split(z, h)
        y = m.ssm_step(H, q, k, v, dt, p["A"], dt_bias=p["dt_bias"], w_r=p["w_r"])
        o = m.output_norm(y.float()[:, None], gate[:, None], p["norm_w"])
        return x + o.flatten(1).bfloat16() @ p["w_out"]


def train(layer, steps=20, B=4, T=512, lr=1.0, max_norm=1.0, seed=1):
    """Fits a fixed random target; returns the losses and the gradient norms."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((B, T, layer.D), generator=gen, device="cuda").bfloat16()
    target = torch.randn((B, T, layer.D), generator=gen, device="cuda")
    names = sorted(layer.p)
    grads = {n: torch.empty_like(layer.p[n], dtype=torch.float32) for n in names}  # one buffer each, for all steps
    plan = m.grad_plan([grads[n] for n in names])
    losses, norms = [], []
    for _ in range(steps):
        out, saved = layer.forward(x)
        diff = out.float() - target
        losses.append(diff.square().mean())
        for n, g in layer.backward(saved, (2.0 / diff.numel() * diff).bfloat16()).items():
            grads[n].copy_(g)
        norms.append(m.grad_clip(plan, max_norm))
        for n in names:
            layer.p[n] -= (lr * grads[n]).to(layer.p[n].dtype)
    return [float(v) for v in losses], [float(v) for v in norms]


def serve(layer, lengths=(37, 1, 130, 64), tokens=4, seed=2):
    """Prompts of several lengths, then `tokens` more of each: returns the
    outputs [B,tokens,D] and those of the same tokens run in one piece."""
    B, T = len(lengths), max(lengths)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((B, T + tokens, layer.D), generator=gen, device="cuda").bfloat16()
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    _, saved = layer.forward(x[:, :T].contiguous(), lengths=lens)
    conv_state, H = saved["conv_state"], saved["H"]
    rows = torch.arange(B, device="cuda")
    got = [layer.step(x[rows, lens.long() + i], conv_state, H) for i in range(tokens)]
    whole, _ = layer.forward(x, lengths=lens + tokens)
    want = torch.stack([whole[rows, lens.long() + i] for i in range(tokens)], 1)
    return torch.stack(got, 1), want


def main():
    layer = HybridLayer()
    losses, norms = train(layer)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps; gradient norm {norms[0]:.4f} -> {norms[-1]:.4f}")
    got, want = serve(layer)
    off = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"tokens one by one against one piece: relative difference {off:.1e}")


if __name__ == "__main__":
    main()
