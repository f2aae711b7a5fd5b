"""Pre-norm residual layers around the gated linear recurrence, trained and
served with the library's operators.

    h = h + branch, norm (one kernel) -> in-projection -> gated linear recurrence
    -> out-projection = the next layer's branch

``train`` runs steps on a synthetic task: forward, backward, global gradient
clipping, and the orthogonalised momentum as the update of the matrices (the
vectors take plain steps).  ``serve`` takes a ragged batch of prompts through the
layers and continues each one token at a time from the states the prompts left,
with the normalised activations in bf16 or in 8 bits with scales.  The
projections are plain matrix products; everything between them, the clipping and
the update run in the library's kernels.

    python examples/linear_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from matrix_state_non_gb300 import binding as m  # noqa: E402


class LinearBlocks:
    """Weights of L layers of D channels with states of C: bf16 matrices, fp32
    norms and gate parameters."""

    def __init__(self, L=2, D=256, C=256, seed=0, device="cuda"):
        self.L, self.D, self.C = L, D, C
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *shape, scale: (scale * torch.randn(shape, generator=gen, device=device)).bfloat16()  # noqa: E731
        self.p = {}
        for i in range(L):
            step = torch.logspace(-2.5, 0, C, device=device)  # decays from a step to hundreds
            self.p.update({f"norm{i}": torch.ones(D, device=device), f"in{i}": rand(D, 2 * C, scale=D ** -0.5),
                           f"alpha{i}": torch.ones(C, device=device), f"beta{i}": torch.log(torch.expm1(step)),
                           f"out{i}": rand(C, D, scale=C ** -0.5)})
        self.p["norm"] = torch.ones(D, device=device)

    def _project(self, y, scale, name):
        """y (in 8 bits: times its scales) through a matrix."""
        if scale is not None:
            y = (y.float() * scale.repeat_interleave(m.SCALE_BLOCK, -1)[..., :y.shape[-1]]).bfloat16()
        return y @ self.p[name]

    def forward(self, x, lengths=None, H=None, dtype=None):
        """x [B,T,D] bf16.  Returns the normalised output and what the backward and the next piece of the sequences need."""
        p, saved, branch, h = self.p, [], x, None
        for i in range(self.L):
            n = m.residual_norm(branch, p[f"norm{i}"], h, dtype=dtype)
            h = n.get("h", x)
            z = self._project(n["y"], n.get("scale"), f"in{i}")
            s = m.linear_scan(z[..., :self.C], z[..., self.C:], p[f"alpha{i}"], p[f"beta{i}"],
                              H_0=None if H is None else H[i], lengths=lengths)
            branch = s["y"] @ p[f"out{i}"]
            saved.append(dict(h=h, y=n["y"], z=z, s=s["y"], H=s["H_T"]))
        n = m.residual_norm(branch, p["norm"], h)
        return n["y"], dict(layers=saved, h=n["h"])

    def backward(self, saved, dout):
        """Gradients of every weight, given the output's gradient [B,T,D]."""
        p, C = self.p, self.C
        flat = lambda t: t.flatten(0, -2)  # noqa: E731
        g = {}
        n = m.residual_norm_backward(saved["h"], p["norm"], dout)
        g["norm"], dh = n["dw"], n["dx"]  # of the stream and of the branch alike
        for i in reversed(range(self.L)):
            s = saved["layers"][i]
            db = dh.bfloat16()
            g[f"out{i}"] = flat(s["s"]).t() @ flat(db)
            b = m.linear_scan_backward(s["z"][..., :C], s["z"][..., C:], p[f"alpha{i}"], p[f"beta{i}"], db @ p[f"out{i}"].t())
            g[f"alpha{i}"], g[f"beta{i}"] = b["dalpha"], b["dbeta"]
            dz = torch.cat([b["dx"], b["da"]], -1).bfloat16()
            g[f"in{i}"] = flat(s["y"]).t() @ flat(dz)
            n = m.residual_norm_backward(s["h"], p[f"norm{i}"], dz @ p[f"in{i}"].t(), dh=dh, out=dict(dx=dh))
            g[f"norm{i}"] = n["dw"]
        return g

    def step(self, x, H, dtype=None):
        """One token for every sequence: x [B,D]; the states advance in place."""
        p, branch, h = self.p, x, None
        for i in range(self.L):
            n = m.residual_norm(branch, p[f"norm{i}"], h, dtype=dtype)
            h = n.get("h", x)
            z = self._project(n["y"], n.get("scale"), f"in{i}")
            branch = m.linear_step(H[i], z[:, :self.C], z[:, self.C:], p[f"alpha{i}"], p[f"beta{i}"]) @ p[f"out{i}"]
        return m.residual_norm(branch, p["norm"], h)["y"]


def train(model, steps=20, B=4, T=512, lr=0.02, momentum=0.9, max_norm=1.0, seed=1):
    """Fits a fixed random target; returns the losses and the gradient norms."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((B, T, model.D), generator=gen, device="cuda").bfloat16()
    target = torch.randn((B, T, model.D), generator=gen, device="cuda")
    names = sorted(model.p)
    grads = {n: torch.empty_like(model.p[n], dtype=torch.float32) for n in names}  # one buffer each, for all steps
    kept = {n: torch.zeros_like(grads[n]) for n in names if model.p[n].dim() == 2}
    plan = m.grad_plan([grads[n] for n in names])
    losses, norms = [], []
    for _ in range(steps):
        out, saved = model.forward(x)
        diff = out.float() - target
        losses.append(diff.square().mean())
        for n, g in model.backward(saved, (2.0 / diff.numel() * diff).bfloat16()).items():
            grads[n].copy_(g)
        norms.append(m.grad_clip(plan, max_norm))
        for n in names:
            if n in kept:
                kept[n].mul_(momentum).add_(grads[n])
                rows, cols = kept[n].shape
                model.p[n] -= (0.2 * lr * max(rows, cols) ** 0.5) * m.orthogonalize(kept[n])
            else:
                model.p[n] -= lr * grads[n]
    return [float(v) for v in losses], [float(v) for v in norms]


def serve(model, lengths=(37, 1, 130, 64), tokens=4, dtype=None, seed=2):
    """Prompts of several lengths, then `tokens` more of each: returns the
    outputs [B,tokens,D] and those of the same tokens run in one piece."""
    B, T = len(lengths), max(lengths)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((B, T + tokens, model.D), generator=gen, device="cuda").bfloat16()
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    _, saved = model.forward(x[:, :T].contiguous(), lengths=lens, dtype=dtype)
    H = [s["H"] for s in saved["layers"]]
    rows = torch.arange(B, device="cuda")
    got = [model.step(x[rows, lens.long() + i], H, dtype=dtype) for i in range(tokens)]
    whole, _ = model.forward(x, lengths=lens + tokens, dtype=dtype)
    want = torch.stack([whole[rows, lens.long() + i] for i in range(tokens)], 1)
    return torch.stack(got, 1), want


def main():
    model = LinearBlocks()
    losses, norms = train(model)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps; gradient norm {norms[0]:.4f} -> {norms[-1]:.4f}")
    for dtype in (None, torch.float8_e4m3fn):
        got, want = serve(model, dtype=dtype)
        off = float((got.float() - want.float()).norm() / want.float().norm())
        print(f"tokens one by one against one piece ({'bf16' if dtype is None else '8 bits'}): relative difference {off:.1e}")


if __name__ == "__main__":
    main()
