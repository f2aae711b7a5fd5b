"""The residual norm, the gated linear recurrence, clipping and the
orthogonalised update together, as the example uses them: its gradients are
those of its layers, serving token by token agrees with one piece, and training
runs."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _blocks_in_64_bits(p, x, L, C):
    """The layers by their definitions, one step after another."""
    import torch
    norm = lambda h, w: w * h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    h = x
    for i in range(L):
        z = norm(h, p[f"norm{i}"]) @ p[f"in{i}"]
        f = torch.exp(-p[f"alpha{i}"] * torch.nn.functional.softplus(z[..., C:] + p[f"beta{i}"]))
        s, ys = x.new_zeros((x.shape[0], C)), []
        for t in range(x.shape[1]):
            s = f[:, t] * s + (1 - f[:, t]) * z[:, t, :C]
            ys.append(s)
        h = h + torch.stack(ys, 1) @ p[f"out{i}"]
    return norm(h, p["norm"])


def test_gradients():
    """Every weight's gradient against torch.autograd through the layers in 64
    bits.  A gradient passes about ten roundings to bf16 (activations, stream,
    gradients between products), 1.7e-3 each in the mean: 5e-3 together; the sums
    over all steps (alpha, beta, norms) cancel by a few: 3e-2 for all."""
    import torch
    from linear_block import LinearBlocks
    model = LinearBlocks(L=2, D=72, C=40, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((2, 100, 72), generator=gen, device="cuda").bfloat16()
    w = torch.randn((2, 100, 72), generator=gen, device="cuda").bfloat16()
    out, saved = model.forward(x)
    got = model.backward(saved, w)
    p = {n: t.double().requires_grad_() for n, t in model.p.items()}
    ref = _blocks_in_64_bits(p, x.double(), 2, 40)
    assert float((out.double() - ref.detach()).norm() / ref.detach().norm()) <= 1e-2
    for n, g in zip(p, torch.autograd.grad((ref * w.double()).sum(), list(p.values()))):
        assert got[n].shape == g.shape
        assert float((got[n].double() - g).norm() / g.norm()) <= 3e-2, n


@pytest.mark.parametrize("eight", [False, True])
def test_serves(eight):
    import torch
    from linear_block import LinearBlocks, serve
    got, want = serve(LinearBlocks(D=200, C=136, seed=5), dtype=torch.float8_e4m3fn if eight else None)
    # bf16 activations: a few roundings of 2^-9 on each path; in 8 bits those move values across a step of 2^-4 now and
    # then, for a few per cent of the values at most
    assert float((got.float() - want.float()).norm() / want.float().norm()) <= (3e-2 if eight else 1e-2)


def test_trains():
    """Steps run, stay finite, clip, and move each matrix by the update's size: its singular values are near 1."""
    import torch
    from linear_block import LinearBlocks, train
    model = LinearBlocks(L=2, D=96, C=64, seed=6)
    before = {n: t.clone() for n, t in model.p.items()}
    losses, norms = train(model, steps=1, B=2, T=130, lr=0.02, max_norm=1e-3)
    assert norms[0] > 1e-3
    for n, t in model.p.items():
        assert bool(t.isfinite().all()), n
        if t.dim() == 2:
            moved = torch.linalg.svdvals((t.float() - before[n].float()) / (0.2 * 0.02 * max(t.shape) ** 0.5))
            # (the weights round the step to bf16)
            assert float(moved.max()) < 1.35 and float(moved.median()) > 0.55, (n, moved)
    losses, norms = train(model, steps=4, B=2, T=130)
    assert all(v == v and v < 1e9 for v in losses + norms)
