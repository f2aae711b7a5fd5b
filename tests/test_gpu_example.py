"""The hybrid layer's example: it learns, its gradients are those of its loss,
and serving token by token agrees with running the sequences in one piece."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_trains_and_clips():
    from hybrid_layer import HybridLayer, train
    losses, norms = train(HybridLayer(D=128, N=4, K=32, V=32), steps=12, B=2, T=200, lr=2.0, max_norm=0.05)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert norms[0] > 0.05  # clipped


def _layer_in_64_bits(p, x, N, G, K, V, W):
    """The layer by its definitions, one step after another."""
    import torch
    C = N * V + 2 * G * K
    z = x @ p["w_in"]
    xs = torch.cat([x.new_zeros((x.shape[0], W - 1, C)), z[..., :C]], 1)
    pre = p["conv_b"] + sum(p["conv_w"][:, w] * xs[:, w:w + x.shape[1]] for w in range(W))
    h = pre * torch.sigmoid(pre)
    v, k, q = h[..., :N * V].unflatten(-1, (N, V)), h[..., N * V:N * V + K], h[..., N * V + K:]
    D = torch.nn.functional.softplus(z[..., C + N * V:] + p["dt_bias"])
    H, ys = x.new_zeros((x.shape[0], N, K, V)), []
    for t in range(x.shape[1]):
        H = torch.exp(D[:, t] * p["A"])[..., None, None] * H + D[:, t, :, None, None] * torch.einsum(
            "bk,bnv->bnkv", k[:, t], v[:, t])
        ys.append(torch.einsum("bk,bnkv->bnv", q[:, t], H) + p["w_r"] * v[:, t])
    y = torch.stack(ys, 1) * z[..., C:C + N * V].unflatten(-1, (N, V))
    o = y * (y.square().mean((2, 3), keepdim=True) + 1e-6).rsqrt() * p["norm_w"]
    return x + o.flatten(2) @ p["w_out"]


def test_example_gradients():
    """Every weight's gradient against torch.autograd through the layer in 64
    bits.  The layer rounds about ten times to bf16 between weights and
    gradients, 1.7e-3 each in the mean: 5e-3 together; the sums over all steps
    (A, dt_bias) cancel by a few: 3e-2 for all."""
    import torch
    from hybrid_layer import HybridLayer
    layer = HybridLayer(D=64, N=2, K=32, V=32, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((2, 100, 64), generator=gen, device="cuda").bfloat16()
    w = torch.randn((2, 100, 64), generator=gen, device="cuda").bfloat16()
    out, saved = layer.forward(x)
    got = layer.backward(saved, w)
    p = {n: t.double().requires_grad_() for n, t in layer.p.items()}
    ref = _layer_in_64_bits(p, x.double(), 2, 1, 32, 32, layer.W)
    assert float((out.double() - ref).norm() / ref.norm()) <= 1e-2
    for n, g in zip(p, torch.autograd.grad((ref * w.double()).sum(), list(p.values()))):
        assert got[n].shape == g.shape
        assert float((got[n].double() - g).norm() / g.norm()) <= 3e-2, n


def test_example_serves():
    from hybrid_layer import HybridLayer, serve
    got, want = serve(HybridLayer(seed=5))
    # bf16 activations: a few roundings of 2^-9 on each path
    assert float((got.float() - want.float()).norm() / want.float().norm()) <= 1e-2
