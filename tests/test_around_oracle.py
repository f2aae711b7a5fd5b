"""Pins of the float64 oracle of the operators around the layers: gradients
against differences, the 8-bit format against torch's, the polynomial of the
singular values against the products."""
import numpy as np
import pytest

from oracle import around_oracle as o


def _differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        x[i] = keep
    return g


def test_norm_gradients():
    r = np.random.default_rng(1)
    h, w, dy, dh = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=(3, 7)), r.normal(size=(3, 7))
    loss = lambda: (o.residual_norm(h, w, eps=1e-3)[0] * dy).sum() + (h * dh).sum()  # noqa: E731
    dx, dw = o.residual_norm_backward(h, w, dy, dh, eps=1e-3)
    np.testing.assert_allclose(dx, _differences(loss, h), atol=1e-7)
    np.testing.assert_allclose(dw, _differences(loss, w), atol=1e-7)


@pytest.mark.parametrize("lengths", [None, (6, 1, 0)])
def test_linear_scan_gradients(lengths):
    r = np.random.default_rng(2)
    p = dict(x=r.normal(size=(3, 6, 4)), a=r.normal(size=(3, 6, 4)), alpha=r.uniform(0.5, 2, 4), beta=r.normal(size=4),
             H_0=r.normal(size=(3, 4)))
    dy, dH_T = r.normal(size=(3, 6, 4)), r.normal(size=(3, 4))

    def loss():
        y, H = o.linear_scan(**p, lengths=lengths)
        return (y * dy).sum() + (H * dH_T).sum()

    got = o.linear_scan_backward(p["x"], p["a"], p["alpha"], p["beta"], dy, p["H_0"], dH_T, lengths)
    for n in p:
        np.testing.assert_allclose(got["d" + n], _differences(loss, p[n]), atol=1e-7, err_msg=n)


def test_scan_in_two_pieces():
    r = np.random.default_rng(3)
    x, a, alpha = r.normal(size=(2, 9, 3)), r.normal(size=(2, 9, 3)), r.uniform(0.1, 1, 3)
    y, H = o.linear_scan(x, a, alpha)
    y1, H1 = o.linear_scan(x[:, :4], a[:, :4], alpha)
    y2, H2 = o.linear_scan(x[:, 4:], a[:, 4:], alpha, H_0=H1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, atol=1e-14)
    np.testing.assert_allclose(H2, H, atol=1e-14)


def test_e4m3_is_torchs():
    import torch
    v = np.concatenate([np.linspace(-448, 448, 4001), np.linspace(-0.05, 0.05, 4001), [2.0 ** -10, 3 * 2.0 ** -10, 0.0]])
    v = v.astype(np.float32).astype(np.float64)
    t = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.e4m3(v), t)


def test_quantize_bounds():
    r = np.random.default_rng(4)
    y = r.normal(size=(5, 300)) * np.exp(r.normal(size=(5, 300)))
    y[2, 128:256] = 0.0
    q, scale = o.quantize(y)
    assert scale.shape == (5, 3) and np.abs(q).max() == 448.0
    wide = np.repeat(scale, 128, 1)[:, :300]
    assert np.all(np.abs(q * wide - y) <= 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * wide)
    assert np.all(q[2, 128:256] == 0.0) and scale[2, 1] == 2.0 ** -126


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6), (2, 4, 7), (1, 3)])
def test_orthogonalize_is_the_products(shape):
    g = np.random.default_rng(5).normal(size=shape)
    a, b, c = o.COEFFICIENTS
    x = g / (np.sqrt((g * g).sum((-2, -1), keepdims=True)) + 1e-7)
    for _ in range(5):
        gram = x @ np.swapaxes(x, -1, -2)
        x = a * x + (b * gram + c * gram @ gram) @ x
    np.testing.assert_allclose(o.orthogonalize(g), x, atol=1e-12)


def test_orthogonalize_brings_singular_values_near_one():
    r = np.random.default_rng(6)
    s = np.linalg.svd(o.orthogonalize(r.normal(size=(40, 60))), compute_uv=False)
    assert 0.65 < s.min() and s.max() < 1.21
    assert np.all(o.orthogonalize(np.zeros((3, 4))) == 0.0)
