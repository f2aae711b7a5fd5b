"""SiLU and its derivative in the fp32 convolution, value by value.

silu(x) = x / (1 + e^-x): the exponential is good to 2 units of 2^-23, the sum,
the quotient and the product to half a unit each: 4 units, 2^-21, wherever
e^-x is in the fp32 range.  The derivative s + x s (1 - s) adds two products
of terms whose sum cancels around x = -1.28 only: 8 units of their sizes."""
import pytest

pytestmark = pytest.mark.gpu


def test_fp32_silu_value_by_value():
    import torch
    from matrix_state_non_gb300 import binding as m
    x = torch.cat([torch.linspace(-87, 87, 200001), torch.linspace(-1e-3, 1e-3, 2001)]).cuda()
    w, one = torch.ones((1, 1), device="cuda"), torch.ones((1, x.numel(), 1), device="cuda")
    y = m.causal_conv(x[None, :, None], w)["y"].flatten().double()
    s = torch.sigmoid(x.double())
    want = x.double() * s
    assert bool(((y - want).abs() <= 2.0 ** -21 * want.abs()).all()), \
        float(((y - want).abs() / want.abs().clamp_min(1e-300)).max() * 2 ** 21)
    dx = m.causal_conv_backward(x[None, :, None], w, None, one)["dx"].flatten().double()
    tail = torch.sigmoid(-x.double())  # 1 - s
    size = s + want.abs() * tail
    err = (dx - (s + want * tail)).abs()
    assert bool((err <= 2.0 ** -20 * size).all()), float((err / size).max() * 2 ** 20)


def test_step_is_the_prompt_value_by_value():
    import torch
    from matrix_state_non_gb300 import binding as m
    x = torch.linspace(-87, 87, 4096, device="cuda")
    w = torch.ones((4096, 1), device="cuda")
    y = m.causal_conv_step(torch.empty((1, 0, 4096), device="cuda"), x[None], w)
    assert torch.equal(y, m.causal_conv(x[None, None], w)["y"][:, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_silu_far_out(dtype):
    """Behind the range of e^-x: 0 and x, slopes 0 and 1; infinity as the formula has it."""
    import torch
    from matrix_state_non_gb300 import binding as m
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.tensor([-3e38, -1e20, -1e4, -300, -128, -100, -90, 90, 100, 300, 1e4, 1e20, 3e38], device="cuda").to(t)
    w = torch.ones((1, 1), device="cuda", dtype=t)
    y = m.causal_conv(x[None, :, None], w)["y"].flatten().float()
    assert bool((y[:7].abs() <= 1e-35).all()) and torch.equal(y[7:], x[7:].float())
    dx = m.causal_conv_backward(x[None, :, None], w, None, torch.ones((1, 13, 1), device="cuda"))["dx"].flatten()
    assert bool((dx[:7].abs() <= 1e-35).all()) and bool((dx[7:] == 1).all())
    bad = torch.tensor([float("inf"), float("nan")], device="cuda").to(t)
    y = m.causal_conv(bad[None, :, None], w)["y"].flatten()
    assert torch.isinf(y[0]) and y[0] > 0 and torch.isnan(y[1])
    assert torch.isnan(m.causal_conv_step(torch.empty((2, 0, 1), device="cuda", dtype=t), bad[:, None], w)[1])
