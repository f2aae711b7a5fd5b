"""Tensors of more than 2^31 values: offsets are 64-bit everywhere.  The last
rows, steps and matrices agree with calls on those alone."""
import pytest

pytestmark = pytest.mark.gpu


def test_norm_rows_behind_2_to_the_31():
    import torch
    from matrix_state_non_gb300 import binding as m
    rows, D = 2_100_003, 1024
    x = torch.zeros((rows, D), device="cuda", dtype=torch.bfloat16)
    res = torch.zeros((rows, D), device="cuda", dtype=torch.bfloat16)
    x[-5:], res[-5:] = torch.randn(5, D, device="cuda").bfloat16(), torch.randn(5, D, device="cuda").bfloat16()
    w = torch.rand(D, device="cuda") + 0.5
    for ty in (torch.bfloat16, torch.float8_e4m3fn):
        r = m.residual_norm(x, w, res, dtype=ty)
        alone = m.residual_norm(x[-5:].clone(), w, res[-5:].clone(), dtype=ty)
        for n in alone:
            assert torch.equal(r[n][-5:].float(), alone[n].float()), n
        h = r["h"]
        del r
    dy = torch.zeros_like(x)
    dy[-5:] = torch.randn(5, D, device="cuda").bfloat16()
    got = m.residual_norm_backward(h, w, dy)
    alone = m.residual_norm_backward(h[-5:].clone(), w, dy[-5:].clone())
    assert torch.equal(got["dx"][-5:], alone["dx"])
    # the other rows add zeros to dw, in another order of five terms
    assert float((got["dw"] - alone["dw"]).abs().max()) <= 1e-6 * float(alone["dw"].abs().max()) * 5


@pytest.mark.parametrize("C", [1024, 1022, 1021])
def test_scan_steps_behind_2_to_the_31(C):
    import torch
    from matrix_state_non_gb300 import binding as m
    T, last = 2_110_000, 700
    x = torch.ones((1, T, C), device="cuda", dtype=torch.bfloat16)
    a = torch.zeros((1, T, C), device="cuda", dtype=torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for t in (x, a):
        t[:, -last:] = torch.randn((1, last, C), generator=gen, device="cuda").bfloat16()
    alpha, beta = torch.rand(C, device="cuda") + 0.1, torch.randn(C, device="cuda")
    r = m.linear_scan(x, a, alpha, beta)
    tail = lambda t: t[:, -last:].clone()  # (not a view: dy has to lie on 16 bytes)  # noqa: E731
    one = torch.ones((1, C), device="cuda")  # what a memory of a few steps has made of ones
    alone = m.linear_scan(tail(x), tail(a), alpha, beta, H_0=one)
    off = lambda p, q: float((p.float() - q.float()).norm() / q.float().norm())  # noqa: E731
    assert off(r["H_T"], alone["H_T"]) <= 1e-5 and off(tail(r["y"]), alone["y"]) <= 1e-4
    del r
    dy = torch.zeros_like(x)
    dy[:, -last:] = torch.randn((1, last, C), generator=gen, device="cuda").bfloat16()
    got = m.linear_scan_backward(x, a, alpha, beta, dy)
    alone = m.linear_scan_backward(tail(x), tail(a), alpha, beta, tail(dy), H_0=one)
    assert off(tail(got["dx"]), alone["dx"]) <= 1e-5 and off(tail(got["da"]), alone["da"]) <= 1e-4


def test_matrices_behind_2_to_the_31():
    import torch
    from matrix_state_non_gb300 import binding as m
    n, rows, cols = 530, 2048, 2000
    g = torch.zeros((n, rows, cols), device="cuda", dtype=torch.bfloat16)
    g[-1] = torch.randn((rows, cols), device="cuda").bfloat16()
    g[0, :, 0] = 1
    got = m.orthogonalize(g)
    alone = m.orthogonalize(g[-1])
    # two paths, each within 2e-3 of the result before its rounding to bf16
    assert float((got[-1].float() - alone.float()).norm() / alone.float().norm()) <= 5e-3
    assert int(got[1:-1].count_nonzero()) == 0
