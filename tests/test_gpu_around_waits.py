"""Failure detection of the operators around the layers, without a GPU fault: a
test hook withholds one input tile, the bounded waits expire (about 2 s each),
the kernel makes the failure visible and returns, and the context stays usable.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def scan_args(B, T, C, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, a, dy = (r(B, T, C).to(dtype) for _ in range(3))
    return x, a, r(C).exp(), r(C) - 3.0, dy


def same(got, want):
    return torch.equal(got, want) and bool(got.isfinite().all())


@pytest.mark.parametrize("dtype,tile", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_recurrence_that_misses_a_tile(dtype, tile):
    """One sequence in a cluster of eight blocks: the tile that block 0 misses in round 1 spoils its channels from there
    on with NaN, in every block, and nothing else."""
    from matrix_state_non_gb300 import binding as m
    T, at = 3000, 8 * tile
    x, a, alpha, beta, dy = scan_args(1, T, 128, dtype)
    want = m.linear_scan(x, a, alpha, beta)
    with m.stall_tile_hook(1):
        got = m.linear_scan(x, a, alpha, beta)
        torch.cuda.synchronize()
    y, H = got["y"], got["H_T"]
    assert same(y[:, :, 64:], want["y"][:, :, 64:]) and same(H[:, 64:], want["H_T"][:, 64:])
    assert same(y[:, :at, :64], want["y"][:, :at, :64])
    assert bool(y[:, at:, :64].isnan().all()) and bool(H[:, :64].isnan().all())
    again = m.linear_scan(x, a, alpha, beta)
    assert same(again["y"], want["y"]) and same(again["H_T"], want["H_T"])


@pytest.mark.parametrize("dtype,tile", [(torch.float32, 64)])
def test_recurrence_in_one_block_that_misses_a_tile(dtype, tile):
    from matrix_state_non_gb300 import binding as m
    x, a, alpha, beta, _ = scan_args(220, 300, 64, dtype)
    want = m.linear_scan(x, a, alpha, beta)
    with m.stall_tile_hook(1):
        got = m.linear_scan(x, a, alpha, beta)
        torch.cuda.synchronize()
    y, H = got["y"], got["H_T"]
    assert same(y[1:], want["y"][1:]) and same(H[1:], want["H_T"][1:])
    assert same(y[0, :tile], want["y"][0, :tile])
    assert bool(y[0, tile:].isnan().all()) and bool(H[0].isnan().all())
    assert same(m.linear_scan(x, a, alpha, beta)["y"], want["y"])


@pytest.mark.parametrize("dtype,tile", [(torch.bfloat16, 64)])
def test_backward_that_misses_a_tile(dtype, tile):
    """In both of its launches: the states from round 1 on, and the gradients of round 1 from the end and before."""
    from matrix_state_non_gb300 import binding as m
    T = 3000
    x, a, alpha, beta, dy = scan_args(1, T, 128, dtype)
    call = lambda: m.linear_scan_backward(x, a, alpha, beta, dy, want_dH0=True)  # noqa: E731
    want = call()
    with m.stall_tile_hook(1):
        got = call()
        torch.cuda.synchronize()
    names = ("dx", "da", "dalpha", "dbeta", "dH_0")
    for k in names:
        assert same(got[k][..., 64:], want[k][..., 64:]), k
    at = (-(-T // tile) - 8) * tile  # behind it lies round 0
    assert same(got["dx"][:, at:, :64], want["dx"][:, at:, :64])
    assert bool(got["dx"][:, :at, :64].isnan().all()) and bool(got["da"][:, :, :64][:, 16 * tile:].isnan().all())
    for k in ("dalpha", "dbeta", "dH_0"):
        assert bool(got[k][..., :64].isnan().all()), k
    again = call()
    for k in names:
        assert same(again[k], want[k]), k


@pytest.mark.parametrize("n,rows,cols,product", [(1, 300, 200, 0), (1, 300, 200, 14), (60, 512, 520, 4), (60, 512, 520, 14),
                                                 (20, 800, 800, 0), (20, 800, 800, 14), (1, 65, 1001, 14)])
def test_update_that_misses_operands(n, rows, cols, product):
    """Narrow tiles, persistent blocks, pairs of SMs, rows that TMA does not store: a product of the first, second and last
    step misses its first operands."""
    from matrix_state_non_gb300 import binding as m
    g = torch.randn((n, rows, cols), generator=torch.Generator(device="cuda").manual_seed(rows), device="cuda")
    want = m.orthogonalize(g)
    ws = torch.empty(m.m2rnn_orthogonalize_workspace_size(n, rows, cols), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    with m.stall_tile_hook(product):
        m.orthogonalize(g, out=out, workspace=ws)
        status, where = m.sync_status(ws)
    assert status == m.M2RNN_ERR_TIMEOUT and where // 10 == 42, (status, where)
    if product < 14:
        assert bool(out.isnan().all())
    else:  # what the block that missed them had to make is NaN, the rest is right
        spoilt = out.isnan()
        assert bool(spoilt[0].any()) and not bool(spoilt.all())
        assert torch.equal(out[~spoilt], want[~spoilt])
    assert same(m.orthogonalize(g, out=out, workspace=ws), want) and m.sync_status(ws)[0] == m.M2RNN_OK
