"""The recurrence's helpers take dense tensors: column slices (of a fused
convolution's y, say) are refused and not read as if they were dense."""
import pytest
import torch

from matrix_state_non_gb300 import binding as m


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            if name.endswith(("_size", "_count")):
                return lambda *a: 1 << 20
            return lambda *a: pytest.fail(f"{name} was called")
    monkeypatch.setattr(m, "load", lambda: Lib())
    monkeypatch.setattr(m, "_stream_handle", lambda s: 0)


def parts(B=2, T=5, N=2, K=8, V=4, dtype=torch.bfloat16):
    z = torch.zeros((B, T, 2 * N * K + N * V), dtype=dtype)
    sl = dict(q=z[..., :N * K].unflatten(-1, (N, K)), k=z[..., N * K:2 * N * K].unflatten(-1, (N, K)),
              v=z[..., 2 * N * K:].unflatten(-1, (N, V)))
    f32 = torch.float32
    return sl, dict(f=torch.zeros((B, T, N), dtype=dtype), W=torch.zeros((N, V, V), dtype=dtype),
                    w_r=torch.zeros((N, V), dtype=dtype)), torch.zeros((B, T, N, V), dtype=f32), \
        torch.zeros((B, N, K, V), dtype=f32)


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_column_slices_are_refused(name):
    sl, rest, dy, H = parts()
    d = {n: x if n == name else x.contiguous() for n, x in sl.items()}
    with pytest.raises(ValueError, match="contiguous"):
        m.forward(d["q"], d["k"], d["v"], rest["f"], rest["W"], rest["w_r"])
    with pytest.raises(ValueError, match="contiguous"):
        m.backward(d["q"], d["k"], d["v"], rest["f"], rest["W"], rest["w_r"], dy)
    step = {n: x[:, 0] for n, x in d.items()}
    with pytest.raises(ValueError, match="contiguous"):
        m.decode_step(H, step["q"], step["k"], step["v"], rest["f"][:, 0].contiguous(), rest["W"], rest["w_r"])


def test_the_other_operands_are_checked_too():
    sl, rest, dy, H = parts()
    d = {n: x.contiguous() for n, x in sl.items()}
    with pytest.raises(ValueError, match="contiguous"):
        m.forward(d["q"], d["k"], d["v"], rest["f"], rest["W"].transpose(1, 2), rest["w_r"])
    with pytest.raises(ValueError, match="contiguous"):
        m.forward(d["q"], d["k"], d["v"], rest["f"], rest["W"], rest["w_r"], H_0=H.transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError, match="contiguous"):
        m.output_norm(dy[..., :3], dy[..., :3], rest["w_r"].float()[:, :3])
