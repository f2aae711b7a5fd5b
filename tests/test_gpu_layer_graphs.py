"""The convolution's and the clipping's calls captured in a CUDA graph and
replayed on other values give the bits of plain calls."""
import pytest

from layer_util import conv_inputs, dev

pytestmark = pytest.mark.gpu


def capture(run):
    """The outputs of run() in a graph, and the graph."""
    import torch
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run()
    return graph, out


@pytest.mark.parametrize("B,T,C,W,dtype", [(2, 300, 64, 4, "bf16"), (2, 130, 33, 3, "f32")])
def test_convolution_in_a_graph(B, T, C, W, dtype):
    import torch
    from matrix_state_non_gb300 import binding as m
    sets = []
    for seed in (1, 2):
        d = conv_inputs(B, T, C, W, dtype, seed=seed, x0=True)
        sets.append({n: dev(a, "f32" if n in ("dy", "dx_T") else dtype) for n, a in d.items()})

    def run(g):
        f = m.causal_conv(g["x"], g["w"], g["bias"], x0=g["x0"], want_state=True)
        state = f["x_T"].clone()
        y = m.causal_conv_step(state, g["x"][:, 0], g["w"], g["bias"])
        b = m.causal_conv_backward(g["x"], g["w"], g["bias"], g["dy"], x0=g["x0"], dx_T=g["dx_T"], want_dx0=True)
        return dict(b, **f, state=state, step=y)

    want = [run(g) for g in sets]
    buf = {n: x.clone() for n, x in sets[0].items()}
    graph, out = capture(lambda: run(buf))
    for g, w in zip(sets[::-1], want[::-1]):
        for n, x in g.items():
            buf[n].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for n in w:
            assert torch.equal(out[n], w[n]), n


def test_clipping_in_a_graph():
    import torch
    from matrix_state_non_gb300 import binding as m
    shapes = [((300, 64), torch.bfloat16), ((70001,), torch.float32), ((5,), torch.float32)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    sets = [[torch.randn(s, generator=gen, device="cuda").to(t) for s, t in shapes] for _ in range(2)]
    want = []
    for g in sets:
        outs = [torch.empty_like(x) for x in g]
        want.append((m.grad_clip(m.grad_plan(g, outs), 1.0), outs))
    buf = [x.clone() for x in sets[0]]
    outs = [torch.empty_like(x) for x in buf]
    plan = m.grad_plan(buf, outs)
    graph, norm = capture(lambda: m.grad_clip(plan, 1.0))
    for g, (n, w) in zip(sets[::-1], want[::-1]):
        for x, y in zip(buf, g):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, n) and all(torch.equal(x, y) for x, y in zip(outs, w))
