"""The tile kernel and the chained products inside captured graphs and on side streams, and the same bits again."""
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu


def randn(*shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def linear_case():
    x, w, r = randn(4096, 512, seed=1), randn(2048, 512, seed=2, scale=0.05), randn(4096, 2048, seed=3)
    y, z = torch.empty(4096, 2048, dtype=torch.bfloat16, device="cuda"), torch.empty(4096, 2048, dtype=torch.bfloat16, device="cuda")
    return [x, w, r], [y, z], lambda stream: zc.linear(x, w, act="gelu", residual=r, preact=z, out=y, stream=stream)


def dgrad_case():
    dy, w, z = randn(4096, 1024, seed=1), randn(1024, 2048, seed=2, scale=0.05), randn(4096, 2048, seed=3)
    dx = torch.empty(4096, 2048, dtype=torch.bfloat16, device="cuda")
    return [dy, w, z], [dx], lambda stream: zc.linear_dgrad(dy, w, preact=z, act="silu", out=dx, stream=stream)


def wgrad_case():
    dy, x = randn(8192, 2048, seed=1), randn(8192, 1024, seed=2)
    dw, db = torch.empty(2048, 1024, device="cuda"), torch.empty(2048, device="cuda")
    return [dy, x], [dw, db], lambda stream: zc.linear_wgrad(dy, x, dw, bias_grad=db, stream=stream)


def chained_case():
    g = randn(12, 512, 1024, seed=1)
    o = torch.empty_like(g)
    ws = torch.empty(zc.lib().dpred_newton_schulz_workspace_bytes(12, 512, 1024), dtype=torch.uint8, device="cuda")
    return [g], [o], lambda stream: zc.newton_schulz(g, out=o, workspace=ws, stream=stream)


def muon_case():
    """Small matrices, chained ones of two shapes; the weights and momenta are set back inside the step."""
    shapes = [(64, 96)] * 3 + [(512, 1024)] * 6 + [(300, 1200)] * 5
    w0, g = [randn(*s, seed=i) for i, s in enumerate(shapes)], [randn(*s, seed=50 + i, scale=1e-3) for i, s in enumerate(shapes)]
    opt = zc.Muon([w.clone() for w in w0])

    def step(stream):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            for w, m, w1 in zip(opt.weights, opt.momenta, w0):
                w.copy_(w1)
                m.fill_(1e-3)
        opt.step(g, 0.01, stream=stream)

    return g, opt.weights + opt.momenta, step


@pytest.mark.parametrize("case", [linear_case, dgrad_case, wgrad_case, chained_case, muon_case])
def test_captured_and_on_a_side_stream(case):
    inputs, outputs, call = case()
    call(None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outputs]

    def check(what):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs, want)), what
        for o in outputs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()

    check("plain")
    call(None)
    check("again")
    side = torch.cuda.Stream()
    call(side)
    side.synchronize()
    check("side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(None)
    for _ in range(3):
        graph.replay()
        check("replayed")
    inputs[0].mul_(-1)  # a graph reads its inputs at replay
    call(None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outputs]
    graph.replay()
    check("replayed with other inputs")
    assert zc.device_status() == 0
