"""The products, the reduction and the optimizer step together (examples/train_step.py),
and what the Python calls refuse."""
import importlib.util
import os

import pytest
import torch

import zero_collectives_gb300 as zc
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def data(block, tokens=160):
    g = torch.Generator(device="cuda").manual_seed(1)
    shift = torch.randn(block.width, block.width, device="cuda", generator=g) / block.width ** 0.5
    xs = [torch.randn(tokens + r, block.width, device="cuda", generator=g).bfloat16() for r in range(block.world)]
    return xs, [(x.float() + torch.tanh(x.float() @ shift)).bfloat16() for x in xs]


def test_reduced_gradients_are_the_mean_of_the_replicas(example):
    """The owners receive the mean over replicas of the gradients that autograd
    computes in 64 bits.  Tolerance (2-norm): z, h, y, dy and dz are rounded to
    bf16 on the way (2^-9 each at most, root mean square), then each replica's
    gradient and the mean: seven roundings, 7 * 2^-9 / sqrt(3) < 8e-3."""
    block = example.Block(world=4, width=72, inner=200)
    xs, ts = data(block)
    want = [0, 0, 0]
    for x, t in zip(xs, ts):
        w1, b1, w2 = (v.double().requires_grad_(True) for v in (block.w1, block.b1, block.w2))
        y = torch.nn.functional.gelu(x.double() @ w1.T + b1, approximate="tanh") @ w2.T + x.double()
        loss = (y - t.double()).square().mean()
        for p, gr in enumerate(torch.autograd.grad(loss, (w1, b1, w2))):
            want[p] = want[p] + gr / block.world
    for r, (x, t) in enumerate(zip(xs, ts)):
        block.replica_step(r, x, t)
    block.ex.flush_all(block.rows)
    for p in range(3):
        got = block.ex.grad.view(block.keeper[p], p).view(block.shapes[p]).double()
        assert float((got - want[p]).norm()) <= 8e-3 * float(want[p].norm()), p
    assert zc.device_status() == 0


def test_training_reduces_the_loss(example):
    block = example.Block()
    xs, ts = data(block)
    losses = [float(block.step(xs, ts)) for _ in range(25)]
    assert losses[-1] < 0.5 * losses[0] and all(l == l for l in losses)


def test_example_runs(example, capsys):
    example.main()
    assert "gradients reduce to one rank" in capsys.readouterr().out


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16, device="cuda")


def test_python_refusals():
    f32 = torch.zeros
    with pytest.raises(TypeError):
        zc.linear(f32(4, 8, device="cuda"), bf(6, 8))
    with pytest.raises(ValueError):
        zc.linear(bf(4, 8), bf(6, 9))
    with pytest.raises(ValueError):
        zc.linear(bf(4, 8), torch.zeros(6, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        zc.linear(bf(4, 16)[:, ::2], bf(6, 8))
    with pytest.raises(ValueError):
        zc.linear(bf(4, 8), bf(6, 8), act="tanh")
    with pytest.raises(ValueError):
        zc.linear(bf(4, 8), bf(6, 8), bias=bf(5))
    with pytest.raises(ValueError):
        zc.linear(bf(4, 8), bf(6, 8), residual=bf(4, 8))
    with pytest.raises(ValueError):
        zc.linear(bf(4, 8), bf(6, 8), out=bf(6, 4))
    with pytest.raises(ValueError):
        zc.linear(bf(8), bf(6, 8))
    with pytest.raises(ValueError):
        zc.linear_dgrad(bf(4, 6), bf(6, 8), act="gelu")
    with pytest.raises(TypeError):
        zc.linear_wgrad(bf(4, 6), bf(4, 8), torch.zeros(6, 8, device="cuda", dtype=torch.float64))
    with pytest.raises(TypeError):
        zc.linear_wgrad(bf(4, 6), bf(4, 8), bf(6, 8), bias_grad=bf(6))
    with pytest.raises(ValueError):
        zc.linear_wgrad(bf(4, 6), bf(5, 8), bf(6, 8))
    with pytest.raises(zc.DpredError) as e:
        zc.linear(bf(4, 9)[:, 1:], bf(6, 8), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -3
    with pytest.raises(ValueError):
        zc.newton_schulz(torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        zc.newton_schulz(torch.zeros(4, 5, device="cuda"), out=bf(5, 4))
    with pytest.raises(zc.DpredError):
        zc.newton_schulz(torch.zeros(4, 5, device="cuda"), steps=0)
    w, m, g = bf(4, 5), torch.zeros(4, 5, device="cuda"), bf(4, 5)
    with pytest.raises(ValueError):
        zc.muon_step([w], [m], [], lr=0.1)
    with pytest.raises(ValueError):
        zc.muon_step([w], [m], [bf(5, 4)], lr=0.1)
    with pytest.raises(TypeError):
        zc.muon_step([w], [bf(4, 5)], [g], lr=0.1)
    with pytest.raises(TypeError):
        zc.muon_step([w, m], [m, m], [g, g], lr=0.1)
    with pytest.raises(zc.DpredError):
        zc.muon_step([w], [m], [g], lr=float("nan"))
    assert zc.device_status() == 0


def test_calls_without_the_extension_module():
    """The same calls through ctypes give the same bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(70, 96, device="cuda", generator=g).bfloat16()
    w = torch.randn(40, 96, device="cuda", generator=g).bfloat16()
    dy = torch.randn(70, 40, device="cuda", generator=g).bfloat16()
    calls = (lambda: zc.linear(x, w, act="silu"), lambda: zc.linear_dgrad(dy, w), lambda: zc.linear_wgrad(dy, x, bf(40, 96)))
    want = [f() for f in calls]
    fast, find = zc._FC, zc._fast_call_module
    try:
        zc._FC, zc._fast_call_module = None, lambda: None
        got = [f() for f in calls]
    finally:
        zc._FC, zc._fast_call_module = fast, find
    assert all(torch.equal(a, b) for a, b in zip(want, got))
