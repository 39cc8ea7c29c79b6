"""The embedding, the block norms, the products, the reduction and the clipping
as one training step: gradients against 64-bit ones, the clipped and reduced
gradients against their formulas, and the step in a captured graph.

Tolerance of a gradient: every tensor between two calls is rounded to bf16 once
(2^-8 of an element's value, at random), some ten roundings lie between the loss
and the deepest parameter, and each acts on the whole result like an error of
2^-8 of its norm at most: 10 * 2^-8 of the gradient's norm.  Gradients are then
stored in bf16."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("lm_step", os.path.join(ROOT, "examples", "lm_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def loss64(model, p, ids, target):
    """The step's loss in 64 bits."""
    def norm(a, w):
        return a * (a.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    x = p["embed"][ids] * model.scale
    h = norm(x, p["norm0"])
    for i in range(model.blocks):
        y = torch.nn.functional.gelu(h @ p[f"w1.{i}"].T, approximate="tanh") @ p[f"w2.{i}"].T
        x = model.residual * x + p[f"gate.{i}"] * norm(y, p[f"post.{i}"])
        h = norm(x, p[f"norm{i + 1}"])
    return (h - target).square().mean()


def inputs(model, tokens, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    vocab, width = model.params["embed"].shape
    ids = [torch.randint(0, vocab, (tokens,), device="cuda", generator=g) // 3 for _ in range(model.world)]
    return ids, [torch.randn(tokens, width, device="cuda", generator=g) for _ in ids]


@pytest.mark.parametrize("world,vocab,width,inner,blocks,tokens", [(2, 300, 64, 128, 1, 40), (3, 501, 72, 104, 2, 333), (2, 97, 33, 50, 2, 1)])
def test_gradients_of_a_step(world, vocab, width, inner, blocks, tokens):
    model = example().Model(world, vocab, width, inner, blocks)
    g = torch.Generator(device="cuda").manual_seed(9)
    for n, w in model.params.items():
        if not n.startswith(("w", "embed")):
            w.add_(torch.randn(w.shape, device="cuda", generator=g), alpha=0.1)
    ids, targets = inputs(model, tokens)
    p = {n: w.double().requires_grad_(True) for n, w in model.params.items()}
    model.rows.fill_(float("nan"))  # every gradient is written whole
    total, mags = {n: 0.0 for n in p}, {n: 0.0 for n in p}
    for r in range(world):
        loss = model.replica_step(r, ids[r], targets[r])
        want = loss64(model, p, ids[r], targets[r].double())
        assert abs(float(loss) - float(want.detach())) <= 10 * 2.0 ** -8 * float(want.detach())
        for n, d in zip(p, torch.autograd.grad(want, list(p.values()))):
            got = model.gradient(r, n).double()
            assert float((got - d).norm()) <= 10 * 2.0 ** -8 * float(d.norm()), n
            total[n], mags[n] = total[n] + got / world, mags[n] + got.abs() / world
    assert bool(torch.isfinite(model.rows).all()) and zc.device_status() == 0
    model.ex.flush_all(model.rows)
    want = torch.sqrt(sum(t.square().sum() for t in total.values()))
    half = float(want) / 2
    norm, c = model.clip.clip(half).tolist()
    # the reduced gradients are bf16: each is off by 2^-8 of itself at most, and by the
    # fp32 roundings of its terms (a division and an addition of each rank, 2^-24 of
    # the terms' magnitudes), which are all that is left where the terms cancel
    assert abs(norm - float(want)) <= 2.0 ** -8 * norm and abs(c - half / (norm + 1e-6)) <= 1e-6
    for i, n in enumerate(model.names):
        held = [v for r in range(world) if (v := model.ex.grad.view(r, i)) is not None]
        assert held
        for v in held:
            want, slack = total[n].flatten() * c, 2 * world * 2.0 ** -24 * c * mags[n].flatten()
            assert bool(((v.double() - want).abs() <= 2.1 * 2.0 ** -8 * want.abs() + slack + 1e-30).all()), n


def test_padding_gives_no_gradient():
    model = example().Model(1, 50, 64, 96, 1)
    ids, targets = inputs(model, 64)
    ids[0][::2] = 7
    model.replica_step(0, ids[0], targets[0], padding=7)
    assert not bool(model.gradient(0, "embed")[7].any())
    others = model.gradient(0, "embed").clone()
    model.replica_step(0, ids[0], targets[0])
    assert bool(model.gradient(0, "embed")[7].any())
    others[7] = model.gradient(0, "embed")[7]
    assert torch.equal(others, model.gradient(0, "embed"))


def test_steps_in_a_captured_graph():
    """A replica's forward and backward, the flush and the clipping, captured and
    replayed on new tokens, leave the bits of plain calls."""
    model = example().Model(2, 400, 128, 192, 2)
    ids, targets = inputs(model, 200)
    held = [i.clone() for i in ids], [t.clone() for t in targets]

    def run():
        for r in range(2):
            model.replica_step(r, held[0][r], held[1][r])
        model.ex.flush_all(model.rows)
        return model.clip.clip(1e-3)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = run()
    for seed in (5, 6):
        new = inputs(model, 200, seed)
        for a, b in zip((*held[0], *held[1]), (*new[0], *new[1])):
            a.copy_(b)
        graph.replay()
        got = [norm.clone(), model.rows.clone(), *(b.clone() for b in model.ex.grad.buf)]
        want = [run(), model.rows, *model.ex.grad.buf]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for r in range(2):
            for i in range(len(model.names)):
                if model.ex.grad.view(r, i) is not None:
                    s = model.ex.grad.slot[r][i]
                    n = int(model.ex.grad.numel[i])
                    assert torch.equal(got[2 + r][s:s + n], want[2 + r][s:s + n])


def test_example_runs():
    m = example()
    model = m.Model(2, 200, 64, 96, 2)
    ids, targets = inputs(model, 100)
    before = {n: w.clone() for n, w in model.params.items()}
    loss, norm = model.step(ids, targets)
    assert np.isfinite(float(loss)) and bool(torch.isfinite(norm).all()) and float(norm[1]) <= 1
    assert all(bool(torch.isfinite(w).all()) for w in model.params.values())
    assert all(not torch.equal(before[n], w) for n, w in model.params.items() if n != "embed")
    assert not torch.equal(before["embed"][ids[0]], model.params["embed"][ids[0]])
    assert zc.device_status() == 0
