"""The gradient of the block norm over the matrix of a gate per token: an output
may be an input of its type and stride."""
import pytest
import torch

from tests.test_gpu_block_norm import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,d", [(7, 256), (7, 777), (5, 8200), (5, 16384), (5, 16383), (400, 16384)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_dx_over_the_gate(m, d, stream):
    c = Case(m, d, stream=stream, gate=m, weights=stream)
    want = c.backward(c.grads())
    k = Case(m, d, stream=stream, gate=m, weights=stream)
    got = k.backward(k.grads(), dx=k.gate)
    assert got[0] is k.gate and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("m,d", [(7, 777), (5, 16384), (5, 16383)])
def test_gate_gradient_over_the_gate(m, d):
    c = Case(m, d, stream=torch.float32, gate=m, weights=torch.float32)
    grads = c.grads()
    want = c.backward(grads)
    k = Case(m, d, stream=torch.float32, gate=m, weights=torch.float32)
    got = k.backward(dict(k.grads(), gate_grad=k.gate))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(k.gate, grads["gate_grad"])
