"""Rows of any alignment whose slots in a block's ring take many rows in turn: the
ends of the matrices are copied element by element into slots that bulk copies
fill before and after them."""
import pytest
import torch

from tests.test_gpu_block_norm import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,d,pad,shift", [(60000, 33, 0, 1), (60000, 97, 2, 3), (20000, 777, 0, 5), (8000, 4097, 0, 7)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_many_turns(m, d, pad, shift, stream):
    c = Case(m, d, stream=stream, pad=pad, shift=shift)
    c.check_forward(*c.forward())
    grads = c.grads()
    c.check_backward(*c.backward(grads), grads)
    t = Case(m, d, stream=stream, gate=m, pad=pad, shift=shift)
    t.check_forward(*t.forward())
