"""The operators around the products from several threads and streams at once: the
results of one thread, to the bit."""
import threading

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu


def work_of(i, stream=None):
    """One pass through all of them on inputs of its own."""
    g = torch.Generator(device="cuda").manual_seed(i)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)

    t, v, d = 700 + i, 90, 264 + 8 * i + i % 2
    ids, table = torch.randint(0, v, (t,), device="cuda", generator=g), randn(v, d)
    y, post, pre, gate = randn(t, d), randn(d, dtype=torch.float32), randn(d, dtype=torch.float32), randn(d, dtype=torch.float32)
    start = [randn(3000, 500), randn(4000, 77, dtype=torch.float32)]
    grads = [torch.empty_like(x) for x in start]
    weights = [torch.zeros(d, device="cuda") for _ in range(3)]
    dw = torch.empty(v, d, device="cuda")
    torch.cuda.synchronize()
    clip = zc.GradClip(grads)

    def work():
        on = dict(stream=stream)
        x = zc.embedding(ids, table, **on)
        r, h = zc.block_norm(x, y=y, post=post, gate=gate, pre=pre, **on)
        dx, dy = zc.block_norm_grad(r, dr=x, dh=h, y=y, post=post, gate=gate, pre=pre, post_grad=weights[0], gate_grad=weights[1],
                                    pre_grad=weights[2], **on)
        zc.embedding_grad(ids, dx, dw, **on)
        with torch.cuda.stream(stream):
            for a, b in zip(grads, start):
                a.copy_(b)
        result = clip.clip(1.0, **on)
        norm = zc.grad_norm([dx, dy], **on)
        with torch.cuda.stream(stream):
            return [z.clone() for z in (x, r, h, dx, dy, dw, *weights, result, norm, *grads)]
    return work


def test_threads_and_streams():
    n = 4
    want = [work_of(i)() for i in range(n)]
    streams = [torch.cuda.Stream() for _ in range(n)]
    calls = [work_of(i, streams[i // 2]) for i in range(n)]  # two threads share a stream
    torch.cuda.synchronize()
    got = [[] for _ in range(n)]

    def run(i):
        for _ in range(15):
            got[i].append(calls[i]())

    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(n):
        assert len(got[i]) == 15
        assert all(torch.equal(a, b) for one in got[i] for a, b in zip(one, want[i])), i
    assert zc.device_status() == 0
