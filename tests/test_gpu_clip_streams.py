"""GradClip on streams other than the one it was made on, and in graphs that live
longer than it: the partial sums of a call lie in memory of the call's stream."""
import pytest
import torch

import zero_collectives_gb300 as zc
from zero_collectives_gb300 import layers

pytestmark = pytest.mark.gpu


def gradients(seed=1):
    """More than one cluster takes in one launch, so that partial sums go through
    the workspace."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(3000, 1024, device="cuda", generator=g), torch.randn(777, device="cuda", generator=g)]


def stream_of(address):
    """The stream whose pool the allocator took an address from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= address < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError(f"{address:#x} is no memory of the allocator")


@pytest.fixture
def spaces(monkeypatch):
    """The addresses of the workspaces that calls get."""
    got, call = [], layers._call

    def watched(name, *args):
        got.append(args[{"grad_norm": 3, "clip_grads": 5}[name]])
        call(name, *args)
    monkeypatch.setattr(layers, "_call", watched)
    return got


@pytest.mark.parametrize("as_integer", [False, True])
def test_workspace_belongs_to_the_stream_of_the_call(spaces, as_integer):
    grads = gradients()
    clip = zc.GradClip(grads)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    clip.norm(stream=s.cuda_stream if as_integer else s)
    clip.clip(0.5, stream=s)
    with torch.cuda.stream(s):
        clip.norm()
    torch.cuda.synchronize()
    clip.norm()
    torch.cuda.synchronize()
    assert [stream_of(p) for p in spaces] == [s.cuda_stream] * 3 + [torch.cuda.current_stream().cuda_stream]
    assert spaces[3] == clip.workspace.data_ptr()


def test_object_that_is_dropped_while_its_call_waits(spaces):
    """The call's memory is not given to the stream that made the object."""
    grads = gradients()
    want = zc.clip_grads([g.clone() for g in grads], 0.5)
    clip = zc.GradClip(grads)
    size = clip.workspace.numel()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        held = torch.ones(1 << 28, device="cuda")  # some milliseconds of work before the call
        for _ in range(20):
            held.mul_(1.0)
    got = clip.clip(0.5, stream=s)
    del clip
    others = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(20)]  # NaN as partial sums
    assert not any(o.data_ptr() <= spaces[-1] < o.data_ptr() + size for o in others)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((o == 255).all()) for o in others)


@pytest.mark.parametrize("own_stream", [False, True])
def test_graph_that_outlives_the_object(own_stream):
    """Captured on the stream that made the object, or on another."""
    grads = gradients()
    start = [g.clone() for g in grads]
    want = zc.clip_grads([g.clone() for g in grads], 0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s if own_stream else torch.cuda.current_stream()):
        clip = zc.GradClip(grads)
    size = clip.workspace.numel()
    out = torch.empty(2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        clip.clip(0.5, out=out)
    torch.cuda.synchronize()
    del clip
    with torch.cuda.stream(s):
        others = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(20)]
    others += [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(20)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, x in zip(grads, start):
            g.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((o == 255).all()) for o in others)
