"""LayerNorm's and the adapters' tensor functions with stream=: what they allocate, workspaces too, belongs to
that stream, and what they return may be read on the caller's stream until it is dropped."""
import pytest
import torch

import mx_block_scaled_x128_amd as mx

pytestmark = pytest.mark.gpu
NAMES = ["layernorm_mx", "layernorm_mx_backward", "adapter_project_mx", "mxfp4_adapted_gemm few rows",
         "mxfp4_adapted_gemm tiles", "adapter_grad_mx"]


def _calls():
    """name -> a call that takes stream; every input is on the device and ready.  The rows are enough for the
    projection's and the gradients' workspaces."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows, cols, n, rank, adapters = 640, 2048, 320, 16, 3

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    x, w, b, dy = normal(rows, cols), normal(cols), normal(cols), normal(rows, cols)
    q, s, _ = mx.quantize_mx(x, mx.E4M3, mx.RULE_CEIL)
    q4, s4 = mx.quantize_mxfp4(normal(n, cols))
    down, up = normal(adapters, rank, cols).bfloat16(), normal(adapters, n, rank).bfloat16()
    ids = (torch.arange(rows, device="cuda") * 5 % (adapters + 1) - 1).int()
    alpha, p = normal(adapters), normal(rows, rank)
    kept = mx.layernorm_mx(x, w, b, 1e-5)[2]
    torch.cuda.synchronize()

    def product(m):
        return lambda stream: mx.mxfp4_adapted_gemm(q[:m], s[:m], mx.E4M3, q4, s4, down, up, ids[:m], alpha, stream=stream)

    def norm(stream):
        out = mx.layernorm_mx(x, w, b, 1e-5, stream=stream)
        return (*out[:2], *(t for t in out[2] if torch.is_tensor(t)))
    return {
        "layernorm_mx": norm,
        "layernorm_mx_backward": lambda stream: mx.layernorm_mx_backward(kept, w, dy, stream=stream),
        "adapter_project_mx": lambda stream: (mx.adapter_project_mx(q, s, mx.E4M3, down, ids, alpha, stream=stream),),
        "mxfp4_adapted_gemm few rows": product(37),
        "mxfp4_adapted_gemm tiles": product(rows),
        "adapter_grad_mx": lambda stream: (mx.adapter_grad_mx(p, q, s, mx.E4M3, ids, adapters, stream=stream),),
    }


def _busy(n=400):
    """Several milliseconds of elementwise work on the current stream, many times what a call takes the host."""
    t = torch.ones(16 << 20, device="cuda")
    for _ in range(n):
        t.mul_(1.0001)
    return t


def _owner(t):
    """The stream whose memory holds t."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_the_given_streams_memory(name):
    call, side = _calls()[name], torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    before = torch.cuda.current_stream()
    got = call(side)
    assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
    for g, w in zip(got, want, strict=True):
        assert torch.equal(g, w)
        assert _owner(g) == side.cuda_stream and _owner(w) == before.cuda_stream


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once(name):
    """One on the current stream behind queued work, one on a side stream at once: each has its own workspace."""
    call, side = _calls()[name], torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    for _ in range(3):
        hold = _busy(40)
        got = call(None), call(side)
        torch.cuda.synchronize()
        for out in got:
            for g, w in zip(out, want, strict=True):
                assert torch.equal(g, w)
        del hold, got


@pytest.mark.parametrize("name", NAMES)
def test_an_output_read_on_the_callers_stream_and_dropped(name):
    """The caller waits for the side stream, reads the output behind other work and drops it at once; the next call
    on the side stream takes other memory."""
    call, side = _calls()[name], torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    first = call(side)
    torch.cuda.current_stream().wait_stream(side)
    hold = _busy()
    read = [t.clone() for t in first]
    taken = {t.data_ptr() for t in first}
    del first
    second = call(side)
    assert not taken & {t.data_ptr() for t in second}
    with torch.cuda.stream(side):
        for t in second:
            t.zero_()
    torch.cuda.synchronize()
    del hold
    for r, w in zip(read, want, strict=True):
        assert torch.equal(r, w)


@pytest.mark.parametrize("name", NAMES)
def test_a_side_stream_in_a_captured_graph(name):
    """A side stream forked from the capturing one: replays give the eager results."""
    call, side = _calls()[name], torch.cuda.Stream()
    want = call(None)
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(out, want, strict=True):
            assert torch.equal(g, w)
        call(None)


def test_two_graphs_with_a_pool_in_common():
    """Two captured graphs that share a memory pool, and so their workspaces, replayed one after the other."""
    calls = _calls()
    graphs, outs = [], []
    for name in NAMES:
        calls[name](None)
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=graphs[0].pool() if graphs else None):
            outs.append([calls[name](None) for name in NAMES])
        graphs.append(graph)
    want = [[t.clone() for t in calls[name](None)] for name in NAMES]
    for k in (0, 1, 1, 0, 1):
        graphs[k].replay()
        torch.cuda.synchronize()
        for got, exp in zip(outs[k], want, strict=True):
            for g, w in zip(got, exp, strict=True):
                assert torch.equal(g, w)
