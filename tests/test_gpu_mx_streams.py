"""The MX operators' tensor functions with stream=: what they allocate belongs to that
stream, so that nothing that another stream still uses is written, and what they return
may be read on the caller's stream until it is dropped."""
import pytest
import torch

import mx_block_scaled_x128_amd as mx

pytestmark = pytest.mark.gpu


def _busy(n=400):
    """Several milliseconds of elementwise work on the current stream, many times what a call takes the host."""
    t = torch.ones(16 << 20, device="cuda")
    for _ in range(n):
        t.mul_(1.0001)
    return t


def _calls(rows=256, cols=512):
    """name -> a call that takes stream; every input is on the device and ready."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(r, c):
        return torch.randn(r, c, generator=gen, device="cuda")
    x, gu, dh, w = normal(rows, cols), normal(rows, 2 * cols), normal(rows, cols), torch.rand(cols, device="cuda")
    q, s, _ = mx.quantize_mx(x, mx.E4M3, mx.RULE_CEIL)
    b, sb = mx.quantize_mxfp4(normal(320, cols))
    act, norm = mx.swiglu_mx(gu)[2], mx.rmsnorm_mx(x, w, 1e-6)[2]
    torch.cuda.synchronize()
    return {
        "quantize_mxfp4": lambda stream: mx.quantize_mxfp4(x, stream=stream),
        "dequantize_mx": lambda stream: (mx.dequantize_mx(q, s, mx.E4M3, stream=stream),),
        "quantize_mx_t": lambda stream: mx.quantize_mx_t(x, stream=stream),
        "requantize_mx_t": lambda stream: mx.requantize_mx_t(q, s, mx.E4M3, stream=stream),
        "mxfp4_scaled_gemm": lambda stream: (mx.mxfp4_scaled_gemm(q, s, mx.E4M3, b, sb, stream=stream),),
        "swiglu_mx": lambda stream: _flat(mx.swiglu_mx(gu, stream=stream)),
        "swiglu_mx_backward": lambda stream: (mx.swiglu_mx_backward(act, dh, stream=stream),),
        "rmsnorm_mx": lambda stream: _flat(mx.rmsnorm_mx(x, w, 1e-6, stream=stream)),
        "rmsnorm_mx_backward": lambda stream: mx.rmsnorm_mx_backward(norm, w, dh, stream=stream),
    }


def _flat(out):
    return (*out[:2], *(t for t in out[2] if torch.is_tensor(t)))


NAMES = ["quantize_mxfp4", "dequantize_mx", "quantize_mx_t", "requantize_mx_t", "mxfp4_scaled_gemm", "swiglu_mx",
         "swiglu_mx_backward", "rmsnorm_mx", "rmsnorm_mx_backward"]


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
    for g, w in zip(got, want):
        assert torch.equal(g, w)
        assert _owner(g) == side.cuda_stream and _owner(w) == before.cuda_stream


def test_two_backward_passes_at_once():
    """One on the current stream behind queued work, one of the same size on a side stream at once: each has a
    workspace of its own, and both dw are what they are alone."""
    rows, cols = 2048, 1024
    w, side = torch.rand(cols, device="cuda"), torch.cuda.Stream()
    kept = mx.rmsnorm_mx(torch.randn(rows, cols, device="cuda"), w, 1e-6)[2]
    dy = [torch.randn(rows, cols, device="cuda") for _ in range(2)]
    want = [mx.rmsnorm_mx_backward(kept, w, d) for d in dy]
    torch.cuda.synchronize()
    for _ in range(5):
        hold = _busy(40)
        got = [mx.rmsnorm_mx_backward(kept, w, dy[0]), mx.rmsnorm_mx_backward(kept, w, dy[1], stream=side)]
        torch.cuda.synchronize()
        for g, e in zip(got, want):
            assert torch.equal(g[0], e[0]) and torch.equal(g[1], e[1])
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
    for r, w in zip(read, want):
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
        for g, w in zip(out, want):
            assert torch.equal(g, w)
        call(None)
