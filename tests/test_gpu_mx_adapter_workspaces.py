"""The adapters' calls whose workspaces hold sums: on a given stream, two at once, in graphs that share a pool, and through
the C ABI with the workspace's neighbours left as they were."""
import pytest
import torch

import mx_block_scaled_x128_amd as mx

pytestmark = pytest.mark.gpu
NAMES = ["grad", "grad transposed", "grad of two", "project", "product"]


def _calls():
    """name -> a call that takes stream and has a workspace of sums; every input is on the device and ready."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows, cols, n, rank = 4096, 2048, 320, 16

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    q, s, _ = mx.quantize_mx(normal(rows, cols), mx.E4M3, mx.RULE_CEIL)
    q4, s4 = mx.quantize_mxfp4(normal(n, cols))
    down, up, p = normal(2, rank, cols).bfloat16(), normal(2, n, rank).bfloat16(), normal(rows, rank)
    one = torch.zeros(rows, dtype=torch.int32, device="cuda")
    two = (torch.arange(rows, device="cuda") % 3 - 1).int()
    for adapters in (1, 2):
        assert mx.mx_adapter_grad_workspace(rows, cols, rank, adapters) > 0
    assert mx.mx_adapter_project_workspace(rows, cols, rank) > 0
    torch.cuda.synchronize()

    def grad(ids, adapters, transposed):
        return lambda stream: (mx.adapter_grad_mx(p, q, s, mx.E4M3, ids, adapters, transposed, stream=stream),)
    return {
        "grad": grad(one, 1, False), "grad transposed": grad(one, 1, True), "grad of two": grad(two, 2, False),
        "project": lambda stream: (mx.adapter_project_mx(q, s, mx.E4M3, down, two, stream=stream),),
        "product": lambda stream: mx.mxfp4_adapted_gemm(q, s, mx.E4M3, q4, s4, down, up, two, stream=stream),
    }


def _same(got, want):
    for g, w in zip(got, want, strict=True):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once(name):
    """One on the current stream behind queued work and one on a side stream, whose blocks are used again at once."""
    call, side = _calls()[name], torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    for _ in range(3):
        hold = torch.ones(16 << 20, device="cuda")
        for _ in range(40):
            hold.mul_(1.0001)
        got = call(None), call(side), call(side)
        torch.cuda.synchronize()
        for out in got:
            _same(out, want)


@pytest.mark.parametrize("name", NAMES)
def test_a_side_stream_in_a_captured_graph(name):
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
        _same(out, want)
        call(None)


def test_two_graphs_with_a_pool_in_common():
    calls = _calls()
    want = {name: [t.clone() for t in calls[name](None)] for name in NAMES}
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=graphs[0].pool() if graphs else None):
            outs.append([calls[name](None) for name in NAMES])
        graphs.append(graph)
    for k in (0, 1, 1, 0, 1):
        graphs[k].replay()
        torch.cuda.synchronize()
        for got, name in zip(outs[k], NAMES, strict=True):
            _same(got, want[name])


@pytest.mark.parametrize("M,C,rank,adapters", [(4096, 2048, 16, 1), (3000, 544, 40, 2), (5000, 96, 8, 3)])
def test_bytes_around_the_workspace(M, C, rank, adapters):
    """The C call on a workspace of exactly the bytes asked for: what lies before and behind it, and grad, stays."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    z, sz, _ = mx.quantize_mx(torch.randn(M, C, generator=gen, device="cuda"), mx.E4M3, mx.RULE_CEIL)
    p = torch.randn(M, rank, generator=gen, device="cuda")
    ids = (torch.arange(M, device="cuda") % adapters).int()
    want = mx.adapter_grad_mx(p, z, sz, mx.E4M3, ids, adapters)
    n, pad = mx.mx_adapter_grad_workspace(M, C, rank, adapters), 4096
    assert n > 0
    work = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((want.numel() + 2 * pad,), 7.0, device="cuda")
    st = mx.mx_adapter_grad(M, C, z.data_ptr(), z.stride(0), mx.E4M3, sz.data_ptr(), p.data_ptr(), rank, ids.data_ptr(), adapters,
                            0, out[pad:].data_ptr(), work[pad:].data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(out[pad:-pad].view_as(want), want)
    assert (out[:pad] == 7.0).all() and (out[-pad:] == 7.0).all()
    assert (work[:pad] == 0x5A).all() and (work[pad + n:] == 0x5A).all()
