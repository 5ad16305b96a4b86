"""The quantizers', products' and sampler's tensor functions with stream=: their outputs are
that stream's memory, and may be read on the caller's stream until they are dropped."""
import pytest
import torch

import mx_block_scaled_x128_amd as mx
from test_gpu_mx_streams import _busy, _owner

pytestmark = pytest.mark.gpu


def _calls(rows=256, cols=512):
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, w = (torch.randn(rows, cols, generator=gen, device="cuda") for _ in range(2))
    q, s = mx.quantize_token(x)
    b, sb = mx.quantize_block(w)
    qf, sf = mx.quantize_token_f32s(x)
    bf, sbf = mx.quantize_block_f32s(w)
    qm, sm, _ = mx.quantize_mx(x)
    bits = torch.full((rows // 32, cols // 32), 6, dtype=torch.int8, device="cuda")
    torch.cuda.synchronize()
    return {
        "quantize_token": lambda st: mx.quantize_token(x, stream=st),
        "quantize_token_t": lambda st: mx.quantize_token(x, axis=mx.COL_T, stream=st),
        "quantize_block": lambda st: mx.quantize_block(w, stream=st),
        "quantize_token_f32s": lambda st: mx.quantize_token_f32s(x, stream=st),
        "quantize_token_f32s_t": lambda st: mx.quantize_token_f32s(x, axis=mx.COL_T, stream=st),
        "quantize_block_f32s": lambda st: mx.quantize_block_f32s(w, stream=st),
        "quantize_token_dual": lambda st: mx.quantize_token_dual(x, stream=st),
        "quantize_block_dual": lambda st: mx.quantize_block_dual(w, stream=st),
        "quantize_mx": lambda st: mx.quantize_mx(x, stream=st),
        "block_scaled_gemm": lambda st: (mx.block_scaled_gemm(q, s, mx.E4M3, b, sb, mx.E4M3, stream=st),),
        "gemm_f32s": lambda st: (mx.gemm_f32s(qf, sf, mx.E4M3, bf, sbf, mx.E4M3, stream=st),),
        "mx_scaled_gemm": lambda st: (mx.mx_scaled_gemm(qm, sm, mx.E4M3, qm, sm, mx.E4M3, stream=st),),
        "gaussws": lambda st: (mx.gaussws(w, bits, 5, stream=st),),
    }


NAMES = ["quantize_token", "quantize_token_t", "quantize_block", "quantize_token_f32s", "quantize_token_f32s_t",
         "quantize_block_f32s", "quantize_token_dual", "quantize_block_dual", "quantize_mx", "block_scaled_gemm",
         "gemm_f32s", "mx_scaled_gemm", "gaussws"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_on_a_given_stream(name):
    call, side = _calls()[name], torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    before = torch.cuda.current_stream()
    first = call(side)
    assert torch.cuda.current_stream() == before
    assert all(_owner(t) == side.cuda_stream for t in first)
    # read behind other work on the caller's stream, dropped at once
    before.wait_stream(side)
    hold = _busy()
    read = [t.clone() for t in first]
    taken = {t.data_ptr() for t in first}
    del first
    second = call(side)
    assert not taken & {t.data_ptr() for t in second}
    torch.cuda.synchronize()
    del hold
    for r, s, w in zip(read, second, want):
        assert torch.equal(r, w) and torch.equal(s, w)
