"""LayerNorm and the adapters on padded inputs: what lies between the rows, and between the adapters, is NaN and changes
no bit; adapters that share their memory (a stride of zero)."""
import pytest
import torch

import mx_block_scaled_x128_amd as mx

pytestmark = pytest.mark.gpu


def padded(t, pad, fill):
    """t's values in rows `pad` elements apart more (matrices 3 pad more), everything between them `fill`."""
    rows, cols = t.shape[-2:]
    n = t.shape[0] if t.dim() == 3 else 1
    step = rows * (cols + pad) + (3 * pad if t.dim() == 3 else 0)
    flat = torch.full((n * step + pad,), fill, dtype=t.dtype, device="cuda")
    shape, strides = ((n, rows, cols), (step, cols + pad, 1)) if t.dim() == 3 else ((rows, cols), (cols + pad, 1))
    return flat.as_strided(shape, strides).copy_(t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 544), (600, 3584), (5, 8960), (3, 20480)])
def test_layernorm(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, dy = (torch.randn(rows, cols, generator=gen, device="cuda").to(dtype) for _ in range(2))
    w, b = (torch.randn(cols, generator=gen, device="cuda") for _ in range(2))
    y, ys, kept = mx.layernorm_mx(x, w, b, 1e-5)
    y2, ys2, kept2 = mx.layernorm_mx(padded(x, 16, float("nan")), w, b, 1e-5)
    assert torch.equal(y, y2) and torch.equal(ys, ys2) and all(torch.equal(p, q) for p, q in zip(kept[:3], kept2[:3]))
    want = mx.layernorm_mx_backward(kept, w, dy)
    got = mx.layernorm_mx_backward(kept._replace(codes=padded(kept.codes, 16, 0x7F)), w, padded(dy, 16, float("nan")))
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2, mx.E2M1])
@pytest.mark.parametrize("M,K,N,rank", [(3, 384, 100, 8), (61, 1152, 520, 24), (300, 256, 2100, 40), (700, 1536, 300, 16),
                                        (4100, 128, 4352, 136)])
def test_adapters(M, K, N, rank, fmt):
    gen = torch.Generator(device="cuda").manual_seed(M)
    x, w = torch.randn(M, K, generator=gen, device="cuda"), torch.randn(N, K, generator=gen, device="cuda")
    a, sa = mx.quantize_mxfp4(x) if fmt == mx.E2M1 else mx.quantize_mx(x, fmt, mx.RULE_CEIL, counts=False)[:2]
    b, sb = mx.quantize_mxfp4(w)
    down, up = (torch.randn(3, *s, generator=gen, device="cuda").bfloat16() for s in ((rank, K), (N, rank)))
    ids = torch.randint(-1, 3, (M,), generator=gen, device="cuda", dtype=torch.int32)
    nan = float("nan")
    wide = padded(a, 16, 0xFF), sa, fmt, padded(b, 16, 0xFF), sb, padded(down, 8, nan), padded(up, 8, nan), ids
    for dtype in (torch.float32, torch.bfloat16):
        y, p = mx.mxfp4_adapted_gemm(a, sa, fmt, b, sb, down, up, ids, out_dtype=dtype)
        y2, p2 = mx.mxfp4_adapted_gemm(*wide, out_dtype=dtype)
        assert torch.isfinite(y).all() and torch.equal(y, y2) and torch.equal(p, p2)
    assert torch.equal(mx.adapter_grad_mx(p, a, sa, fmt, ids, 3), mx.adapter_grad_mx(p, wide[0], sa, fmt, ids, 3))
    # one matrix under three names: the same products, added in another order where the few-row kernel deals the
    # adapters that are named to its waves (rank + 16 additions of each call, 2^-24 of the sizes)
    one = down[:1].expand(3, -1, -1), up[:1].expand(3, -1, -1)
    y, p = mx.mxfp4_adapted_gemm(a, sa, fmt, b, sb, *one, ids)
    y2, p2 = mx.mxfp4_adapted_gemm(a, sa, fmt, b, sb, down[:1], up[:1], ids.clamp(max=0))
    assert torch.equal(p, p2)
    size = p.abs() @ up[0].float().abs().t() + mx.dequantize_mx(a, sa, fmt).abs() @ mx.dequantize_mx(b, sb, mx.E2M1).abs().t()
    assert ((y - y2).abs() <= 2 * (rank + 16) * 2.0 ** -24 * size).all()
