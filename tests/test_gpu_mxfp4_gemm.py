"""mxfp4_gemm against fp64 products over the same codes (E2M1 on the right; E2M1, E4M3 or
E5M2 on the left).

Tolerance: 2^-12 * sum |a b| per element, as for the other products, and for bf16 output one
rounding (2^-8) more.  E2M1 products span 6 binades and are exact in the matrix cores; what is
left for two E2M1 operands is the fp32 accumulation."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref
from gpu_helpers import assert_gemm_close, dev, dev_ld16, host

pytestmark = pytest.mark.gpu
FMTS = [mx.E2M1, mx.E4M3, mx.E5M2]


def operand(rows, K, fmt, seed, spread=6):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (rows, K)) * mxref.pow2(rng.integers(-spread, spread + 1, (rows, K // 32)).repeat(32, axis=1))
    return mxref.quantize(x, fmt, mxref.CEIL)


def product(a, sa, a_fmt, b, sb):
    A, B = mxref.dequantize(a, sa, a_fmt), mxref.dequantize(b, sb, mxref.E2M1)
    return A @ B.T, np.abs(A) @ np.abs(B).T


def run(a, sa, a_fmt, b, sb, dtype, pad=0):
    a_d = dev(a, pitch=a.shape[1] + pad) if a.shape[1] else dev(a)
    b_d = dev(b, pitch=b.shape[1] + pad) if b.shape[1] else dev(b)
    out = mx.mxfp4_scaled_gemm(a_d, dev(sa), a_fmt, b_d, dev(sb), out_dtype=dtype)
    torch.cuda.synchronize()
    return host(out)


SHAPES = [(1, 1, 128), (1, 16, 256), (1, 300, 3584), (2, 100, 384), (15, 17, 640), (16, 256, 1152), (17, 33, 256),
          (33, 520, 128), (37, 1536, 1280), (64, 64, 512), (65, 70, 896), (100, 258, 384), (128, 128, 256),
          (129, 300, 640), (200, 515, 1024), (256, 256, 512), (300, 260, 128), (520, 1030, 1664)]


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(M, N, K, a_fmt):
    a, sa = operand(M, K, a_fmt, M)
    b, sb = operand(N, K, mx.E2M1, N + 7)
    y, t = product(a, sa, a_fmt, b, sb)
    assert_gemm_close(run(a, sa, a_fmt, b, sb, torch.float32, pad=16), y, t, False)
    assert_gemm_close(run(a, sa, a_fmt, b, sb, torch.bfloat16), y, t, True)


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N", [(3, 40), (40, 40), (140, 150), (300, 600)])
def test_each_element_meets_its_partner_and_scales(M, N, a_fmt):
    """One nonzero element per row of A, random everything in B: the product is a single
    term, exact in fp32, so a wrong k, row or scale anywhere shows."""
    K = 768
    rng = np.random.default_rng(M)
    a = np.zeros((M, K), dtype=np.uint8)
    at = (np.arange(M) * 131) % K
    a[np.arange(M), at] = mxref.cast(np.array([1.5]), a_fmt)[0]
    a = mxref.pack(a) if a_fmt == mx.E2M1 else a
    sa = rng.integers(117, 138, (M, K // 32)).astype(np.uint8)
    b = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    sb = rng.integers(117, 138, (N, K // 32)).astype(np.uint8)
    y, _ = product(a, sa, a_fmt, b, sb)
    assert np.array_equal(run(a, sa, a_fmt, b, sb, torch.float32).astype(np.float64), y)


@pytest.mark.parametrize("M,N", [(5, 64), (70, 96), (260, 300)])
def test_whole_sums_are_exact(M, N):
    """E2M1 codes under scales of 1: every partial sum is a multiple of 1/4 below 2^22, exact in fp32."""
    K = 2048
    rng = np.random.default_rng(N)
    a = rng.integers(0, 256, (M, K // 2)).astype(np.uint8)
    b = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    sa, sb = np.full((M, K // 32), 127, np.uint8), np.full((N, K // 32), 127, np.uint8)
    y, _ = product(a, sa, mx.E2M1, b, sb)
    assert np.array_equal(run(a, sa, mx.E2M1, b, sb, torch.float32).astype(np.float64), y)


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(8, 512, 512), (512, 512, 512)])
def test_nan_blocks_reach_their_outputs_only(M, N, K, a_fmt):
    a, sa = operand(M, K, a_fmt, 1)
    b, sb = operand(N, K, mx.E2M1, 2)
    sa[3, 2] = 255
    sb[40, K // 32 - 1] = 255
    y = run(a, sa, a_fmt, b, sb, torch.float32)
    want = np.zeros((M, N), bool)
    want[3, :] = want[:, 40] = True
    assert np.array_equal(np.isnan(y), want)


@pytest.mark.parametrize("a_fmt", FMTS)
def test_k_zero_and_padding(a_fmt):
    e = torch.empty((5, 0), dtype=torch.uint8, device="cuda")
    y = mx.mxfp4_scaled_gemm(e, e, a_fmt, torch.empty((40, 0), dtype=torch.uint8, device="cuda"),
                             torch.empty((40, 0), dtype=torch.uint8, device="cuda"))
    assert y.shape == (5, 40) and not host(y).any()
    for M in (5, 300):
        a, sa = operand(M, 256, a_fmt, 1)
        b, sb = operand(50, 256, mx.E2M1, 2)
        buf = torch.full((M, 64), 7.0, device="cuda")
        mx.mxfp4_scaled_gemm(dev_ld16(a), dev(sa), a_fmt, dev_ld16(b), dev(sb), out=buf[:, :50])
        ref, t = product(a, sa, a_fmt, b, sb)
        assert_gemm_close(host(buf)[:, :50], ref, t, False)
        assert (host(buf)[:, 50:] == 7.0).all()


@pytest.mark.parametrize("a_fmt", FMTS)
def test_same_bits_every_time(a_fmt):
    for M in (4, 48, 400):
        a, sa = operand(M, 1024, a_fmt, 1)
        b, sb = operand(700, 1024, mx.E2M1, 2)
        first = run(a, sa, a_fmt, b, sb, torch.float32)
        for _ in range(3):
            assert np.array_equal(run(a, sa, a_fmt, b, sb, torch.float32), first)


def test_quantize_then_product():
    """The library's own codes through the product: forward, and the data gradient on the transposed weight."""
    rng = np.random.default_rng(0)
    x, w = rng.normal(0, 1, (200, 256)).astype(np.float32), rng.normal(0, 0.02, (384, 256)).astype(np.float32)
    dy = rng.normal(0, 1e-3, (200, 384)).astype(np.float32)
    wq, ws = mx.quantize_mxfp4(torch.from_numpy(w).cuda())
    wt, wts = mx.quantize_mx_t(torch.from_numpy(w).cuda(), mx.E2M1, mx.RULE_FLOOR)
    xq, xs, _ = mx.quantize_mx(torch.from_numpy(x).cuda(), mx.E4M3, mx.RULE_CEIL)
    gq, gs, _ = mx.quantize_mx(torch.from_numpy(dy).cuda(), mx.E5M2, mx.RULE_CEIL)
    y = mx.mxfp4_scaled_gemm(xq, xs, mx.E4M3, wq, ws)
    dx = mx.mxfp4_scaled_gemm(gq, gs, mx.E5M2, wt, wts)
    assert_gemm_close(host(y), *product(host(xq), host(xs), 0, host(wq), host(ws)), False)
    assert_gemm_close(host(dx), *product(host(gq), host(gs), 1, host(wt), host(wts)), False)


def test_full_k_and_large_extents():
    """Long K at every few-row width, and a wide N: sums over 18944."""
    for M, N, K, fmt in ((1, 512, 18944, mx.E4M3), (24, 512, 18944, mx.E2M1), (512, 512, 18944, mx.E5M2),
                         (2, 40000, 128, mx.E2M1), (3000, 64, 256, mx.E4M3)):
        a, sa = operand(M, K, fmt, 1, spread=0)
        b, sb = operand(N, K, mx.E2M1, 2, spread=0)
        y, t = product(a, sa, fmt, b, sb)
        assert_gemm_close(run(a, sa, fmt, b, sb, torch.float32), y, t, False, what=str((M, N, K)))


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(900, 900, 128), (900, 900, 256), (2100, 420, 384), (700, 1100, 0)])
def test_tiles_with_one_k_block_or_none(M, N, K, a_fmt):
    a, sa = operand(M, K, a_fmt, 3) if K else (np.zeros((M, 0), np.uint8), np.zeros((M, 0), np.uint8))
    b, sb = operand(N, K, mx.E2M1, 4) if K else (np.zeros((N, 0), np.uint8), np.zeros((N, 0), np.uint8))
    y, t = product(a, sa, a_fmt, b, sb) if K else (np.zeros((M, N)), np.zeros((M, N)))
    assert_gemm_close(run(a, sa, a_fmt, b, sb, torch.float32), y, t, False)


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(2600, 2570, 512), (2600, 2570, 640), (4100, 4200, 256), (512, 8704, 1152)])
def test_large_tiles_and_their_tail(M, N, K, a_fmt):
    """256 x 256 tiles, with and without a last round cut in quadrants, sampled against fp64."""
    a, sa = operand(M, K, a_fmt, 5, spread=2)
    b, sb = operand(N, K, mx.E2M1, 6, spread=2)
    y, t = product(a, sa, a_fmt, b, sb)
    assert_gemm_close(run(a, sa, a_fmt, b, sb, torch.float32), y, t, False)
    assert_gemm_close(run(a, sa, a_fmt, b, sb, torch.bfloat16, pad=32), y, t, True)


@pytest.mark.parametrize("a_fmt", FMTS)
def test_scales_at_odd_addresses(a_fmt):
    """Scale pointers on 4-byte boundaries only (the copies and tiles then load 4 bytes a lane)."""
    for M, N, K in ((3, 100, 512), (40, 200, 1024), (1000, 1000, 1024)):
        a, sa = operand(M, K, a_fmt, 7)
        b, sb = operand(N, K, mx.E2M1, 8)
        flat_a = torch.empty(sa.size + 4, dtype=torch.uint8, device="cuda")
        flat_b = torch.empty(sb.size + 4, dtype=torch.uint8, device="cuda")
        va, vb = flat_a[4:].view(sa.shape), flat_b[4:].view(sb.shape)
        va.copy_(dev(sa))
        vb.copy_(dev(sb))
        out = mx.mxfp4_scaled_gemm(dev_ld16(a), va, a_fmt, dev_ld16(b), vb)
        y, t = product(a, sa, a_fmt, b, sb)
        assert_gemm_close(host(out), y, t, False, what=str((M, N, K)))


@pytest.mark.parametrize("a_fmt", FMTS)
def test_graph_and_stream(a_fmt):
    a, sa = operand(9, 1024, a_fmt, 1)
    b, sb = operand(300, 1024, mx.E2M1, 2)
    a_d, sa_d, b_d, sb_d = dev(a), dev(sa), dev(b), dev(sb)
    out = torch.zeros((9, 304), device="cuda")[:, :300]
    want = mx.mxfp4_scaled_gemm(a_d, sa_d, a_fmt, b_d, sb_d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mx.mxfp4_scaled_gemm(a_d, sa_d, a_fmt, b_d, sb_d, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mxfp4_scaled_gemm(a_d, sa_d, a_fmt, b_d, sb_d, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.mxfp4_scaled_gemm(a_d, sa_d, a_fmt, b_d, sb_d))


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("K", [1536, 1664, 1792, 1920, 2048, 2176, 2304, 2432])
def test_long_k_in_few_tiles(K, a_fmt):
    """Every remainder of the K blocks, in 128 x 128 tiles that leave compute units idle."""
    M, N = 700, 1000
    a, sa = operand(M, K, a_fmt, 9, spread=2)
    b, sb = operand(N, K, mx.E2M1, 10, spread=2)
    y, t = product(a, sa, a_fmt, b, sb)
    assert_gemm_close(run(a, sa, a_fmt, b, sb, torch.float32), y, t, False)


def test_output_past_four_gib():
    """C of 4.6 GB: its last rows and columns against fp64."""
    M, N, K = 70000, 33000, 256
    a, sa = operand(64, K, mx.E4M3, 11, spread=1)
    b, sb = operand(N, K, mx.E2M1, 12, spread=1)
    a_d = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    sa_d = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
    a_d[-64:], sa_d[-64:] = dev(a), dev(sa)
    out = mx.mxfp4_scaled_gemm(a_d, sa_d, mx.E4M3, dev(b), dev(sb), out_dtype=torch.bfloat16)
    y, t = product(a, sa, mx.E4M3, b, sb)
    assert_gemm_close(host(out[-64:]), y, t, True)
    assert not out[:-64].any()


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(17, 8300, 128), (40, 7900, 256), (128, 3584, 384), (257, 1000, 640), (513, 900, 1920),
                                   (250, 1100, 4864)])
def test_one_round_of_wide_few_row_workgroups(M, N, K, a_fmt):
    """More 32 x 32 blocks of C than compute units, fewer 32 x 64 ones: with A in LDS and without, runs of K shorter
    than the waves are many, ragged edges."""
    a, sa = operand(M, K, a_fmt, 13, spread=2)
    b, sb = operand(N, K, mx.E2M1, 14, spread=2)
    y, t = product(a, sa, a_fmt, b, sb)
    first = run(a, sa, a_fmt, b, sb, torch.float32, pad=16)
    assert_gemm_close(first, y, t, False)
    assert_gemm_close(run(a, sa, a_fmt, b, sb, torch.bfloat16), y, t, True)
    assert np.array_equal(run(a, sa, a_fmt, b, sb, torch.float32, pad=16), first)


@pytest.mark.parametrize("K", [51200, 51328])
def test_scales_that_just_fill_lds_and_that_do_not(K):
    a, sa = operand(257, K, mx.E2M1, 15, spread=1)
    b, sb = operand(900, K, mx.E2M1, 16, spread=1)
    y, t = product(a, sa, mx.E2M1, b, sb)
    assert_gemm_close(run(a, sa, mx.E2M1, b, sb, torch.float32), y, t, False)


@pytest.mark.parametrize("a_fmt", FMTS)
def test_one_row_of_any_stride(a_fmt):
    """The last token of one long sequence: a single row 2^22 + 16 bytes and more from its neighbour, and an odd dense
    output row."""
    K, N = 512, 300
    a, sa = operand(1, K, a_fmt, 17)
    b, sb = operand(N, K, mx.E2M1, 18)
    width = a.shape[1]
    for stride in ((1 << 22) + 16, width + 1):
        far = torch.zeros(2 * stride, dtype=torch.uint8, device="cuda").as_strided((1, width), (stride, 1))
        far.copy_(dev(a))
        out = torch.full((1, N), 7.0, device="cuda")
        mx.mxfp4_scaled_gemm(far, dev(sa), a_fmt, dev_ld16(b), dev(sb), out=out)
        y, t = product(a, sa, a_fmt, b, sb)
        assert_gemm_close(host(out), y, t, False)
    row = torch.randn(65, device="cuda")[:64].as_strided((1, 64), (65, 1))
    q, s = mx.quantize_mxfp4(row)
    want = mx.quantize_mxfp4(row.clone())
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])
    h, hs, kept = mx.swiglu_mx(row)
    dx = mx.swiglu_mx_backward(kept, row[:, :32])
    want = mx.swiglu_mx(row.clone())
    assert torch.equal(h, want[0]) and torch.equal(hs, want[1])
    assert torch.equal(dx, mx.swiglu_mx_backward(want[2], row[:, :32].clone()))
