"""The MX operators in every form that their launch rules choose on 256 compute units: tiles
of 256 x 256 over a long K with and without a split tail, each few-row product with the left
operand in LDS and not, several units a lane, grids that are walked in rounds, each number of
waves and units of a row.  Large calls are compared bit for bit with calls on slices that are
small enough for the forms that the other tests check against the 64-bit implementation;
products with float64 products of the same codes, within 2^-12 * sum |a b| and for bf16 output
one rounding (2^-8) more."""
import functools

import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref
from test_gpu_mx_act import U, given, tensor
from test_gpu_mx_act import test_rmsnorm as check_rmsnorm
from test_gpu_mx_act import test_swiglu as check_swiglu

pytestmark = pytest.mark.gpu
FMTS = [mx.E2M1, mx.E4M3, mx.E5M2]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# magnitudes of a few binades around 1
CODES = {mx.E4M3: (0x28, 0x48), mx.E5M2: (0x34, 0x44)}


@functools.lru_cache(None)
def table(fmt):
    return torch.from_numpy(mxref.code_values(fmt)).cuda()


def codes(rows, K, fmt, gen):
    if fmt == mx.E2M1:
        return torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    sign = torch.randint(0, 2, (rows, K), dtype=torch.uint8, device="cuda", generator=gen) << 7
    return sign | torch.randint(*CODES[fmt], (rows, K), dtype=torch.uint8, device="cuda", generator=gen)


def operand(rows, K, fmt, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = codes(rows, K, fmt, gen)
    return q, torch.randint(121, 134, (rows, K // 32), dtype=torch.uint8, device="cuda", generator=gen)


def decoded(q, s, fmt):
    c = torch.stack((q & 15, q >> 4), -1).flatten(1) if fmt == mx.E2M1 else q
    v = table(fmt)[c.int()].view(c.shape[0], -1, 32)
    factor = (s.long() + (1023 - 127) << 52).view(torch.float64)  # put together from its bits: torch.ldexp takes a power
    return (v * factor[..., None]).flatten(1)


def moved(t, shift):
    """The same bytes `shift` bytes further from a 256-byte boundary."""
    flat = torch.empty(t.numel() + shift, dtype=torch.uint8, device="cuda")
    return flat[shift:].view(t.shape).copy_(t)


def pitched(t, ld):
    buf = torch.zeros((t.shape[0], ld), dtype=torch.uint8, device="cuda")
    return buf[:, :t.shape[1]].copy_(t)


def check_product(a, sa, a_fmt, b, sb, out, exact=None):
    if exact is None:
        exact = expected(a, sa, a_fmt, b, sb)
    y, t = exact
    tol = t * 2.0 ** -12
    if out.dtype == torch.bfloat16:
        tol = tol + (y.abs() + tol) * 2.0 ** -8
    off = (out.double() - y).abs()
    assert bool((off <= tol).all()), (float((off / tol).max()), (off > tol).nonzero()[:3].tolist())
    return exact


def expected(a, sa, a_fmt, b, sb):
    A, B = decoded(a, sa, a_fmt), decoded(b, sb, mx.E2M1)
    return A @ B.t().contiguous(), A.abs() @ B.abs().t().contiguous()


# --------------------------------------------------------------------------- products

@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("K", [2176, 2304, 2560, 2688, 2944])
@pytest.mark.parametrize("M,N", [(2900, 2950), (4300, 4050), (4500, 5001), (4290, 5300)])
def test_tiles_of_256_over_a_long_k(M, N, K, a_fmt):
    """144 tiles; 272, of which 16 are cut into quadrants; 360 and 357, whose last round is left as it is, with and
    without the bands of the XCDs.  K leaves every remainder of the loop's K blocks and, but for 2304 and 2560, half a
    block of E2M1 pairs; at 2560 scale rows are loaded 16 bytes a lane unless they start elsewhere."""
    a, sa = operand(M, K, a_fmt, M)
    b, sb = operand(N, K, mx.E2M1, N)
    exact = None
    for dtype in (torch.float32, torch.bfloat16):
        out = mx.mxfp4_scaled_gemm(a, sa, a_fmt, b, sb, out_dtype=dtype)
        exact = check_product(a, sa, a_fmt, b, sb, out, exact)
    if K == 2560:
        other = mx.mxfp4_scaled_gemm(a, moved(sa, 4), a_fmt, b, moved(sb, 8), out_dtype=torch.bfloat16)
        assert torch.equal(other, out)


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (16, 8200, 4608), (16, 8200, 18944),                      # 16 x 32, eight waves: much of A to each workgroup
    (1, 8200, 4096), (7, 9001, 2176), (12, 300, 2048),        # 16 x 16, two waves
    (5, 200, 2304), (16, 201, 18944), (1, 17, 40960),         # 16 x 16, four waves
    (40, 500, 4096), (48, 999, 18944),                        # the same for up to 48 rows
    (64, 1500, 512), (49, 700, 18944),                        # 16 x 32, eight waves
    (100, 1500, 1024), (200, 1000, 8192), (33, 2200, 18944),  # 32 x 32
    (129, 1900, 1280), (250, 1900, 7680)])                    # 32 x 64
def test_few_rows_with_a_in_lds_and_not(M, N, K, a_fmt):
    a, sa = operand(M, K, a_fmt, M)
    b, sb = operand(N, K, mx.E2M1, N)
    out = mx.mxfp4_scaled_gemm(a, sa, a_fmt, b, sb)
    check_product(a, sa, a_fmt, b, sb, out)
    assert torch.equal(mx.mxfp4_scaled_gemm(a, moved(sa, 4), a_fmt, b, moved(sb, 12)), out)


LD = 1 << 22  # the largest leading dimension, in bytes


@pytest.mark.parametrize("a_fmt", FMTS)
@pytest.mark.parametrize("M,N,K,lda,ldb", [(40, 64, 512, LD, LD), (17, 40, 18944, LD, LD), (256, 33024, 384, LD, None),
                                           (33024, 256, 384, None, LD)])
def test_largest_leading_dimensions(M, N, K, lda, ldb, a_fmt):
    """Rows 2^22 bytes apart for the few-row kernels and for tiles of 256 x 256 (516 tiles of 128 x 128)."""
    a, sa = operand(M, K, a_fmt, M)
    b, sb = operand(N, K, mx.E2M1, N)
    far_a, far_b = pitched(a, lda) if lda else a, pitched(b, ldb) if ldb else b
    out = mx.mxfp4_scaled_gemm(far_a, sa, a_fmt, far_b, sb)
    del far_a, far_b
    check_product(a, sa, a_fmt, b, sb, out)


# ---------------------------------------------------------- quantizer and its inverse

def numbers(rows, cols, dtype, seed=1):
    """Rows of very different sizes."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    return x.mul_(torch.ldexp(torch.ones(rows, 1, device="cuda"), torch.arange(rows, device="cuda")[:, None] % 37 - 18)).to(
        DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
@pytest.mark.parametrize("rows,cols", [(40000, 96), (70000, 32), (750000, 96)])
def test_rows_e2m1_several_units_a_lane(rows, cols, rule, dtype):
    """Rows that end within a lane's units; the last shape walks the grid and loads past the caches."""
    x = numbers(rows, cols, dtype)
    q, s = mx.quantize_mxfp4(x, rule)
    step = 20000  # at most 240000 units: one a lane
    for at in range(0, rows, step):
        want = mx.quantize_mxfp4(x[at:at + step], rule)
        assert torch.equal(q[at:at + step], want[0]) and torch.equal(s[at:at + step], want[1]), at
    head = x[-300:].double().cpu().numpy()
    ref_q, ref_s = mxref.quantize(head, mxref.E2M1, rule)
    assert np.array_equal(q[-300:].cpu().numpy(), ref_q) and np.array_equal(s[-300:].cpu().numpy(), ref_s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", [(40000, 96), (70000, 32), (750000, 96)])
def test_dequantize_several_units_a_lane(rows, cols, fmt, dtype):
    q, s = operand(rows, cols, fmt, 2)
    y = mx.dequantize_mx(q, s, fmt, DT[dtype])
    assert y.dtype == DT[dtype]
    for at in range(0, rows, 100000):  # exact in both types
        assert torch.equal(y[at:at + 100000].double(), decoded(q[at:at + 100000], s[at:at + 100000], fmt)), at


# ------------------------------------------------------------------------------ SwiGLU

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_swiglu_two_units_a_lane(dtype):
    """260 units a row: the third item of a row is 4 units long.  Against the formulas, forward and backward."""
    check_swiglu(2100, 2080, None, mx.RULE_CEIL, mx.E4M3, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
@pytest.mark.parametrize("rows,cols,step", [(2100, 2080, 500), (17000, 2080, 2000), (300000, 32, 60000)])
def test_swiglu_large(rows, cols, step, rule, fmt, dtype):
    """Ordinary accesses; accesses past the caches; grids walked in rounds, forward and backward."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, 2 * cols, generator=gen, device="cuda").mul_(3.0).to(DT[dtype])
    dh = torch.randn(rows, cols, generator=gen, device="cuda").mul_(1e-3).to(DT[dtype])
    h, hs, kept = mx.swiglu_mx(x, fmt, rule)
    only, only_s, _ = mx.swiglu_mx(x, fmt, rule, keep=False)
    assert torch.equal(only, h) and torch.equal(only_s, hs)
    dx = mx.swiglu_mx_backward(kept, dh)
    for at in range(0, rows, step):
        part = slice(at, at + step)
        want = mx.swiglu_mx(x[part], fmt, rule)
        assert torch.equal(h[part], want[0]) and torch.equal(hs[part], want[1]), at
        assert torch.equal(kept.codes[part], want[2].codes) and torch.equal(kept.scales[part], want[2].scales), at
        assert torch.equal(dx[part], mx.swiglu_mx_backward(want[2], dh[part])), at


# ----------------------------------------------------------------------------- RMSNorm

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [992, 2016, 2560, 2592, 6144, 8160, 12288, 14304, 16352, 24576])
def test_rmsnorm_units_of_a_lane(cols, dtype):
    """2, 4, 5 and 6 units a lane with one wave a row; 3, 4, 6, 7 and 8 with four; 3 with sixteen: the formulas."""
    check_rmsnorm(37, cols, None, mx.RULE_CEIL, mx.E4M3, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("rows,cols", [(5000, 544), (5000, 2016), (5000, 2560), (9001, 2592), (5000, 3584), (5000, 4096),
                                       (1100, 6144), (1100, 8160), (1100, 12288), (1100, 14304), (1100, 20480),
                                       (1030, 32768)])
def test_rmsnorm_rows_in_rounds(rows, cols, fmt, dtype):
    """More rows than the grids hold at once, forward and backward, so that each wave (or workgroup) walks several with
    the next one on its way.  dw's bound counts an fp32 sum of `rows` terms, as for few rows."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, cols, generator=gen, device="cuda").mul_(
        torch.linspace(-2, 3, cols, device="cuda").exp()).to(DT[dtype])
    dy = torch.randn(rows, cols, generator=gen, device="cuda").mul_(1e-3).to(DT[dtype])
    w = torch.rand(cols, generator=gen, device="cuda").add_(0.5)
    y, ys, kept = mx.rmsnorm_mx(x, w, 1e-5, fmt)
    only, only_s, _ = mx.rmsnorm_mx(x, w, 1e-5, fmt, keep=False)
    assert torch.equal(only, y) and torch.equal(only_s, ys)
    dx, dw = mx.rmsnorm_mx_backward(kept, w, dy)
    step = 250
    total, size = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for at in range(0, rows, step):
        part = slice(at, at + step)
        want = mx.rmsnorm_mx(x[part], w, 1e-5, fmt)
        assert torch.equal(y[part], want[0]) and torch.equal(ys[part], want[1]), at
        assert torch.equal(kept.codes[part], want[2].codes) and torch.equal(kept.scales[part], want[2].scales), at
        assert torch.equal(kept.rstd[part], want[2].rstd), at
        assert torch.equal(dx[part], mx.rmsnorm_mx_backward(want[2], w, dy[part])[0]), at
        term = dy[part].double() * decoded(kept.codes[part], kept.scales[part], fmt) * kept.rstd[part].double()[:, None]
        total += term.sum(0)
        size += term.abs().sum(0)
    off, tol = (dw.double() - total).abs(), size * (8 + rows ** 0.5) * U
    assert bool((off <= tol).all()), float((off / tol).max())
    again = mx.rmsnorm_mx_backward(kept, w, dy)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_rmsnorm_strided_rows_in_rounds():
    """Padded rows of x and dy at more rows than the grids hold."""
    x, dy = given((4500, 1536), 1.0, 1, "bf16"), given((4500, 1536), 1e-3, 2, "bf16")
    w = torch.rand(1536, device="cuda")
    a, b = mx.rmsnorm_mx(tensor(x, "bf16", 48), w, 1e-6), mx.rmsnorm_mx(tensor(x, "bf16"), w, 1e-6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2].rstd, b[2].rstd)
    da = mx.rmsnorm_mx_backward(a[2], w, tensor(dy, "bf16", 16))
    db = mx.rmsnorm_mx_backward(b[2], w, tensor(dy, "bf16"))
    assert torch.equal(da[0], db[0]) and torch.equal(da[1], db[1])
