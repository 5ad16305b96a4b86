"""MX quantizers (rows in E2M1; transposed in E4M3, E5M2, E2M1, from tensors and from 8-bit
codes) and mx_dequantize, bit for bit against the plain implementation of mxref."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def values(rows, cols, seed, dtype):
    """Rows of very different sizes, with zero blocks, ties, subnormals and huge values among them."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (rows, cols)) * mxref.pow2(rng.integers(-20, 20, (rows, 1)))
    x = x.astype(np.float32)
    flat = x.reshape(-1)
    at = rng.permutation(flat.size)[: max(1, flat.size // 9)]
    flat[at] = (rng.integers(-16, 17, at.size) * 0.25 * mxref.pow2(rng.integers(-3, 4, at.size))).astype(np.float32)
    if rows > 2 and cols >= 64:
        x[1, :32] = 0.0
        x[1, 32:64] = -0.0
        x[2, :32] = np.float32(1e-40)
        x[2, 32:64] = np.float32(3e38)
    return x if dtype == "f32" else mxref.bf16(x)


def to_dev(x, dtype, pitch=None):
    t = torch.zeros((x.shape[0], pitch or x.shape[1]), dtype=DT[dtype])
    t[:, :x.shape[1]] = torch.from_numpy(x).to(DT[dtype])
    return t.cuda()[:, :x.shape[1]]


def same(q, s, ref_q, ref_s):
    assert np.array_equal(host(s), ref_s)
    assert np.array_equal(host(q), ref_q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
@pytest.mark.parametrize("rows,cols,pitch", [(1, 32, None), (1, 3584, None), (3, 96, 112), (5, 64, None), (67, 160, 176),
                                             (33, 2080, None), (300, 4096, 4112), (1100, 1056, None)])
def test_rows_e2m1(rows, cols, pitch, rule, dtype):
    x = values(rows, cols, rows + cols, dtype)
    q, s = mx.quantize_mxfp4(to_dev(x, dtype, pitch), rule)
    same(q, s, *mxref.quantize(x.astype(np.float64), mxref.E2M1, rule))


def test_rows_e2m1_every_bf16_pattern():
    """Each finite bf16 pattern below 8 (and its negative) as it is: 6 planted in its block fixes the
    exponent at 0, and the floor rule then leaves (6, 8) to saturate."""
    bits = np.arange(0, 0x4100, dtype=np.uint32)  # 0 .. just below 8
    v = (bits << 16).view(np.float32)
    v = np.concatenate((v, -v))
    n = -(-v.size // 31)
    x = np.zeros((n, 32), dtype=np.float32)
    x[:, 0] = 6.0
    x[:, 1:].reshape(-1)[:] = 0.0
    flat = np.zeros(n * 31, dtype=np.float32)
    flat[:v.size] = v
    x[:, 1:] = flat.reshape(n, 31)
    q, s = mx.quantize_mxfp4(to_dev(x, "f32"), mx.RULE_FLOOR)
    same(q, s, *mxref.quantize(x.astype(np.float64), mxref.E2M1, mxref.FLOOR))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2, mx.E2M1])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
@pytest.mark.parametrize("rows,cols,rows_out,pitch", [(1, 16, None, None), (32, 48, 32, 64), (77, 96, 96, None),
                                                      (128, 128, None, 144), (129, 272, 160, None), (300, 144, None, None),
                                                      (515, 400, 1024, None)])
def test_transposed(rows, cols, rows_out, pitch, rule, fmt, dtype):
    x = values(rows, cols, rows + cols, dtype)
    out = rows_out or (rows + 127) // 128 * 128
    q, s = mx.quantize_mx_t(to_dev(x, dtype, pitch), fmt, rule, rows_out)
    same(q, s, *mxref.quantize_t(x.astype(np.float64), fmt, rule, out))


@pytest.mark.parametrize("q_fmt", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2, mx.E2M1])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
@pytest.mark.parametrize("rows,cols,rows_out", [(1, 32, 32), (77, 96, 96), (130, 160, None), (515, 416, None)])
def test_transposed_from_codes(rows, cols, rows_out, rule, fmt, q_fmt):
    rng = np.random.default_rng(rows)
    q0 = rng.integers(0, 256, (rows, cols)).astype(np.uint8)
    q0 = np.where(np.isnan(mxref.code_values(q_fmt)[q0]), 0x81, q0).astype(np.uint8)
    s0 = rng.integers(100, 150, (rows, cols // 32)).astype(np.uint8)
    s0[0, 0] = 0  # 2^-127, a subnormal scale
    out = rows_out or (rows + 127) // 128 * 128
    q, s = mx.requantize_mx_t(dev(q0), dev(s0), q_fmt, fmt, rule, rows_out)
    same(q, s, *mxref.quantize_t(mxref.dequantize(q0, s0, q_fmt), fmt, rule, out))


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2, mx.E2M1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,pitch", [(1, 32, None), (1, 3584, None), (9, 96, 16), (130, 2080, None),
                                             (1100, 1056, 32)])
def test_dequantize(rows, cols, pitch, dtype, fmt):
    rng = np.random.default_rng(cols)
    q = rng.integers(0, 256, (rows, cols // 2 if fmt == mx.E2M1 else cols)).astype(np.uint8)
    if fmt != mx.E2M1:
        q = np.where(np.isnan(mxref.code_values(fmt)[q]), 0x80, q).astype(np.uint8)
    s = rng.integers(64, 190, (rows, cols // 32)).astype(np.uint8)
    s[-1, -1] = 255
    qd = dev(q, pitch=q.shape[1] + (pitch or 0))
    y = mx.dequantize_mx(qd, dev(s), fmt, dtype)
    assert y.dtype == dtype
    # every value fits both types: at most 4 significant bits, exponents far from the types' ends
    assert np.array_equal(host(y).astype(np.float64), mxref.dequantize(q, s, fmt), equal_nan=True)


def test_dequantize_ends_of_the_scale_range():
    q = np.tile(np.arange(16, dtype=np.uint8) * 17, (3, 1))
    s = np.array([[0], [1], [253]], dtype=np.uint8)
    y = host(mx.dequantize_mx(dev(q), dev(s), mx.E2M1, torch.float32)).astype(np.float64)
    ref = mxref.dequantize(q, s, mxref.E2M1)
    big = np.abs(ref) > np.finfo(np.float32).max
    assert np.array_equal(y[~big], ref[~big]) and np.isinf(y[big]).all()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
def test_non_finite_blocks(bad, dtype, rule):
    x = values(64, 128, 3, dtype)
    x[5, 40] = bad
    x[17, 127] = bad
    x64 = x.astype(np.float64)
    q, s = mx.quantize_mxfp4(to_dev(x, dtype), rule)
    same(q, s, *mxref.quantize(x64, mxref.E2M1, rule))
    y = host(mx.dequantize_mx(q, s, mx.E2M1))
    assert np.isnan(y[5, 32:64]).all() and np.isnan(y[17, 96:]).all() and np.isnan(y).sum() == 64
    for fmt in (mx.E4M3, mx.E5M2, mx.E2M1):
        q, s = mx.quantize_mx_t(to_dev(x, dtype), fmt, rule)
        same(q, s, *mxref.quantize_t(x64, fmt, rule, 128))
    # a kept block that is NaN stays NaN when it is turned
    q8, s8 = mxref.quantize(x64, mxref.E4M3, rule)
    q, s = mx.requantize_mx_t(dev(q8), dev(s8), mx.E4M3, mx.E5M2, rule)
    same(q, s, *mxref.quantize_t(mxref.dequantize(q8, s8, mxref.E4M3), mxref.E5M2, rule, 128))


def test_empty():
    e = torch.empty((0, 64), device="cuda")
    q, s = mx.quantize_mxfp4(e)
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert mx.dequantize_mx(q, s, mx.E2M1).shape == (0, 64)
    q, s = mx.quantize_mx_t(e, mx.E4M3)
    assert q.shape == (64, 0) and s.shape == (64, 0)
    q, s = mx.quantize_mx_t(e, mx.E4M3, rows_out=64)  # nothing but filling: zeros
    assert not host(q).any() and not host(s).any() and q.shape == (64, 64)
    q, s = mx.requantize_mx_t(torch.empty((0, 64), dtype=torch.uint8, device="cuda"),
                              torch.empty((0, 2), dtype=torch.uint8, device="cuda"), mx.E4M3, rows_out=32)
    assert not host(q).any() and not host(s).any()


def test_padding_untouched_and_streams():
    """Codes beyond a row's width stay as they were; work goes to the given stream."""
    x = values(40, 96, 8, "bf16")
    buf = torch.full((40, 64), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.empty((40, 3), dtype=torch.uint8, device="cuda")
    xd = to_dev(x, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert mx.mxfp4_quantize(xd.data_ptr(), mx.BF16, 40, 96, 96, mx.RULE_FLOOR, buf.data_ptr(), 64, s.data_ptr(),
                             side.cuda_stream) == 0
    torch.cuda.current_stream().wait_stream(side)
    ref_q, ref_s = mxref.quantize(x.astype(np.float64), mxref.E2M1, mxref.FLOOR)
    same(buf[:, :48], s, ref_q, ref_s)
    assert (host(buf)[:, 48:] == 0xA5).all()
    qt = torch.full((96, 96), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.empty((96, 2), dtype=torch.uint8, device="cuda")
    assert mx.mx_quantize_t(xd.data_ptr(), mx.BF16, 40, 96, 96, mx.E4M3, mx.RULE_CEIL, qt.data_ptr(), 96, 64,
                            st.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    same(qt[:, :64], st, *mxref.quantize_t(x.astype(np.float64), mxref.E4M3, mxref.CEIL, 64))
    assert (host(qt)[:, 64:] == 0xA5).all()


def test_past_four_gib():
    """Offsets beyond 32 bits: a bf16 matrix of 4.3 GiB, its last rows against the plain form."""
    rows, cols = 72000, 32768
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = values(64, cols, 4, "bf16")
    x[-64:] = torch.from_numpy(tail).to(torch.bfloat16).cuda()
    q, s = mx.quantize_mxfp4(x, mx.RULE_CEIL)
    same(q[-64:], s[-64:], *mxref.quantize(tail.astype(np.float64), mxref.E2M1, mxref.CEIL))
    assert not q[:-64].any() and not s[:-64].any()
    y = mx.dequantize_mx(q, s, mx.E2M1, torch.bfloat16)
    ref = mxref.dequantize(host(q[-64:]), host(s[-64:]), mxref.E2M1)
    ref[np.abs(ref) >= 2.0 ** 128] *= np.inf  # rounding 3e38 up leaves the range of fp32 and bf16
    assert np.array_equal(host(y[-64:]).astype(np.float64), ref)
    del q, s, y
    q, s = mx.quantize_mx_t(x, mx.E4M3)
    out = (rows + 127) // 128 * 128
    ref_q, ref_s = mxref.quantize_t(tail.astype(np.float64), mxref.E4M3, mxref.CEIL, 64 + out - rows)
    same(q[:, rows - 64:], s[:, (rows - 64) // 32:], ref_q, ref_s)


@pytest.mark.parametrize("source", ["bf16", "codes"])
@pytest.mark.parametrize("fmt,rows,cols", [(mx.E4M3, 2 ** 25 + 160, 32), (mx.E5M2, 2 ** 25 + 160, 32),
                                           (mx.E2M1, 2 ** 26 + 160, 32)])
def test_transposed_token_offsets_past_32_bits(fmt, rows, cols, source):
    """More tokens than a 32-bit token * tile-bytes product holds (2^25 for FP8 codes, 2^26 for E2M1): the first
    and the last tokens, which differ, against the plain form, and nothing but zeros between them."""
    first, last = values(128, cols, 21, "bf16"), values(160, cols, 22, "bf16")
    out = (rows + 127) // 128 * 128
    if source == "bf16":
        x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
        x[:128], x[-160:] = to_dev(first, "bf16"), to_dev(last, "bf16")
        q, s = mx.quantize_mx_t(x, fmt)
        f64, l64 = first.astype(np.float64), last.astype(np.float64)
    else:
        x = torch.zeros((rows, cols), dtype=torch.uint8, device="cuda")
        xs = torch.zeros((rows, cols // 32), dtype=torch.uint8, device="cuda")
        (fq, fs), (lq, ls) = (mxref.quantize(v.astype(np.float64), mxref.E4M3, mxref.CEIL) for v in (first, last))
        x[:128], x[-160:], xs[:128], xs[-160:] = dev(fq), dev(lq), dev(fs), dev(ls)
        q, s = mx.requantize_mx_t(x, xs, mx.E4M3, fmt)
        f64, l64 = mxref.dequantize(fq, fs, mxref.E4M3), mxref.dequantize(lq, ls, mxref.E4M3)
    tail = 160 + out - rows
    per = 2 if fmt == mx.E2M1 else 1  # tokens a byte
    same(q[:, :128 // per], s[:, :4], *mxref.quantize_t(f64, fmt, mxref.CEIL, 128))
    same(q[:, (out - tail) // per:], s[:, (out - tail) // 32:], *mxref.quantize_t(l64, fmt, mxref.CEIL, tail))
    assert not q[:, 128 // per:(out - tail) // per].any() and not s[:, 4:(out - tail) // 32].any()
