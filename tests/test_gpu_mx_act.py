"""SwiGLU and RMSNorm with inputs kept in 8 bits, against the formulas in 64 bits.

Tolerances.  u = 2^-24 is fp32's half step.  What is kept is a plain quantization of the
input: bit for bit.  h and y are computed in fp32 with a relative error d of at most
(16 + 1.5 |g|) u for SwiGLU (exp2 argument |g| log2 e u, exp2 and rcp 1 ulp = 2 u each, five
products) and (12 + sqrt(cols)) u for RMSNorm (the sum of squares, the root, three products),
then cast: off by half a step of the format (or half its smallest value times the scale) more.
Gradients: the same d per product plus the rounding to their own type; terms that cancel
count with their absolute sizes."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OWN = {"f32": U, "bf16": 2.0 ** -8}
SIZES = [(1, 32, None), (1, 3584, None), (7, 96, 16), (33, 1536, None), (130, 544, 48), (300, 4096, None), (65, 8960, None)]


def tensor(x, dtype, pad=None):
    t = torch.zeros((x.shape[0], x.shape[1] + (pad or 0)), dtype=DT[dtype])
    t[:, :x.shape[1]] = torch.from_numpy(x).to(DT[dtype])
    return t.cuda()[:, :x.shape[1]]


def given(shape, scale, seed, dtype):
    x = (np.random.default_rng(seed).normal(0, 1, shape) * scale).astype(np.float32)
    return x if dtype == "f32" else mxref.bf16(x)


def check_codes(q, s, exact, d, fmt, rule):
    """Codes of values that lie within a relative d of `exact`."""
    q, s = host(q), host(s)
    amax = np.abs(exact).reshape(exact.shape[0], -1, 32).max(-1)
    low = mxref.exponent(amax * (1 - d.reshape(amax.shape + (32,)).max(-1)), fmt, rule) + 127
    high = mxref.exponent(amax * (1 + d.reshape(amax.shape + (32,)).max(-1)), fmt, rule) + 127
    assert ((s >= low) & (s <= high)).all()
    scale = np.repeat(mxref.pow2(s.astype(np.int64) - 127), 32, axis=1)
    top = mxref.fmax(fmt) * scale
    got = mxref.dequantize(q, s, fmt)
    want = np.clip(exact, -top, top)  # the floor rule saturates
    tol = np.maximum(mxref.half_step(fmt) * np.abs(want), mxref.smallest(fmt) / 2 * scale)
    tol = tol * (1 + 2 * d) + d * np.abs(want)
    off = np.abs(got - want) / np.maximum(tol, 1e-300)
    assert (off <= 1).all(), (off.max(), np.argwhere(off > 1)[:3])


def close(y, exact, tol):
    off = np.abs(host(y).astype(np.float64) - exact)
    assert (off <= tol).all(), ((off / np.maximum(tol, 1e-300)).max(), np.argwhere(off > tol)[:3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
@pytest.mark.parametrize("rows,cols,pad", SIZES)
def test_swiglu(rows, cols, pad, rule, fmt, dtype):
    x = given((rows, 2 * cols), 3.0, rows + cols, dtype)
    x[0, :4] = [-60.0, 60.0, 0.0, -0.0]
    x64 = x.astype(np.float64)
    xd = tensor(x, dtype, pad)
    h, hs, kept = mx.swiglu_mx(xd, fmt, rule)
    ref_q, ref_s = mxref.quantize(x64, fmt, rule)
    assert np.array_equal(host(kept.scales), ref_s) and np.array_equal(host(kept.codes), ref_q)
    check_codes(h, hs, mxref.swiglu(x64), (16 + 1.5 * np.abs(x64[:, :cols])) * U, fmt, rule)
    only, only_s, none = mx.swiglu_mx(xd, fmt, rule, keep=False)
    assert none is None and torch.equal(only, h) and torch.equal(only_s, hs)
    # backward, at the kept values
    dh = given((rows, cols), 1e-3, 5, dtype)
    dx = mx.swiglu_mx_backward(kept, tensor(dh, dtype, pad))
    assert dx.dtype == DT[dtype]
    xk, d64 = mxref.dequantize(ref_q, ref_s, fmt), dh.astype(np.float64)
    exact = mxref.swiglu_grad(xk, d64)
    g, u = xk[:, :cols], xk[:, cols:]
    sg = mxref.sigmoid(g)
    rel = (20 + 1.5 * np.abs(g)) * U
    part = np.abs(d64 * sg) * np.concatenate((np.abs(u) * (1 + np.abs(g)), np.abs(g)), axis=1).reshape(rows, 2, cols).swapaxes(0, 1)
    tol = np.concatenate((part[0] * rel, part[1] * rel), axis=1)
    close(dx, exact, tol + OWN[dtype] * (np.abs(exact) + tol) + 1e-44)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("rule", [mx.RULE_CEIL, mx.RULE_FLOOR])
@pytest.mark.parametrize("rows,cols,pad", SIZES + [(5, 16384, None), (3, 20480, 16), (2, 32768, None), (0, 64, None)])
def test_rmsnorm(rows, cols, pad, rule, fmt, dtype):
    x = given((rows, cols), np.exp(np.linspace(-2, 3, cols)), rows + cols, dtype)
    if rows > 2:
        x[1] = 0.0
    x64, eps = x.astype(np.float64), 1e-5
    w = (1 + 0.2 * np.random.default_rng(9).normal(0, 1, cols)).astype(np.float32)
    w64 = w.astype(np.float64)
    xd, wd = tensor(x, dtype, pad), torch.from_numpy(w).cuda()
    y, ys, kept = mx.rmsnorm_mx(xd, wd, eps, fmt, rule)
    dy = given((rows, cols), 1e-3, 6, dtype)
    dx, dw = mx.rmsnorm_mx_backward(kept, wd, tensor(dy, dtype, pad))
    again = mx.rmsnorm_mx_backward(kept, wd, tensor(dy, dtype, pad))
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    if rows == 0:
        assert not host(dw).any() and dx.shape == (0, cols)
        return
    ref_q, ref_s = mxref.quantize(x64, fmt, rule)
    assert np.array_equal(host(kept.scales), ref_s) and np.array_equal(host(kept.codes), ref_q)
    r = mxref.rstd(x64, eps)
    d = (12 + np.sqrt(cols)) * U
    close(kept.rstd, r, d * r)
    check_codes(y, ys, x64 * r[:, None] * w64, np.full(x.shape, d), fmt, rule)
    only, only_s, none = mx.rmsnorm_mx(xd, wd, eps, fmt, rule, keep=False)
    assert none is None and torch.equal(only, y) and torch.equal(only_s, ys)
    rk, d64 = host(kept.rstd).astype(np.float64), dy.astype(np.float64)
    xk = mxref.dequantize(ref_q, ref_s, fmt)
    ex, ew = mxref.rmsnorm_grad(xk, rk, w64, d64)
    xh, c = np.abs(xk * rk[:, None]), np.abs(d64 * w64)
    size = (c + xh * (c * xh).mean(1, keepdims=True)) * rk[:, None]
    tol = size * d
    close(dx, ex, tol + OWN[dtype] * (np.abs(ex) + tol) + 1e-44)
    close(dw, ew, (np.abs(d64) * xh).sum(0) * (8 + np.sqrt(rows)) * U + 1e-44)


def test_non_finite():
    """A bad input spoils its own block of what SwiGLU gives and keeps, and its row of RMSNorm."""
    x = given((4, 128), 1.0, 1, "f32")
    x[1, 3], x[2, 70] = np.inf, np.nan
    h, hs, kept = mx.swiglu_mx(tensor(x, "f32"))
    y = host(mx.dequantize_mx(h, hs, mx.E4M3))
    bad = np.zeros((4, 64), bool)
    bad[1, :32] = bad[2, :32] = True
    assert np.array_equal(np.isnan(y), bad)
    dx = host(mx.swiglu_mx_backward(kept, torch.ones((4, 64), device="cuda")))
    bad_u = bad.copy()
    bad_u[2] = False  # du = dh g s has no u in it
    assert np.array_equal(np.isnan(dx), np.concatenate((bad, bad_u), axis=1))
    w = torch.ones(128, device="cuda")
    y, ys, kept = mx.rmsnorm_mx(tensor(x, "f32"), w, 1e-6)
    v = host(mx.dequantize_mx(y, ys, mx.E4M3))
    assert np.isfinite(v[[0, 3]]).all() and np.isnan(v[2]).all() and np.isnan(v[1, :32]).all()
    dx, dw = mx.rmsnorm_mx_backward(kept, w, torch.ones((4, 128), device="cuda"))
    dx = host(dx)
    assert np.isfinite(dx[[0, 3]]).all() and np.isnan(dx[[1, 2]]).all()


def test_graph_replays():
    """Forward and backward captured once, replayed on changed inputs with eager work between."""
    x, dh = tensor(given((64, 512), 2.0, 1, "bf16"), "bf16"), tensor(given((64, 256), 1e-3, 2, "bf16"), "bf16")
    w = torch.rand(512, device="cuda")
    dy = tensor(given((64, 512), 1e-3, 3, "bf16"), "bf16")

    def step():
        h, hs, kept = mx.swiglu_mx(x)
        y, ys, nk = mx.rmsnorm_mx(x, w, 1e-6)
        return (h, hs, mx.swiglu_mx_backward(kept, dh), y, ys) + mx.rmsnorm_mx_backward(nk, w, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(tensor(given((64, 512), 2.0, 10 + k, "bf16"), "bf16"))
        dy.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_other_stream():
    x, w = tensor(given((256, 1024), 1.0, 1, "f32"), "f32"), torch.rand(1024, device="cuda")
    dy = tensor(given((256, 1024), 1.0, 2, "f32"), "f32")
    want = mx.rmsnorm_mx(x, w, 1e-6)
    want_b = mx.rmsnorm_mx_backward(want[2], w, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, ys, kept = mx.rmsnorm_mx(x, w, 1e-6, stream=side)
    dx, dw = mx.rmsnorm_mx_backward(kept, w, dy, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0]) and torch.equal(ys, want[1])
    assert torch.equal(dx, want_b[0]) and torch.equal(dw, want_b[1])


def test_past_four_gib():
    """Offsets beyond 32 bits in every tensor: 4.6 GB of x, of dx and of what is kept, and the last
    rows against a call on them alone."""
    rows, cols = 70400, 16384
    x = torch.zeros((rows, 2 * cols), dtype=torch.bfloat16, device="cuda")
    dh = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail_x, tail_d = tensor(given((16, 2 * cols), 2.0, 1, "bf16"), "bf16"), tensor(given((16, cols), 1.0, 2, "bf16"), "bf16")
    x[-16:], dh[-16:] = tail_x, tail_d
    h, hs, kept = mx.swiglu_mx(x)
    want = mx.swiglu_mx(tail_x)
    assert torch.equal(h[-16:], want[0]) and torch.equal(hs[-16:], want[1])
    assert torch.equal(kept.codes[-16:], want[2].codes) and not kept.codes[:-16].any()
    dx = mx.swiglu_mx_backward(kept, dh)
    assert torch.equal(dx[-16:], mx.swiglu_mx_backward(want[2], tail_d)) and not dx[:-16].any()
    del h, hs, kept, dx, dh
    w = torch.rand(2 * cols, device="cuda")
    y, ys, kept = mx.rmsnorm_mx(x, w, 1e-6)
    want = mx.rmsnorm_mx(tail_x, w, 1e-6)
    assert torch.equal(y[-16:], want[0]) and torch.equal(kept.rstd[-16:], want[2].rstd)
    dx, dw = mx.rmsnorm_mx_backward(kept, w, x)
    want_dx, want_dw = mx.rmsnorm_mx_backward(want[2], w, tail_x)
    assert torch.equal(dx[-16:], want_dx)
    assert torch.allclose(dw, want_dw, rtol=1e-5, atol=1e-4)  # another order of the same 16 rows' sum


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [544, 8960, 20480])
def test_rmsnorm_of_rows_whose_squares_leave_fp32(cols, dtype):
    """Rows scaled by powers of two whose squares overflow or vanish in fp32, with eps = 0, at every number of waves
    a row; a zero row has no root (0 / 0), rows with an infinity or a NaN are as ever."""
    powers = np.array([0, 40, 66, 100, 120, -40, -52, -66, -100, -110, 0, 90, -90])
    rows = len(powers)
    x = given((rows, cols), mxref.pow2(powers)[:, None], 31, dtype)
    x64 = x.astype(np.float64)
    w = (1 + 0.2 * np.random.default_rng(9).normal(0, 1, cols)).astype(np.float32)
    w64, wd = w.astype(np.float64), torch.from_numpy(w).cuda()
    y, ys, kept = mx.rmsnorm_mx(tensor(x, dtype), wd, 0.0)
    r = mxref.rstd(x64, 0.0)
    d = (12 + np.sqrt(cols)) * U
    close(kept.rstd, r, d * r)
    check_codes(y, ys, x64 * r[:, None] * w64, np.full(x.shape, d), mx.E4M3, mx.RULE_CEIL)
    ref_q, ref_s = mxref.quantize(x64, mx.E4M3, mx.RULE_CEIL)
    assert np.array_equal(host(kept.scales), ref_s) and np.array_equal(host(kept.codes), ref_q)
    dy = given((rows, cols), 1e-3, 6, dtype)
    dx, dw = mx.rmsnorm_mx_backward(kept, wd, tensor(dy, dtype))
    rk, d64, xk = host(kept.rstd).astype(np.float64), dy.astype(np.float64), mxref.dequantize(ref_q, ref_s, mx.E4M3)
    ex, ew = mxref.rmsnorm_grad(xk, rk, w64, d64)
    xh, c = np.abs(xk * rk[:, None]), np.abs(d64 * w64)
    tol = (c + xh * (c * xh).mean(1, keepdims=True)) * rk[:, None] * d
    smallest = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133}[dtype]  # the type's own step below its normal range
    close(dx, ex, tol + OWN[dtype] * (np.abs(ex) + tol) + smallest)
    close(dw, ew, (np.abs(d64) * xh).sum(0) * (8 + np.sqrt(rows)) * U + 1e-44)
    # rows without a finite root
    x[0], x[1, 5], x[2, 40] = 0.0, np.inf, np.nan
    y, ys, kept = mx.rmsnorm_mx(tensor(x, dtype), wd, 0.0)
    v, rk = host(mx.dequantize_mx(y, ys, mx.E4M3)), host(kept.rstd)
    assert np.isnan(v[0]).all() and np.isnan(v[2]).all() and np.isnan(v[1, :32]).all() and not v[1, 32:].any()
    assert np.isinf(rk[0]) and rk[1] == 0 and np.isnan(rk[2]) and np.isfinite(v[3:]).all()
    close(kept.rstd[3:], r[3:], d * r[3:])
