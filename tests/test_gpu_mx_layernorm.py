"""LayerNorm on MX codes against the formulas in 64 bits.

Tolerances, u = 2^-24 (fp32's half step).  x - m0 is off by u of itself, the mean of x - m0 by
at most T u of the mean of |x - m0| (T additions a sum: 8 a unit, up to 4 units a lane, 6 over
the lanes, 15 over the waves), r by T u / 2 for its sum and 3 u for the rest.  So xh is off by
(T / 2 + 6) u |xh| + T u (mean |x - mu| r <= 1), y by |w| times that and 2 u (|xh w| + |b|);
then the cast's half step.  Gradients: T + 8 u of the absolute sizes that are added, and half a
step of their own type; dw and db rows + 16 additions."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref
from gpu_helpers import host

pytestmark = pytest.mark.gpu
U, T = 2.0 ** -24, 53
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OWN = {"f32": U, "bf16": 2.0 ** -8}
SIZES = [(1, 32, None), (1, 3584, None), (7, 96, 16), (33, 1536, None), (130, 544, 48), (300, 4096, None),
         (65, 8960, None), (2100, 64, None), (4, 8192, None), (5, 8224, None), (3, 16384, None), (6, 16416, 16),
         (2, 32768, None), (0, 64, None)]


def tensor(x, dtype, pad=None):
    t = torch.zeros((x.shape[0], x.shape[1] + (pad or 0)), dtype=DT[dtype])
    t[:, :x.shape[1]] = torch.from_numpy(x).to(DT[dtype])
    return t.cuda()[:, :x.shape[1]]


def given(shape, scale, seed, dtype, mean=0.0):
    x = (np.random.default_rng(seed).normal(0, 1, shape) * scale + mean).astype(np.float32)
    return x if dtype == "f32" else mxref.bf16(x)


def vectors(cols, seed=9):
    rng = np.random.default_rng(seed)
    return ((1 + 0.2 * rng.normal(0, 1, cols)).astype(np.float32), (0.3 * rng.normal(0, 1, cols)).astype(np.float32))


def dev32(v):
    return None if v is None else torch.from_numpy(v).cuda()


def normalised(x, eps):
    d = x - x.mean(1, keepdims=True)
    d = d - d.mean(1, keepdims=True)
    r = 1 / np.sqrt((d * d).mean(1) + eps)
    return d * r[:, None], r


def xh_error(xh):
    return ((T / 2 + 6) * np.abs(xh) + T) * U


def check_codes(q, s, exact, e, fmt, rule):
    """Codes of values that lie within e of `exact`."""
    q, s = host(q), host(s)
    block = (exact.shape[0], -1, 32)
    low = mxref.exponent(np.maximum(np.abs(exact) - e, 0).reshape(block).max(-1), fmt, rule) + 127
    high = mxref.exponent((np.abs(exact) + e).reshape(block).max(-1), fmt, rule) + 127
    assert ((s >= low) & (s <= high)).all()
    scale = np.repeat(mxref.pow2(s.astype(np.int64) - 127), 32, axis=1)
    top = mxref.fmax(fmt) * scale
    want = np.clip(exact, -top, top)  # the floor rule saturates
    tol = np.maximum(mxref.half_step(fmt) * (np.abs(want) + e), mxref.smallest(fmt) / 2 * scale) + e
    off = np.abs(mxref.dequantize(q, s, fmt) - want) / tol
    assert (off <= 1).all(), (off.max(), np.argwhere(off > 1)[:3])


def close(y, exact, tol):
    off = np.abs(host(y).astype(np.float64) - exact)
    assert (off <= tol).all(), ((off / np.maximum(tol, 1e-300)).max(), np.argwhere(off > tol)[:3])


def gradients(xh, r, w, dy):
    c = dy * w
    dx = (c - c.mean(1, keepdims=True) - xh * (c * xh).mean(1, keepdims=True)) * r[:, None]
    return dx, (dy * xh).sum(0), dy.sum(0)


def check_backward(kept, w, dy, dtype, got):
    """The gradients at what was kept, as it came out."""
    xh = mxref.dequantize(host(kept.codes), host(kept.scales), kept.fmt)
    r, d64 = host(kept.rstd).astype(np.float64), dy.astype(np.float64)
    w64 = np.ones(xh.shape[1]) if w is None else w.astype(np.float64)
    ex, ew, eb = gradients(xh, r, w64, d64)
    c, a = np.abs(d64 * w64), np.abs(xh)
    tol = (c + c.mean(1, keepdims=True) + a * (c * a).mean(1, keepdims=True)) * r[:, None] * (T + 8) * U
    close(got[0], ex, tol + OWN[dtype] * (np.abs(ex) + tol) + 1e-44)
    if w is None:
        assert got[1] is None and got[2] is None
        return
    n = (16 + len(dy)) * U
    close(got[1], ew, (np.abs(d64) * a).sum(0) * n + 1e-44)
    close(got[2], eb, np.abs(d64).sum(0) * n + 1e-44)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt,rule", [(mx.E4M3, mx.RULE_CEIL), (mx.E5M2, mx.RULE_FLOOR), (mx.E4M3, mx.RULE_FLOOR),
                                      (mx.E5M2, mx.RULE_CEIL)])
@pytest.mark.parametrize("rows,cols,pad", SIZES)
def test_layernorm(rows, cols, pad, fmt, rule, dtype):
    eps = 1e-5
    x = given((rows, cols), np.exp(np.linspace(-2, 3, cols)), rows + cols, dtype, 0.7)
    if rows > 2:
        x[1] = 0.0
        x[2] = 3.0
    w, b = vectors(cols)
    xd, wd, bd = tensor(x, dtype, pad), dev32(w), dev32(b)
    y, ys, kept = mx.layernorm_mx(xd, wd, bd, eps, fmt, rule)
    assert y.shape == x.shape and kept.fmt == fmt
    dy = given((rows, cols), 1e-3, 6, dtype)
    got = mx.layernorm_mx_backward(kept, wd, tensor(dy, dtype, pad))
    again = mx.layernorm_mx_backward(kept, wd, tensor(dy, dtype, pad))
    assert got[0].dtype == DT[dtype] and all(torch.equal(p, q) for p, q in zip(got, again))
    if rows == 0:
        assert got[0].shape == (0, cols) and not host(got[1]).any() and not host(got[2]).any()
        return
    only, only_s, none = mx.layernorm_mx(xd, wd, bd, eps, fmt, rule, keep=False)
    assert none is None and torch.equal(only, y) and torch.equal(only_s, ys)
    xh, r = normalised(x.astype(np.float64), eps)
    e, w64, b64 = xh_error(xh), w.astype(np.float64), b.astype(np.float64)
    close(kept.rstd, r, (T / 2 + 4) * U * r)
    check_codes(kept.codes, kept.scales, xh, e, fmt, rule)
    check_codes(y, ys, xh * w64 + b64, e * np.abs(w64) + 2 * U * (np.abs(xh * w64) + np.abs(b64)), fmt, rule)
    check_backward(kept, w, dy, dtype, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [96, 3584, 12288, 20480])
def test_without_bias_and_without_weight(cols, dtype):
    rows, eps = 9, 1e-6
    x = given((rows, cols), 2.0, 3, dtype, -1.0)
    w, _ = vectors(cols)
    xh, _ = normalised(x.astype(np.float64), eps)
    dy = given((rows, cols), 1e-2, 4, dtype)
    for weight in (w, None):
        y, ys, kept = mx.layernorm_mx(tensor(x, dtype), dev32(weight), None, eps)
        w64 = np.ones(cols) if weight is None else weight.astype(np.float64)
        check_codes(y, ys, xh * w64, xh_error(xh) * w64 + 2 * U * np.abs(xh * w64), mx.E4M3, mx.RULE_CEIL)
        if weight is None:
            assert torch.equal(y, kept.codes) and torch.equal(ys, kept.scales)
        got = mx.layernorm_mx_backward(kept, dev32(weight), tensor(dy, dtype))
        check_backward(kept, weight, dy, dtype, got)


@pytest.mark.parametrize("cols", [64, 3584, 9216])
@pytest.mark.parametrize("offset", [300.0, -5e4, 2.0 ** 21])
def test_rows_far_from_zero(offset, cols):
    """Values whose mean is many times their spread: the result is that of the values as they are."""
    x = (np.random.default_rng(5).normal(0, 1, (6, cols)) + offset).astype(np.float32)
    xh, r = normalised(x.astype(np.float64), 0.0)
    y, ys, kept = mx.layernorm_mx(tensor(x, "f32"), None, None, 0.0)
    close(kept.rstd, r, (T / 2 + 4) * U * r)
    check_codes(y, ys, xh, xh_error(xh), mx.E4M3, mx.RULE_CEIL)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [544, 8960, 20480])
def test_rows_whose_squares_leave_fp32(cols, dtype):
    """Rows scaled by powers of two whose squares or sums overflow or vanish in fp32, with eps = 0; rows of
    equal values have no root (0 / 0), rows with an infinity or a NaN no mean."""
    powers = np.array([0, 40, 66, 100, 120, -40, -52, -66, -100, -110, 0, 90, -90])
    rows = len(powers)
    x = given((rows, cols), mxref.pow2(powers)[:, None], 31, dtype)
    x[3] += mxref.bf16(np.float32(2.0 ** 101)) if dtype == "f32" else 0
    w, b = vectors(cols)
    xh, r = normalised(x.astype(np.float64), 0.0)
    y, ys, kept = mx.layernorm_mx(tensor(x, dtype), dev32(w), dev32(b), 0.0)
    w64, b64 = w.astype(np.float64), b.astype(np.float64)
    close(kept.rstd, r, (T / 2 + 4) * U * r)
    check_codes(kept.codes, kept.scales, xh, xh_error(xh), mx.E4M3, mx.RULE_CEIL)
    check_codes(y, ys, xh * w64 + b64, xh_error(xh) * np.abs(w64) + 2 * U * (np.abs(xh * w64) + np.abs(b64)), mx.E4M3,
                mx.RULE_CEIL)
    x[0], x[1, 5], x[2, 40] = 3.0, np.inf, np.nan
    y, ys, kept = mx.layernorm_mx(tensor(x, dtype), dev32(w), dev32(b), 0.0)
    v, rk = host(mx.dequantize_mx(y, ys, mx.E4M3)), host(kept.rstd)
    assert np.isnan(v[:3]).all() and np.isinf(rk[0]) and np.isnan(rk[1:3]).all() and np.isfinite(v[3:]).all()
    # their gradients are NaN, the others' are not touched
    dx, _, _ = mx.layernorm_mx_backward(kept, dev32(w), tensor(given(x.shape, 1.0, 6, dtype) * 2.0 ** -20, dtype))
    dx = host(dx)
    assert np.isnan(dx[:3]).all() and np.isfinite(dx[3:7]).all()


def test_an_infinite_gradient_spoils_its_row_alone():
    x, dy = given((5, 128), 1.0, 1, "f32"), given((5, 128), 1.0, 2, "f32")
    w = torch.ones(128, device="cuda")
    kept = mx.layernorm_mx(tensor(x, "f32"), w, w, 1e-5)[2]
    dy[1, 3], dy[3, 70] = np.inf, np.nan
    dx, dw, db = (host(t) for t in mx.layernorm_mx_backward(kept, w, tensor(dy, "f32")))
    assert np.isfinite(dx[[0, 2, 4]]).all() and not np.isfinite(dx[[1, 3]]).any()
    bad = np.zeros(128, bool)
    bad[[3, 70]] = True
    assert np.array_equal(~np.isfinite(dw), bad) and np.array_equal(~np.isfinite(db), bad)


def test_gradients_against_differences():
    """The whole operator's derivative: the loss's change along a direction, in 64 bits, against the gradient that
    the kernel gives at its 8-bit xh.  xh is off by half a step of E4M3, 2^-4 of itself, so each term of the sums
    is by 2^-4 of its size at most, twice in xh mean(c xh)."""
    rows, cols, eps, h = 6, 256, 1e-5, 1e-5
    x, dy = given((rows, cols), 2.0, 1, "f32", 1.0).astype(np.float64), given((rows, cols), 1.0, 2, "f32").astype(np.float64)
    w, b = vectors(cols)
    w64, b64 = w.astype(np.float64), b.astype(np.float64)
    kept = mx.layernorm_mx(tensor(x.astype(np.float32), "f32"), dev32(w), dev32(b), eps)[2]
    dx, dw, db = (host(t).astype(np.float64) for t in mx.layernorm_mx_backward(kept, dev32(w), tensor(dy.astype(np.float32), "f32")))

    def loss(x, w, b):
        return ((normalised(x, eps)[0] * w + b) * dy).sum(-1)
    v = np.random.default_rng(3).normal(0, 1, (rows, cols))
    num = (loss(x + h * v, w64, b64) - loss(x - h * v, w64, b64)) / (2 * h)
    xh, r = normalised(x, eps)
    c = np.abs(dy * w64)
    off = np.abs(xh) * (c * np.abs(xh)).mean(1, keepdims=True) * r[:, None]
    assert (np.abs((dx * v).sum(1) - num) <= (off * np.abs(v)).sum(1) * 2 * 2.0 ** -4 + 1e-6).all()
    for k in range(0, cols, 37):
        d = np.zeros(cols)
        d[k] = h
        num_w = (loss(x, w64 + d, b64) - loss(x, w64 - d, b64)).sum() / (2 * h)
        num_b = (loss(x, w64, b64 + d) - loss(x, w64, b64 - d)).sum() / (2 * h)
        assert abs(dw[k] - num_w) <= 2.0 ** -4 * np.abs(dy[:, k] * xh[:, k]).sum() + 1e-5
        assert abs(db[k] - num_b) <= 1e-5


def test_graph_replays_and_other_streams():
    x, dy = tensor(given((70, 512), 2.0, 1, "bf16"), "bf16"), tensor(given((70, 512), 1e-3, 3, "bf16"), "bf16")
    w, b = torch.rand(512, device="cuda"), torch.rand(512, device="cuda")

    def step(stream=None):
        y, ys, kept = mx.layernorm_mx(x, w, b, 1e-5, stream=stream)
        return (y, ys, kept.codes, kept.scales, kept.rstd) + mx.layernorm_mx_backward(kept, w, dy, stream=stream)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(tensor(given((70, 512), 2.0, 10 + k, "bf16"), "bf16"))
        dy.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip([t.clone() for t in out], step()):
            assert torch.equal(p, q)


def test_past_four_gib():
    """Offsets beyond 32 bits in x, dx and what is kept; the last rows against a call on them alone."""
    rows, cols = 70400, 32768
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = tensor(given((16, cols), 2.0, 1, "bf16"), "bf16")
    x[-16:] = tail
    w, b = torch.rand(cols, device="cuda"), torch.rand(cols, device="cuda")
    y, ys, kept = mx.layernorm_mx(x, w, b, 1e-5)
    want = mx.layernorm_mx(tail, w, b, 1e-5)
    assert torch.equal(y[-16:], want[0]) and torch.equal(ys[-16:], want[1])
    assert torch.equal(kept.codes[-16:], want[2].codes) and torch.equal(kept.rstd[-16:], want[2].rstd)
    dx, dw, db = mx.layernorm_mx_backward(kept, w, x)
    want_dx, want_dw, want_db = mx.layernorm_mx_backward(want[2], w, tail)
    assert torch.equal(dx[-16:], want_dx)
    # another order of the same 16 rows' sums: at most 32 u of the sizes added, 16 of them below 10
    assert torch.allclose(dw, want_dw, rtol=0, atol=32 * 160 * U) and torch.allclose(db, want_db, rtol=0, atol=32 * 160 * U)
