"""The MX operators' refusals (no GPU): every invalid argument gets its documented status
before any HIP call (fake, never-dereferenced pointers), the tensor functions raise
ValueError, and the plain 64-bit implementation of the tests agrees with torch's formats."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref

OK, NULL, SHAPE, LD, ALIGN, ENUM, ALIAS = 0, 1, 2, 3, 4, 5, 6
X, Q, S, C, P, R = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000
MIS = 0x700008


def test_mxfp4_quantize():
    def f(x=X, dt=1, rows=64, cols=256, ldx=256, rule=1, q=Q, ldq=128, s=S):
        return mx.mxfp4_quantize(x, dt, rows, cols, ldx, rule, q, ldq, s, None)
    assert f(dt=2) == ENUM and f(dt=-1) == ENUM and f(rule=2) == ENUM
    assert f(rows=-1) == SHAPE and f(cols=48, ldx=48) == SHAPE and f(rows=2 ** 31) == SHAPE
    assert f(rows=0, x=None, q=None, s=None) == OK and f(cols=0, x=None) == OK
    assert f(x=None) == NULL and f(q=None) == NULL and f(s=None) == NULL
    assert f(ldx=240) == LD and f(ldx=264) == LD and f(ldq=112) == LD and f(ldq=136) == LD
    assert f(x=MIS) == ALIGN and f(q=MIS) == ALIGN
    assert f(q=X) == ALIAS and f(s=X) == ALIAS and f(s=Q) == ALIAS


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_mx_dequantize(fmt):
    row = 128 if fmt == 2 else 256

    def f(q=Q, ldq=row, fm=fmt, s=S, rows=64, cols=256, y=C, dt=0, ldy=256):
        return mx.mx_dequantize(q, ldq, fm, s, rows, cols, y, dt, ldy, None)
    assert f(fm=3) == ENUM and f(dt=2) == ENUM
    assert f(cols=16) == SHAPE and f(rows=-2) == SHAPE
    assert f(rows=0, q=None, s=None, y=None) == OK
    assert f(q=None) == NULL and f(s=None) == NULL and f(y=None) == NULL
    assert f(ldq=row - 16) == LD and f(ldq=row + 8) == LD and f(ldy=128) == LD
    assert f(q=MIS) == ALIGN and f(y=MIS) == ALIGN
    assert f(y=Q) == ALIAS and f(y=S) == ALIAS


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_mx_quantize_t(fmt):
    row = 64 if fmt == 2 else 128

    def f(x=X, dt=1, rows=100, cols=256, ldx=256, fm=fmt, rule=0, qt=Q, ldqt=row, out=128, st=S):
        return mx.mx_quantize_t(x, dt, rows, cols, ldx, fm, rule, qt, ldqt, out, st, None)
    assert f(fm=3) == ENUM and f(dt=2) == ENUM and f(rule=-1) == ENUM
    assert f(out=96) == SHAPE and f(out=112) == SHAPE and f(cols=24, ldx=32) == SHAPE and f(rows=-1) == SHAPE
    assert f(rows=2 ** 30, cols=2 ** 20, ldx=2 ** 20, out=2 ** 30, ldqt=2 ** 30) == SHAPE  # too many tiles
    assert f(out=0, rows=0, x=None, qt=None, st=None) == OK and f(cols=0, x=None) == OK
    assert f(x=None) == NULL and f(qt=None) == NULL and f(st=None) == NULL
    assert f(ldx=240) == LD and f(ldqt=row - 16) == LD and f(ldqt=row + 8) == LD
    assert f(x=MIS) == ALIGN and f(qt=MIS) == ALIGN
    assert f(qt=X) == ALIAS and f(st=X) == ALIAS and f(st=Q) == ALIAS


def test_mx_requantize_t():
    def f(q=X, ldq=256, qf=0, s=P, rows=100, cols=256, fm=1, rule=0, qt=Q, ldqt=128, out=128, st=S):
        return mx.mx_requantize_t(q, ldq, qf, s, rows, cols, fm, rule, qt, ldqt, out, st, None)
    assert f(qf=2) == ENUM and f(fm=3) == ENUM and f(rule=2) == ENUM
    assert f(cols=48, ldq=48) == SHAPE and f(out=64) == SHAPE
    assert f(out=0, rows=0, q=None) == OK
    assert f(q=None) == NULL and f(s=None) == NULL and f(qt=None) == NULL and f(st=None) == NULL
    assert f(ldq=128) == LD and f(ldqt=96) == LD
    assert f(q=MIS) == ALIGN and f(qt=MIS) == ALIGN
    assert f(qt=X) == ALIAS and f(qt=P) == ALIAS and f(st=P) == ALIAS and f(st=Q) == ALIAS


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_mxfp4_gemm(fmt):
    row = 256 if fmt == 2 else 512

    def f(M=64, N=256, K=512, a=X, lda=row, af=fmt, sa=S, b=Q, ldb=256, sb=P, c=C, ldc=256, dt=0):
        return mx.mxfp4_gemm(M, N, K, a, lda, af, sa, b, ldb, sb, c, ldc, dt, None)
    assert f(af=3) == ENUM and f(dt=2) == ENUM
    assert f(K=480) == SHAPE and f(K=32) == SHAPE and f(M=-1) == SHAPE and f(N=2 ** 31) == SHAPE
    assert f(M=0, a=None) == OK and f(N=0, c=None) == OK
    assert f(c=None) == NULL and f(a=None) == NULL and f(b=None) == NULL and f(sa=None) == NULL and f(sb=None) == NULL
    assert f(lda=row - 16) == LD and f(ldb=240) == LD and f(ldb=264) == LD and f(ldc=240) == LD
    assert f(lda=(1 << 24) + 16) == LD and f(ldb=(1 << 24) + 16) == LD
    assert f(a=MIS) == ALIGN and f(b=MIS) == ALIGN and f(c=MIS) == ALIGN
    assert f(sa=S + 2) == ALIGN and f(sb=P + 1) == ALIGN
    assert f(c=X) == ALIAS and f(c=Q) == ALIAS and f(c=S) == ALIAS and f(c=P) == ALIAS


def test_mx_swiglu():
    def f(x=X, dt=1, rows=8, cols=64, ldx=128, fm=0, rule=0, h=Q, ldh=64, hs=S, k=C, ldk=128, ks=P):
        return mx.mx_swiglu_forward(x, dt, rows, cols, ldx, fm, rule, h, ldh, hs, k, ldk, ks, None)

    def b(k=C, ldk=128, ks=P, fm=0, dh=X, dt=1, lddh=64, rows=8, cols=64, dx=Q, lddx=128):
        return mx.mx_swiglu_backward(k, ldk, ks, fm, dh, dt, lddh, rows, cols, dx, lddx, None)
    assert f(fm=2) == ENUM and f(dt=2) == ENUM and f(rule=2) == ENUM and b(fm=2) == ENUM and b(dt=3) == ENUM
    assert f(cols=48) == SHAPE and f(rows=-1) == SHAPE and b(cols=40) == SHAPE
    assert f(rows=0, x=None) == OK and b(rows=0, k=None) == OK
    assert f(x=None) == NULL and f(h=None) == NULL and f(hs=None) == NULL and f(k=None) == NULL and f(ks=None) == NULL
    assert b(k=None) == NULL and b(ks=None) == NULL and b(dh=None) == NULL and b(dx=None) == NULL
    assert f(ldx=64) == LD and f(ldh=72) == LD and f(ldk=64) == LD
    assert b(ldk=64) == LD and b(lddh=48) == LD and b(lddx=64) == LD
    assert f(x=MIS) == ALIGN and f(h=MIS) == ALIGN and f(k=MIS) == ALIGN and b(dx=MIS) == ALIGN and b(dh=MIS) == ALIGN
    assert f(h=X) == ALIAS and f(k=X) == ALIAS and f(k=Q) == ALIAS and f(ks=S) == ALIAS
    assert b(dx=X) == ALIAS and b(dx=C) == ALIAS


def test_mx_rmsnorm():
    def f(x=X, dt=1, rows=8, cols=64, ldx=64, w=P, eps=1e-6, fm=0, rule=0, y=Q, ldy=64, ys=S, k=C, ldk=64, ks=R,
          r=0x800000):
        return mx.mx_rmsnorm_forward(x, dt, rows, cols, ldx, w, eps, fm, rule, y, ldy, ys, k, ldk, ks, r, None)

    def b(k=C, ldk=64, ks=R, r=0x800000, fm=0, w=P, dy=X, dt=1, lddy=64, rows=8, cols=64, dx=Q, lddx=64, dw=0x900000,
          work=0xA00000):
        return mx.mx_rmsnorm_backward(k, ldk, ks, r, fm, w, dy, dt, lddy, rows, cols, dx, lddx, dw, work, None)
    assert f(fm=2) == ENUM and f(dt=2) == ENUM and f(rule=2) == ENUM and b(fm=2) == ENUM and b(dt=2) == ENUM
    assert f(cols=48) == SHAPE and f(cols=32768 + 32, ldx=40000, ldy=40000, ldk=40000) == SHAPE and b(cols=40) == SHAPE
    assert f(eps=-1.0) == SHAPE and f(eps=float("nan")) == SHAPE and f(eps=float("inf")) == SHAPE
    assert f(rows=0, x=None) == OK and b(cols=0, dw=None) == OK
    for k in ("x", "w", "y", "ys", "k", "ks", "r"):
        assert f(**{k: None}) == NULL, k
    for k in ("k", "ks", "r", "w", "dy", "dx", "dw", "work"):
        assert b(**{k: None}) == NULL, k
    assert f(ldx=48) == LD and f(ldy=72) == LD and f(ldk=48) == LD
    assert b(ldk=48) == LD and b(lddy=72) == LD and b(lddx=48) == LD
    assert f(w=MIS) == ALIGN and f(r=0x800002) == ALIGN and b(dw=MIS) == ALIGN and b(work=MIS) == ALIGN
    assert f(y=X) == ALIAS and f(k=X) == ALIAS and f(y=P) == ALIAS and f(k=Q) == ALIAS
    assert b(dx=X) == ALIAS and b(dw=P) == ALIAS and b(work=C) == ALIAS and b(work=Q) == ALIAS
    assert mx.mx_rmsnorm_backward_workspace(8, 64) >= 256
    assert mx.mx_rmsnorm_backward_workspace(8, 48) == 0 and mx.mx_rmsnorm_backward_workspace(-1, 64) == 0


def test_tensor_functions_refuse():
    x = torch.zeros(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    q4 = torch.zeros(4, 32, dtype=torch.uint8)
    w = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mx.quantize_mxfp4(x)
    with pytest.raises(ValueError, match="multiple of 32"):
        mx.quantize_mxfp4(torch.zeros(4, 48))
    with pytest.raises(ValueError, match="float32 or"):
        mx.quantize_mxfp4(x.half())
    with pytest.raises(ValueError, match="fmt"):
        mx.dequantize_mx(q, s, 3)
    with pytest.raises(ValueError, match="scales"):
        mx.dequantize_mx(q4, s[:, :1], mx.E2M1)
    with pytest.raises(ValueError, match="dtype"):
        mx.dequantize_mx(q, s, mx.E4M3, torch.float16)
    with pytest.raises(ValueError, match="rows_out"):
        mx.quantize_mx_t(x, rows_out=2)
    with pytest.raises(ValueError, match="multiple of 16"):
        mx.quantize_mx_t(torch.zeros(4, 40)[:, :24])
    with pytest.raises(ValueError, match="q_fmt"):
        mx.requantize_mx_t(q4, s, mx.E2M1)
    with pytest.raises(ValueError, match="K = "):
        mx.mxfp4_scaled_gemm(q, s, mx.E4M3, q4[:, :16], s)
    with pytest.raises(ValueError, match="multiple of 128"):
        mx.mxfp4_scaled_gemm(q, s, mx.E4M3, q4, s)
    with pytest.raises(ValueError, match="twice"):
        mx.swiglu_mx(torch.zeros(4, 32))
    with pytest.raises(ValueError, match="dh"):
        mx.swiglu_mx_backward(mx.SwigluKept(q, s, mx.E4M3), torch.zeros(4, 64))
    with pytest.raises(ValueError, match="w must"):
        mx.rmsnorm_mx(x, w.double(), 1e-6)
    with pytest.raises(ValueError, match="rstd"):
        mx.rmsnorm_mx_backward(mx.RmsnormKept(q, s, w, mx.E4M3), w, x)


@pytest.mark.parametrize("fmt", [mxref.E4M3, mxref.E5M2])
def test_reference_formats_agree_with_torch(fmt):
    dt = torch.float8_e4m3fn if fmt == mxref.E4M3 else torch.float8_e5m2
    v = torch.arange(256, dtype=torch.uint8).view(dt).float().double().numpy()
    mine = mxref.code_values(fmt)
    fine = np.isfinite(mine)
    assert np.array_equal(mine[fine], v[fine])
    x = np.random.default_rng(0).normal(0, 30, 20000)
    x = np.clip(x, -mxref.fmax(fmt), mxref.fmax(fmt)).astype(np.float32)
    assert np.array_equal(mxref.cast(x.astype(np.float64), fmt), torch.from_numpy(x).to(dt).view(torch.uint8).numpy())


def test_reference_e2m1():
    assert list(mxref.code_values(mxref.E2M1)[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    # ties go to the even code, values above 6 saturate, the sign of zero is kept
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.001, 9.0, -0.0, -0.25])
    assert list(mxref.cast(v, mxref.E2M1)) == [0, 2, 2, 4, 4, 6, 6, 7, 7, 8, 8]
    assert mxref.exponent(np.array([6.0, 6.001, 12.0, 0.0]), mxref.E2M1, mxref.CEIL).tolist() == [0, 1, 1, -127]
    assert mxref.exponent(np.array([4.0, 7.9, 8.0]), mxref.E2M1, mxref.FLOOR).tolist() == [0, 0, 1]


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(1)
    x, dh = rng.normal(0, 2, (3, 64)), rng.normal(0, 1, (3, 32))
    dx = mxref.swiglu_grad(x, dh)
    for k in range(0, 64, 7):
        d = np.zeros_like(x)
        d[:, k] = 1e-6
        num = ((mxref.swiglu(x + d) - mxref.swiglu(x - d)) * dh).sum(1) / 2e-6
        assert np.allclose(num, dx[:, k], rtol=1e-6, atol=1e-8)
    x, w, dy = rng.normal(0, 2, (3, 32)), rng.normal(1, 0.1, 32), rng.normal(0, 1, (3, 32))

    def y(x, w):
        return x * mxref.rstd(x, 1e-6)[:, None] * w
    dx, dw = mxref.rmsnorm_grad(x, mxref.rstd(x, 1e-6), w, dy)
    for k in range(0, 32, 5):
        d = np.zeros_like(x)
        d[:, k] = 1e-6
        assert np.allclose(((y(x + d, w) - y(x - d, w)) * dy).sum(1) / 2e-6, dx[:, k], rtol=1e-5, atol=1e-8)
        e = np.zeros(32)
        e[k] = 1e-6
        assert np.allclose(((y(x, w + e) - y(x, w - e)) * dy).sum() / 2e-6, dw[k], rtol=1e-6, atol=1e-8)


def test_tensor_functions_fail_loudly_without_the_extension(monkeypatch):
    import importlib

    def missing(name, *a):
        raise ImportError("no module named " + name)
    monkeypatch.setattr(mx, "_tensors", None)
    monkeypatch.setattr(importlib, "import_module", missing)
    with pytest.raises(ImportError, match="_tensors is not built"):
        mx.quantize_mxfp4(torch.zeros(1, 32))


def test_library_errors_name_their_call():
    with pytest.raises(mx.MxFp8Error, match="mx_rmsnorm_forward"):
        mx._check(2, "mx_rmsnorm_forward")


def _in_a_new_process(code):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr


def test_a_failed_binding_is_not_taken_for_a_bound_extension():
    """The second call after a failed one fails the same way, and works once the library is there."""
    _in_a_new_process("""
import torch, mx_block_scaled_x128_amd as mx
x, path = torch.zeros(1, 32), mx._LIB_PATH
mx.load_library()
mx._LIB_PATH = path + ".absent"
for _ in range(2):
    try:
        mx.quantize_mxfp4(x)
    except ImportError as e:
        assert "absent" in str(e), e
    else:
        raise AssertionError("no error")
mx._LIB_PATH = path
try:
    mx.quantize_mxfp4(x)
except ValueError as e:
    assert "CUDA tensor" in str(e), e
else:
    raise AssertionError("no error")
""")


def test_the_extension_alone_refuses_to_run():
    """Imported without the package's binding, its functions raise; the package binds it all the same."""
    _in_a_new_process("""
import torch, mx_block_scaled_x128_amd as mx
from mx_block_scaled_x128_amd import _mx_tensors
x = torch.zeros(1, 32)
for call, error in ((_mx_tensors.quantize_mxfp4, ImportError), (mx.quantize_mxfp4, ValueError)):
    try:
        call(x, 1, None)
    except error:
        pass
    else:
        raise AssertionError("no error")
""")


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_transposed_grids_stay_below_the_launch_limit(fmt):
    """Tiles are launched in multiples of 8 with up to 512 threads each, fewer than 2^32 in all: 2^23 - 8 tiles pass
    the shape check (the null pointer is then what is refused), one more does not."""
    most = 2 ** 23 - 8
    for tiles, status in ((most, NULL), (most + 1, SHAPE), (most + 7, SHAPE), (most + 8, SHAPE)):
        out = 128 * tiles
        ld = out // 2 if fmt == 2 else out
        assert mx.mx_quantize_t(None, 1, 100, 128, 128, fmt, 0, Q, ld, out, S, None) == status, tiles
        assert mx.mx_requantize_t(None, 128, 0, P, 100, 128, fmt, 0, Q, ld, out, S, None) == status, tiles
    assert mx.mx_quantize_t(None, 1, 100, 112, 112, fmt, 0, Q, ld, 128 * most - 96, S, None) == NULL


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_mxfp4_gemm_refuses_rows_past_its_offsets(fmt):
    """2^22 bytes from row to row are taken (a misaligned output is what is refused here), 16 more are not."""
    most = 1 << 22
    for lda, ldb, status in ((most, most, OK), (most + 16, 256, LD), (512, most + 16, LD)):
        got = mx.mxfp4_gemm(64, 256, 512, X, lda, fmt, S, Q, ldb, P, MIS if status == OK else C, 256, 0, None)
        assert got == (ALIGN if status == OK else status)
