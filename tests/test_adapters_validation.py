"""Refusals of LayerNorm and of the low-rank adapters (no GPU): every invalid argument gets its
documented status before any HIP call (fake, never-dereferenced pointers), and the tensor
functions raise ValueError."""
import pytest
import torch

import mx_block_scaled_x128_amd as mx

OK, NULL, SHAPE, LD, ALIGN, ENUM, ALIAS = 0, 1, 2, 3, 4, 5, 6
X, Q, S, C, P, R, W, B = (0x100000 * i for i in range(1, 9))
MIS = 0x900008


def test_mx_layernorm_forward():
    def f(x=X, dt=1, rows=64, cols=256, ldx=256, w=W, b=B, eps=1e-5, fmt=0, rule=0, y=Q, ldy=256, ys=S, k=C, ldk=256,
          ks=P, r=R):
        return mx.mx_layernorm_forward(x, dt, rows, cols, ldx, w, b, eps, fmt, rule, y, ldy, ys, k, ldk, ks, r, None)
    assert f(dt=2) == ENUM and f(fmt=2) == ENUM and f(rule=-1) == ENUM
    assert f(rows=-1) == SHAPE and f(cols=48, ldx=48) == SHAPE and f(cols=32800, ldx=32800) == SHAPE
    assert f(eps=-1e-6) == SHAPE and f(eps=float("nan")) == SHAPE and f(eps=float("inf")) == SHAPE
    assert f(rows=0, x=None, w=None, b=None, y=None, ys=None, k=None, ks=None, r=None) == OK and f(cols=0, x=None) == OK
    assert f(x=None) == NULL and f(y=None) == NULL and f(ys=None) == NULL and f(w=None) == NULL  # b without w
    assert f(k=None) == NULL and f(ks=None) == NULL and f(r=None) == NULL and f(k=None, ks=None) == NULL
    assert f(ldx=240) == LD and f(ldx=264) == LD and f(ldy=248) == LD and f(ldk=128) == LD
    for name in ("x", "w", "b", "y", "k"):
        assert f(**{name: MIS}) == ALIGN, name
    assert f(r=R + 2) == ALIGN
    assert f(y=X) == ALIAS and f(ys=W) == ALIAS and f(k=B) == ALIAS and f(ks=S) == ALIAS and f(r=X) == ALIAS


def test_mx_layernorm_backward():
    def f(k=C, ldk=256, ks=P, r=R, fmt=1, w=W, dy=X, dt=0, lddy=256, rows=64, cols=256, dx=Q, lddx=256, dw=S, db=B,
          work=0xA00000):
        return mx.mx_layernorm_backward(k, ldk, ks, r, fmt, w, dy, dt, lddy, rows, cols, dx, lddx, dw, db, work, None)
    assert f(dt=3) == ENUM and f(fmt=2) == ENUM
    assert f(rows=-1) == SHAPE and f(cols=16) == SHAPE and f(cols=32800) == SHAPE
    assert f(cols=0, dw=None, db=None) == OK
    for name in ("k", "ks", "r", "dy", "dx", "dw", "db", "work"):
        assert f(**{name: None}) == NULL, name
    assert f(ldk=240) == LD and f(lddy=264) == LD and f(lddx=128) == LD
    for name in ("k", "w", "dy", "dx", "dw", "db", "work"):
        assert f(**{name: MIS}) == ALIGN, name
    assert f(r=R + 1) == ALIGN
    assert f(dx=X) == ALIAS and f(dw=W) == ALIAS and f(db=S) == ALIAS and f(work=X) == ALIAS and f(work=Q) == ALIAS


def test_layernorm_workspace():
    assert mx.mx_layernorm_backward_workspace(0, 256) == 0 and mx.mx_layernorm_backward_workspace(5, 48) == 0
    assert mx.mx_layernorm_backward_workspace(-1, 256) == 0 and mx.mx_layernorm_backward_workspace(5, 40000) == 0
    assert mx.mx_layernorm_backward_workspace(1, 256) == 2 * 256 * 4
    assert 0 < mx.mx_layernorm_backward_workspace(1 << 20, 32768) < 1 << 27


def test_layernorm_tensors():
    x, w = torch.zeros(4, 64), torch.zeros(64)
    q, s, r = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), torch.zeros(4)
    kept = mx.LayernormKept(q, s, r, mx.E4M3)
    for call, match in ((lambda: mx.layernorm_mx(x, w, w, 1e-5), "CUDA tensor"),
                        (lambda: mx.layernorm_mx(x.half(), w, w, 1e-5), "float32 or bfloat16"),
                        (lambda: mx.layernorm_mx(x[:, :40], None, None, 1e-5), "multiple of 32"),
                        (lambda: mx.layernorm_mx(x, w[:32], None, 1e-5), "w must"),
                        (lambda: mx.layernorm_mx(x, w, w.double(), 1e-5), "b must"),
                        (lambda: mx.layernorm_mx(x, None, w, 1e-5), "b without w"),
                        (lambda: mx.layernorm_mx(x, w, w, 1e-5, mx.E2M1), "fmt"),
                        (lambda: mx.layernorm_mx(x.t(), w, w, 1e-5), "column stride"),
                        (lambda: mx.layernorm_mx_backward(kept, w, x), "CUDA tensor"),
                        (lambda: mx.layernorm_mx_backward(kept._replace(rstd=r[:3]), w, x), "rstd"),
                        (lambda: mx.layernorm_mx_backward(kept._replace(scales=s[:, :1]), w, x), "scales"),
                        (lambda: mx.layernorm_mx_backward(kept, w, x[:, :32]), "dy"),
                        (lambda: mx.layernorm_mx_backward(kept, x, x), "w must")):
        with pytest.raises(ValueError, match=match):
            call()
