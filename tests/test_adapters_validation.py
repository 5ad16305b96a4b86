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


U, V = 0xB00000, 0xC00000


def test_mx_adapter_project():
    def f(M=64, K=256, a=X, lda=256, fmt=0, sa=S, ids=B, n=4, rank=16, down=W, ldd=256, stride=4096, alpha=R, p=C, work=V):
        return mx.mx_adapter_project(M, K, a, lda, fmt, sa, ids, n, rank, down, ldd, stride, alpha, p, work, None)
    assert f(fmt=3) == ENUM and f(fmt=-1) == ENUM
    assert f(M=-1) == SHAPE and f(M=2 ** 27 + 1) == SHAPE and f(K=192) == SHAPE and f(K=-128) == SHAPE
    assert f(n=-1) == SHAPE and f(n=2 ** 30 + 1) == SHAPE
    assert f(rank=0) == SHAPE and f(rank=12) == SHAPE and f(rank=264) == SHAPE and f(rank=-8) == SHAPE
    assert f(M=0, a=None, sa=None, ids=None, down=None, alpha=None, p=None) == OK
    for name in ("a", "sa", "ids", "down", "p"):
        assert f(**{name: None}) == NULL, name
    assert f(lda=240) == LD and f(lda=264) == LD and f(lda=2 ** 22 + 16) == LD
    assert f(ldd=248) == LD and f(ldd=260) == LD and f(ldd=2 ** 22 + 8) == LD and f(stride=4) == LD and f(stride=-8) == LD
    assert mx.mx_adapter_project_workspace(2000, 4096, 16) > 0
    large = dict(M=2000, K=4096, lda=4096, ldd=4096, stride=65536)
    assert f(work=None, **large) == NULL and f(work=X, **large) == ALIAS and f(work=C, **large) == ALIAS
    for name in ("a", "down", "p", "work"):
        assert f(**{name: MIS}) == ALIGN, name
    assert f(sa=S + 2) == ALIGN and f(ids=B + 2) == ALIGN and f(alpha=R + 1) == ALIGN
    for other in (X, S, B, W, R):
        assert f(p=other) == ALIAS, other


def test_mxfp4_gemm_adapted():
    def f(M=64, N=96, K=256, a=X, lda=256, fmt=0, sa=S, b=Q, ldb=128, sb=P, ids=B, n=4, rank=16, down=W, ldd=256, ds=4096,
          up=U, ldu=16, us=1536, alpha=R, p=V, c=C, ldc=96, dt=0, work=0xD00000):
        return mx.mxfp4_gemm_adapted(M, N, K, a, lda, fmt, sa, b, ldb, sb, ids, n, rank, down, ldd, ds, up, ldu, us, alpha,
                                     p, c, ldc, dt, work, None)
    assert f(fmt=3) == ENUM and f(dt=2) == ENUM
    assert f(M=-1) == SHAPE and f(N=-1) == SHAPE and f(K=100) == SHAPE and f(rank=20) == SHAPE and f(n=-2) == SHAPE
    assert f(M=2 ** 27 + 1) == SHAPE and f(N=2 ** 30) == SHAPE and f(K=2 ** 30) == SHAPE
    assert f(M=0, a=None, b=None, c=None, p=None, ids=None) == OK
    for name in ("a", "sa", "b", "sb", "ids", "down", "up", "p", "c"):
        assert f(**{name: None}) == NULL, name
    assert f(lda=128) == LD and f(ldb=136) == LD and f(ldc=80) == LD and f(ldc=104) == LD
    assert f(lda=2 ** 22 + 16) == LD and f(ldb=2 ** 22 + 16) == LD
    assert f(ldd=128) == LD and f(ldu=8) == LD and f(ldu=20) == LD and f(us=1540) == LD and f(ds=-8) == LD
    large = dict(M=2000, K=4096, lda=4096, ldb=2048, ldd=4096, ds=65536)
    assert f(work=None, **large) == NULL and f(work=U, **large) == ALIAS and f(work=V, **large) == ALIAS
    for name in ("a", "b", "down", "up", "p", "c", "work"):
        assert f(**{name: MIS}) == ALIGN, name
    assert f(sa=S + 1) == ALIGN and f(sb=P + 2) == ALIGN and f(ids=B + 1) == ALIGN and f(alpha=R + 2) == ALIGN
    for other in (X, Q, S, P, B, W, U, R):
        assert f(p=other) == ALIAS and f(c=other) == ALIAS, other
    assert f(c=V) == ALIAS


def test_mx_adapter_grad():
    def f(M=64, cols=256, z=X, ldz=256, fmt=0, sz=S, p=P, rank=16, ids=B, n=4, t=0, grad=C, work=V):
        return mx.mx_adapter_grad(M, cols, z, ldz, fmt, sz, p, rank, ids, n, t, grad, work, None)
    assert f(fmt=3) == ENUM
    assert f(M=-1) == SHAPE and f(M=2 ** 27 + 1) == SHAPE and f(cols=48) == SHAPE and f(cols=-32) == SHAPE
    assert f(rank=4) == SHAPE and f(n=-1) == SHAPE and f(n=2 ** 24, cols=256) == SHAPE and f(M=0, n=2 ** 24) == SHAPE
    assert f(cols=0, z=None, grad=None) == OK and f(n=0, grad=None) == OK
    for name in ("z", "sz", "p", "ids", "grad"):
        assert f(**{name: None}) == NULL, name
    assert mx.mx_adapter_grad_workspace(8192, 256, 16, 1) > 0 and f(M=8192, n=1, work=None) == NULL
    assert f(ldz=240) == LD and f(ldz=264) == LD and f(ldz=2 ** 22 + 16) == LD
    for name in ("z", "p", "grad", "work"):
        assert f(**{name: MIS}) == ALIGN, name
    assert f(ids=B + 2) == ALIGN
    for other in (X, S, P, B):
        assert f(grad=other) == ALIAS and f(M=8192, n=1, work=other) == ALIAS, other
    assert f(M=8192, n=1, work=C) == ALIAS


def test_adapter_project_workspace():
    for bad in ((-1, 256, 16), (64, 200, 16), (64, 256, 9), (0, 256, 16), (2 ** 27 + 1, 256, 16), (64, 18944, 64)):
        assert mx.mx_adapter_project_workspace(*bad) == 0, bad
    for M, K, rank in ((256, 18944, 64), (257, 1 << 22, 256), (65536, 18944, 256), (8192, 18944, 16), (1 << 27, 128, 8)):
        assert mx.mx_adapter_project_workspace(M, K, rank) <= 512 * 128 * rank * 4


def test_adapter_grad_workspace():
    for bad in ((-1, 256, 16, 1), (64, 40, 16, 1), (64, 256, 9, 1), (64, 256, 16, -1), (64, 256, 16, 0), (0, 256, 16, 1)):
        assert mx.mx_adapter_grad_workspace(*bad) == 0, bad
    # at most 256 MB of sums, and the counts
    for M, C, rank, n in ((1 << 20, 18944, 256, 1), (1 << 20, 18944, 16, 8), (1 << 27, 32, 8, 1), (8192, 16384, 128, 48)):
        assert mx.mx_adapter_grad_workspace(M, C, rank, n) <= (256 << 20) + (1 << 16)


def test_adapter_tensors():
    a, sa = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8)
    b, sb = torch.zeros(32, 128, dtype=torch.uint8), torch.zeros(32, 8, dtype=torch.uint8)
    down, up = torch.zeros(3, 16, 256, dtype=torch.bfloat16), torch.zeros(3, 32, 16, dtype=torch.bfloat16)
    ids, alpha, p = torch.zeros(4, dtype=torch.int32), torch.zeros(3), torch.zeros(4, 16)

    def project(a=a, sa=sa, fmt=mx.E4M3, down=down, ids=ids, alpha=alpha):
        return mx.adapter_project_mx(a, sa, fmt, down, ids, alpha)

    def gemm(a=a, sa=sa, b=b, sb=sb, down=down, up=up, ids=ids, alpha=alpha, **kw):
        return mx.mxfp4_adapted_gemm(a, sa, mx.E4M3, b, sb, down, up, ids, alpha, **kw)

    def grad(p=p, z=a, sz=sa, ids=ids, n=3):
        return mx.adapter_grad_mx(p, z, sz, mx.E4M3, ids, n)
    for call, match in ((project, "CUDA tensor"), (gemm, "CUDA tensor"), (grad, "CUDA tensor"),
                        (lambda: project(fmt=5), "a_fmt"), (lambda: project(a=a[:, :96], sa=sa[:, :3]), "multiple of 128"),
                        (lambda: project(down=down.float()), "bfloat16"), (lambda: project(down=down[0]), "3-D"),
                        (lambda: project(down=down[:, :12]), "rank"), (lambda: project(down=down[:, :, :128]), "down must have"),
                        (lambda: project(down=down.transpose(1, 2).contiguous().transpose(1, 2)), "column stride"),
                        (lambda: project(ids=ids.long()), "ids must"), (lambda: project(ids=ids[:3]), "ids must"),
                        (lambda: project(alpha=alpha[:2]), "alpha must"), (lambda: project(sa=sa[:, :4]), "a_scales"),
                        (lambda: gemm(up=up[:2]), "up must have"), (lambda: gemm(up=up[:, :31]), "up must have"),
                        (lambda: gemm(up=up.half()), "bfloat16"), (lambda: gemm(b=b[:, :64]), "K = "),
                        (lambda: gemm(sb=sb[:3]), "b_scales"), (lambda: gemm(out_dtype=torch.float16), "out_dtype"),
                        (lambda: gemm(out=torch.zeros(4, 31)), "out must"), (lambda: grad(p=p.double()), "p must"),
                        (lambda: grad(p=p[:, :12].contiguous()), "rank"), (lambda: grad(p=p[:3]), "p must"),
                        (lambda: grad(n=-1), "negative"), (lambda: grad(ids=ids[:2]), "ids must"),
                        (lambda: grad(z=a[:, :48], sz=sa), "multiple of 32")):
        with pytest.raises(ValueError, match=match):
            call()
