"""Low-rank adapters beside the MXFP4 product, and their gradients, against plain sums in 64 bits.

Tolerances, u = 2^-24.  p adds K exact products in fp32: a lane or matrix instruction adds at
most K / 8 in a row, the joints 64 more, and alpha rounds once: (K / 8 + 66) u of the absolute
sizes.  What an adapter adds to c is p times up: rank + 8 additions, that many u of the sizes, and
what p is off by.  (Tiles with bf16 results take p's leading 16 bits; 2^-16 of the sizes is
inside the bf16 results' own bound, which has the products' 2^-12.)  The shared product itself is off by 2^-12 of its
sizes, as everywhere; a row without an adapter has its bits.  A gradient adds its rows in fp32:
rows + 16 u.  bf16 rounds once more (2^-8 of the value)."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref
from gpu_helpers import dev, dev_ld16, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FMTS = [mx.E4M3, mx.E5M2, mx.E2M1]


def codes(rows, K, fmt, seed, spread=2):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (rows, K)) * mxref.pow2(rng.integers(-spread, spread + 1, (rows, K // 32)).repeat(32, axis=1))
    return mxref.quantize(x, fmt, mxref.CEIL)


def matrices(shape, seed, scale):
    return mxref.bf16((np.random.default_rng(seed).normal(0, 1, shape) * scale).astype(np.float32))


def some_ids(rows, adapters, order, seed=3):
    """"mixed": any id, one row in six without (-1, or past the last one); "runs": runs of random lengths;
    "one": the last adapter everywhere; "none"."""
    rng = np.random.default_rng(seed)
    if order == "one":
        return np.full(rows, adapters - 1, np.int32)
    if order == "none":
        return np.where(np.arange(rows) % 2, -1, adapters).astype(np.int32)
    if order == "runs":
        ends = np.sort(rng.integers(0, rows + 1, 2 * adapters))
        return rng.integers(-1, adapters, 2 * adapters + 1)[np.searchsorted(ends, np.arange(rows), side="right")].astype(np.int32)
    ids = rng.integers(0, adapters, rows)
    bad = rng.choice([-1, adapters, 2 ** 31 - 1, -2 ** 31], rows)
    return np.where(rng.random(rows) < 1 / 6, bad, ids).astype(np.int32)


class Case:
    def __init__(self, M, K, N, fmt, rank, adapters, order, seed=1, alpha=True, pad=0):
        self.M, self.K, self.N, self.fmt, self.rank, self.adapters = M, K, N, fmt, rank, adapters
        self.a, self.sa = codes(M, K, fmt, seed)
        self.b, self.sb = codes(N, K, mx.E2M1, seed + 1)
        self.down, self.up = matrices((adapters, rank, K), seed + 2, K ** -0.5), matrices((adapters, N, rank), seed + 3, 0.5)
        self.alpha = np.linspace(0.5, 2.0, adapters).astype(np.float32) if alpha else None
        self.ids = some_ids(M, adapters, order, seed)
        self.put(pad)

    def put(self, pad=0):
        self.a_d, self.sa_d = dev_ld16(self.a), dev(self.sa)
        self.b_d, self.sb_d = dev_ld16(self.b), dev(self.sb)
        self.down_d, self.up_d = on_device(self.down, pad), on_device(self.up, pad)
        self.ids_d = torch.from_numpy(self.ids).cuda()
        self.alpha_d = None if self.alpha is None else torch.from_numpy(self.alpha).cuda()

    def project(self, **kw):
        return mx.adapter_project_mx(self.a_d, self.sa_d, self.fmt, self.down_d, self.ids_d, self.alpha_d, **kw)

    def product(self, **kw):
        return mx.mxfp4_adapted_gemm(self.a_d, self.sa_d, self.fmt, self.b_d, self.sb_d, self.down_d, self.up_d,
                                     self.ids_d, self.alpha_d, **kw)

    def base(self, **kw):
        return mx.mxfp4_scaled_gemm(self.a_d, self.sa_d, self.fmt, self.b_d, self.sb_d, **kw)

    def own(self, n):
        return np.nonzero(self.ids == n)[0]

    def exact_p(self):
        """p and the bound of its error."""
        x = mxref.dequantize(self.a, self.sa, self.fmt)
        p, size = np.zeros((self.M, self.rank)), np.zeros((self.M, self.rank))
        for n in range(self.adapters):
            rows, f = self.own(n), 1.0 if self.alpha is None else float(self.alpha[n])
            d = self.down[n].astype(np.float64)
            p[rows], size[rows] = f * (x[rows] @ d.T), f * (np.abs(x[rows]) @ np.abs(d).T)
        return p, (self.K / 8 + 66) * U * size

    def exact_c(self):
        x, w = mxref.dequantize(self.a, self.sa, self.fmt), mxref.dequantize(self.b, self.sb, mx.E2M1)
        c, tol = x @ w.T, 2.0 ** -12 * (np.abs(x) @ np.abs(w).T)
        p, off = self.exact_p()
        for n in range(self.adapters):
            rows, u = self.own(n), self.up[n].astype(np.float64)
            c[rows] += p[rows] @ u.T
            tol[rows] += (off[rows] + (self.rank + 8) * U * np.abs(p[rows])) @ np.abs(u).T
        return c, tol


def on_device(m, pad):
    """bf16 [n][rows][cols], with pad: rows pad elements apart more, matrices 3 pad more."""
    t = torch.from_numpy(m).bfloat16()
    if not pad:
        return t.cuda()
    n, rows, cols = m.shape
    flat = torch.zeros(n * (rows * (cols + pad) + 3 * pad), dtype=torch.bfloat16, device="cuda")
    view = flat.as_strided((n, rows, cols), (rows * (cols + pad) + 3 * pad, cols + pad, 1))
    view.copy_(t)
    return view


def close(y, exact, tol):
    off = np.abs(host(y).astype(np.float64) - exact)
    assert (off <= tol).all(), ((off / np.maximum(tol, 1e-300)).max(), np.argwhere(~(off <= tol))[:3])


PROJECT = [(1, 128, 8, 1, "one"), (1, 3584, 16, 4, "one"), (3, 384, 24, 2, "mixed"), (61, 4992, 64, 9, "mixed"),
           (256, 1152, 8, 300, "mixed"), (257, 256, 8, 5, "mixed"), (300, 2176, 16, 3, "runs"), (515, 896, 40, 2, "runs"),
           (1000, 128, 128, 7, "mixed"), (290, 640, 256, 2, "runs"), (40, 512, 256, 3, "mixed"), (70, 256, 16, 3, "none"),
           (333, 256, 16, 3, "none"), (1025, 8960, 16, 1, "one")]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,rank,adapters,order", PROJECT)
def test_project(M, K, rank, adapters, order, fmt):
    for alpha, pad in ((True, 0), (False, 16)):
        c = Case(M, K, 32, fmt, rank, adapters, order, alpha=alpha, pad=pad)
        p = c.project()
        assert p.shape == (M, rank) and p.dtype == torch.float32 and torch.equal(p, c.project())
        exact, tol = c.exact_p()
        close(p, exact, tol)


# every form of the product: few rows (1, 2 and 4 tiles wide, with and without A in LDS), 128 x 128 tiles with
# four and two buffers, 256 x 256 ones, with a tail of quadrants
PRODUCT = [(1, 128, 1, 8, 1, "one"), (1, 3584, 300, 16, 3, "one"), (2, 384, 100, 8, 2, "mixed"),
           (13, 1152, 17, 24, 5, "mixed"), (16, 3584, 8200, 16, 4, "mixed"), (9, 2304, 50, 256, 3, "mixed"),
           (37, 1280, 1536, 64, 9, "mixed"), (61, 18944, 64, 40, 4, "mixed"), (48, 640, 2200, 8, 6, "mixed"),
           (64, 512, 9000, 16, 3, "runs"), (100, 384, 258, 32, 11, "mixed"), (200, 1024, 515, 16, 3, "runs"),
           (300, 128, 260, 64, 3, "runs"), (520, 1664, 1030, 8, 4, "mixed"), (700, 256, 3000, 40, 5, "runs"),
           (2049, 256, 4100, 16, 6, "runs"), (4100, 384, 4352, 24, 3, "runs")]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N,rank,adapters,order", PRODUCT)
def test_product(M, K, N, rank, adapters, order, fmt):
    c = Case(M, K, N, fmt, rank, adapters, order, pad=8)
    y, p = c.product()
    assert y.shape == (M, N) and y.dtype == torch.float32 and torch.equal(p, c.project())
    exact, tol = c.exact_c()
    close(y, exact, tol)
    half, p16 = c.product(out_dtype=torch.bfloat16)
    assert half.dtype == torch.bfloat16 and torch.equal(p16, p)
    close(half, exact, tol + 2.0 ** -8 * (np.abs(exact) + tol))
    # rows without an adapter: the shared product, bit for bit
    none = torch.from_numpy((c.ids < 0) | (c.ids >= adapters)).cuda()
    assert torch.equal(y[none], c.base()[none])
    assert torch.equal(half[none], c.base(out_dtype=torch.bfloat16)[none])


# past 256 rows several workgroups share the adapters of the projection's tiles; a wave of the large tiles may name 128
@pytest.mark.parametrize("M,K,N,rank,adapters", [(257, 640, 64, 16, 150), (300, 1280, 260, 8, 2), (700, 256, 300, 40, 90),
                                                 (515, 2176, 130, 64, 1000), (4100, 128, 4352, 8, 400)])
def test_rows_of_many_adapters(M, K, N, rank, adapters):
    c = Case(M, K, N, mx.E4M3, rank, adapters, "mixed")
    y, p = c.product()
    p64, tol = c.exact_p()
    close(p, p64, tol)
    exact, tol = c.exact_c()
    close(y, exact, tol)
    close(c.product(out_dtype=torch.bfloat16)[0], exact, tol + 2.0 ** -8 * (np.abs(exact) + tol))
    assert torch.equal(p, c.project()) and torch.equal(y, c.product()[0])


@pytest.mark.parametrize("M,K,N,rank,adapters,order", [s for s in PRODUCT if s[0] * s[2] < 3e6])
def test_what_the_adapter_adds(M, K, N, rank, adapters, order):
    """The shared weight zero: c is the adapters' part alone, with fp32's precision."""
    c = Case(M, K, N, mx.E4M3, rank, adapters, order, seed=5)
    c.b[:], c.sb[:] = 0, 127
    c.put()
    y, p = c.product()
    p64 = host(p).astype(np.float64)
    exact, size = np.zeros((M, N)), np.zeros((M, N))
    for n in range(adapters):
        rows, u = c.own(n), c.up[n].astype(np.float64)
        exact[rows], size[rows] = p64[rows] @ u.T, np.abs(p64[rows]) @ np.abs(u).T
    close(y, exact, (rank + 8) * U * size)


@pytest.mark.parametrize("order", ["none", "one", "mixed"])
@pytest.mark.parametrize("M,N", [(5, 300), (300, 700)])
def test_no_adapters_no_columns_no_k(M, N, order):
    c = Case(M, 256, N, mx.E4M3, 8, 2, order)
    empty = c.down_d[:0], c.up_d[:0]
    y, p = mx.mxfp4_adapted_gemm(c.a_d, c.sa_d, c.fmt, c.b_d, c.sb_d, *empty, c.ids_d)
    assert torch.equal(y, c.base()) and not p.any() and p.shape == (M, 8)
    y, p = mx.mxfp4_adapted_gemm(c.a_d, c.sa_d, c.fmt, c.b_d[:0], c.sb_d[:0], c.down_d, c.up_d[:, :0], c.ids_d, c.alpha_d)
    assert y.shape == (M, 0) and torch.equal(p, c.project())
    z = torch.empty((M, 0), dtype=torch.uint8, device="cuda")
    y, p = mx.mxfp4_adapted_gemm(z, z, c.fmt, c.b_d[:, :0], c.sb_d[:, :0], c.down_d[:, :, :0], c.up_d, c.ids_d, c.alpha_d)
    assert y.shape == (M, N) and not y.any() and not p.any()
    y, p = mx.mxfp4_adapted_gemm(c.a_d[:0], c.sa_d[:0], c.fmt, c.b_d, c.sb_d, c.down_d, c.up_d, c.ids_d[:0])
    assert y.shape == (0, N) and p.shape == (0, 8)
    assert mx.adapter_grad_mx(p, c.a_d[:0], c.sa_d[:0], c.fmt, c.ids_d[:0], 3).eq(0).all()
    assert mx.adapter_grad_mx(c.project(), c.a_d, c.sa_d, c.fmt, c.ids_d, 0).shape == (0, 8, 256)


@pytest.mark.parametrize("M,N,K", [(7, 96, 256), (40, 520, 256), (100, 300, 384), (700, 700, 256), (4100, 4352, 128)])
@pytest.mark.parametrize("part", ["down", "up", "row"])
def test_bad_values_stay_with_their_adapter(part, M, N, K):
    """An infinity or a NaN in one adapter, or in one row, changes no bit of the rows of others."""
    c = Case(M, K, N, mx.E4M3, 16, 3, "mixed")
    c.ids[:2] = 2, 1
    c.put()
    want, want_p = c.product()
    grad = mx.adapter_grad_mx(want_p, c.a_d, c.sa_d, c.fmt, c.ids_d, 3)
    if part == "row":
        bad = np.zeros(M, bool)
        bad[0] = True
        c.sa[0, :] = 255
    else:
        bad = c.ids == 2
        m = getattr(c, part)[2]
        m[:, :] = np.nan
        m[::2, 1] = np.inf
    c.put()
    y, p = c.product()
    ok = torch.from_numpy(~bad).cuda()
    assert torch.equal(y[ok], want[ok]) and torch.equal(p[ok], want_p[ok])
    assert not torch.isfinite(y[~ok]).any()
    got = mx.adapter_grad_mx(p, c.a_d, c.sa_d, c.fmt, c.ids_d, 3)
    if part != "up":
        assert torch.equal(got[:2], grad[:2]) and not torch.isfinite(got[2]).all()


GRAD = [(1, 32, 8, 1, "one"), (5, 96, 8, 2, "mixed"), (515, 8960, 8, 3, "runs"), (600, 288, 16, 2, "mixed"),
        (300, 1536, 24, 5, "mixed"), (1100, 544, 64, 3, "runs"), (2600, 256, 32, 1, "one"), (4097, 128, 128, 2, "runs"),
        (900, 64, 256, 4, "mixed"), (70, 128, 16, 40, "mixed"), (333, 256, 16, 3, "none"), (3000, 512, 8, 1100, "mixed")]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,C,rank,adapters,order", GRAD)
def test_grad(M, C, rank, adapters, order, fmt):
    z, sz = codes(M, C, fmt, M + C)
    p = np.random.default_rng(2).normal(0, 1, (M, rank)).astype(np.float32)
    ids = some_ids(M, adapters, order)
    args = torch.from_numpy(p).cuda(), dev(z, pitch=z.shape[1] + (-z.shape[1]) % 16 + 16), dev(sz), fmt, torch.from_numpy(ids).cuda(), adapters
    got = mx.adapter_grad_mx(*args)
    turned = mx.adapter_grad_mx(*args, transposed=True)
    assert got.shape == (adapters, rank, C) and turned.shape == (adapters, C, rank)
    assert torch.equal(turned.transpose(1, 2), got) and torch.equal(got, mx.adapter_grad_mx(*args))
    v, p64 = mxref.dequantize(z, sz, fmt), p.astype(np.float64)
    exact, size = np.zeros((adapters, rank, C)), np.zeros((adapters, rank, C))
    count = np.zeros(adapters)
    for n in np.unique(ids[(ids >= 0) & (ids < adapters)]):
        rows = ids == n
        exact[n], size[n], count[n] = p64[rows].T @ v[rows], np.abs(p64[rows]).T @ np.abs(v[rows]), rows.sum()
    close(got, exact, (count + 16)[:, None, None] * U * size)


def test_grad_of_values_that_take_all_of_fp32():
    """p of every size from 2^-40 to 2^40 and codes under every scale: each row alone, so that nothing is added."""
    M, C, rank = 64, 64, 8
    z, sz = codes(M, C, mx.E4M3, 1, spread=30)
    p = (np.random.default_rng(4).normal(0, 1, (M, rank)) * mxref.pow2(np.arange(M) % 81 - 40)[:, None]).astype(np.float32)
    got = mx.adapter_grad_mx(torch.from_numpy(p).cuda(), dev(z), dev(sz), mx.E4M3, torch.arange(M, dtype=torch.int32, device="cuda"), M)
    exact = p.astype(np.float64)[:, :, None] * mxref.dequantize(z, sz, mx.E4M3)[:, None, :]
    close(got, exact, 3 * U * np.abs(exact))  # three parts' products added


def test_scales_at_their_ends():
    """Blocks under the smallest and the largest scales, and the NaN one, through p and the gradients."""
    c = Case(300, 128, 32, mx.E4M3, 8, 1, "one", alpha=False)
    c.sa[0::4], c.sa[1::4], c.sa[2::4] = 0, 1, 254
    c.a[2::4] = np.where((c.a[2::4] & 0x7F) > 0x30, 0x30, c.a[2::4])  # at most 0.5, so that 2^127 times it and sums of 128 stay finite
    c.down *= mxref.pow2(-10).astype(np.float32)
    c.sa[3::4, 1] = 255
    c.put()
    for rows in (slice(0, 300), slice(0, 200)):  # both kernels
        p = mx.adapter_project_mx(c.a_d[rows], c.sa_d[rows], c.fmt, c.down_d, c.ids_d[rows])
        x = mxref.dequantize(c.a[rows], c.sa[rows], c.fmt)
        exact, size = x @ c.down[0].astype(np.float64).T, np.abs(x) @ np.abs(c.down[0].astype(np.float64)).T
        nan = np.isnan(exact)
        assert np.array_equal(np.isnan(host(p)), nan) and nan[3].all() and not nan[:3].any()
        # values below bf16's and sums below fp32's least subnormal may be lost: half a step of 2^-133 each, times down
        tol = (c.K / 8 + 66) * U * size + 2.0 ** -134 * np.abs(c.down[0].astype(np.float64)).sum(1) + c.K * 2.0 ** -149
        close(p[torch.from_numpy(~nan[:, 0]).cuda()], exact[~nan[:, 0]], tol[~nan[:, 0]])


def test_the_layers_gradients_against_differences():
    """The adapted layer's four gradients: a direction's difference of the loss in 64 bits against the library's.
    The loss is linear in x, and in each adapter's parts, so differences are exact but for their own rounding."""
    M, K, N, rank, adapters = 150, 256, 384, 16, 3
    c = Case(M, K, N, mx.E4M3, rank, adapters, "runs")
    g, sg = codes(M, N, mx.E5M2, 8)
    w = mxref.dequantize(c.b, c.sb, mx.E2M1)
    wt, swt = mxref.quantize(np.ascontiguousarray(w.T), mx.E2M1, mx.RULE_CEIL)
    w = mxref.dequantize(wt, swt, mx.E2M1).T  # the weight that the data gradient's product holds
    gv, x = mxref.dequantize(g, sg, mx.E5M2), mxref.dequantize(c.a, c.sa, mx.E4M3)
    g_d, sg_d = dev(g), dev(sg)
    _, p = c.product()
    dx, u = mx.mxfp4_adapted_gemm(g_d, sg_d, mx.E5M2, dev(wt), dev(swt), c.up_d.transpose(1, 2).contiguous(),
                                  c.down_d.transpose(1, 2).contiguous(), c.ids_d, c.alpha_d)
    d_down = mx.adapter_grad_mx(u, c.a_d, c.sa_d, mx.E4M3, c.ids_d, adapters)
    d_up = mx.adapter_grad_mx(p, g_d, sg_d, mx.E5M2, c.ids_d, adapters, transposed=True)

    def loss(x, down, up, parts=np.multiply):
        total = parts(x @ w.T, gv).sum()
        for n in range(adapters):
            rows = c.own(n)
            total += parts(float(c.alpha[n]) * (x[rows] @ down[n].T) @ up[n].T, gv[rows]).sum()
        return total
    rng = np.random.default_rng(1)
    down, up = c.down.astype(np.float64), c.up.astype(np.float64)
    vx, vd, vu = rng.normal(0, 1, x.shape), rng.normal(0, 1, down.shape), rng.normal(0, 1, up.shape)
    # errors of the gradients, relative to the absolute sizes along the direction: 2^-12 of the shared product's
    # for dx, and for all the additions' (K / 8, rank, rows: below 200 u) and u's and p's (K / 8 + 66, N / 8 + 66)
    size = {"x": np.abs(gv) @ np.abs(w), "d": 0, "u": 0}
    for got, v, num, bound in (
            (dx, vx, loss(x + vx, down, up) - loss(x, down, up), 2.0 ** -11),
            (d_down, vd, loss(x, down + vd, up) - loss(x, down, up), 400 * U),
            (d_up, vu, loss(x, down, up + vu) - loss(x, down, up), 400 * U)):
        if got is dx:
            along = (size["x"] * np.abs(v)).sum()
            for n in range(adapters):
                rows = c.own(n)
                along += (np.abs(c.alpha[n] * gv[rows]) @ np.abs(up[n]) @ np.abs(down[n]) * np.abs(v[rows])).sum()
        else:
            along = 0.0
            for n in range(adapters):
                rows, f = c.own(n), float(c.alpha[n])
                if got is d_down:
                    along += (f * np.abs(x[rows]) @ np.abs(v[n]).T @ np.abs(up[n]).T * np.abs(gv[rows])).sum()
                else:
                    along += (f * np.abs(x[rows]) @ np.abs(down[n]).T @ np.abs(v[n]).T * np.abs(gv[rows])).sum()
        assert abs((host(got).astype(np.float64) * v).sum() - num) <= bound * along


def test_graph_replays_other_streams_and_two_calls_at_once():
    c = Case(300, 512, 640, mx.E4M3, 16, 4, "runs")

    def step(stream=None):
        y, p = c.product(stream=stream, out_dtype=torch.bfloat16)
        return y, p, c.project(stream=stream), mx.adapter_grad_mx(p, c.a_d, c.sa_d, c.fmt, c.ids_d, 4, stream=stream)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, here = step(side), step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b, w in zip(got, here, want):
        assert torch.equal(a, w) and torch.equal(b, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        c.ids_d.copy_(torch.from_numpy(some_ids(300, 4, "mixed", 20 + k)))
        c.up_d.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([t.clone() for t in out], step()):
            assert torch.equal(a, b)


def test_two_gradients_at_once():
    """Calls on two streams have workspaces of their own."""
    M, C = 8192, 512
    z, sz = codes(M, C, mx.E4M3, 1)
    z_d, sz_d, ids = dev(z), dev(sz), torch.zeros(M, dtype=torch.int32, device="cuda")
    ps = [torch.randn(M, 16, device="cuda") for _ in range(2)]
    assert mx.mx_adapter_grad_workspace(M, C, 16, 1) > 0
    want = [mx.adapter_grad_mx(p, z_d, sz_d, mx.E4M3, ids, 1) for p in ps]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = [mx.adapter_grad_mx(ps[0], z_d, sz_d, mx.E4M3, ids, 1), mx.adapter_grad_mx(ps[1], z_d, sz_d, mx.E4M3, ids, 1, stream=side)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_unaligned_ids_and_outputs_untouched_around():
    """ids four bytes off 16, out a view of a wider buffer: what lies around it stays."""
    for M in (3, 300):
        c = Case(M, 256, 50, mx.E4M3, 8, 3, "mixed")
        wide = torch.zeros(M + 1, dtype=torch.int32, device="cuda")
        wide[1:] = c.ids_d
        want, p = c.product()
        buf = torch.full((M, 64), 7.0, device="cuda")
        got, p2 = mx.mxfp4_adapted_gemm(c.a_d, c.sa_d, c.fmt, c.b_d, c.sb_d, c.down_d, c.up_d, wide[1:], c.alpha_d, out=buf[:, :50])
        assert got.data_ptr() == buf.data_ptr() and torch.equal(buf[:, :50], want) and torch.equal(p2, p)
        assert (buf[:, 50:] == 7.0).all()


def test_past_four_gib():
    """The last of 40000 adapters, 5.2 GB from the first; rows whose p lies past 4 GiB; codes past 4 GiB in the gradient."""
    adapters, rank, K, N = 40000, 64, 1024, 1024
    c = Case(5, K, N, mx.E4M3, rank, 1, "one", alpha=False)
    down = torch.zeros((adapters, rank, K), dtype=torch.bfloat16, device="cuda")
    up = torch.zeros((adapters, N, rank), dtype=torch.bfloat16, device="cuda")
    down[-1], up[-1] = c.down_d[0], c.up_d[0]
    ids = torch.full((5,), adapters - 1, dtype=torch.int32, device="cuda")
    want = c.product()
    got = mx.mxfp4_adapted_gemm(c.a_d, c.sa_d, c.fmt, c.b_d, c.sb_d, down, up, ids)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del down, up
    M = (1 << 24) + 4096
    c = Case(64, 128, 32, mx.E4M3, rank, 2, "one", alpha=False)
    a = torch.zeros((M, 512), dtype=torch.uint8, device="cuda")[:, :128]  # rows 512 bytes apart: 8 GiB
    s = torch.zeros((M, 4), dtype=torch.uint8, device="cuda")
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    a[-64:], s[-64:], ids[-64:] = c.a_d, c.sa_d, 1
    y, p = mx.mxfp4_adapted_gemm(a, s, c.fmt, c.b_d, c.sb_d, c.down_d, c.up_d, ids, out_dtype=torch.bfloat16)
    exact, tol = c.exact_p()
    close(p[-64:], exact, tol)
    assert not p[:-64].any()
    exact, tol = c.exact_c()
    close(y[-64:], exact, tol + 2.0 ** -8 * (np.abs(exact) + tol))
    assert not y[:-64].any()
    grad = mx.adapter_grad_mx(p, a, s, c.fmt, ids, 2)
    few = mx.adapter_grad_mx(p[-64:].contiguous(), c.a_d, c.sa_d, c.fmt, c.ids_d, 2)
    p64, x = np.abs(host(p[-64:])).astype(np.float64), np.abs(mxref.dequantize(c.a, c.sa, c.fmt))
    close(grad[1], host(few[1]).astype(np.float64), 2 * (64 + 16) * U * (p64.T @ x))
    assert not grad[0].any()
