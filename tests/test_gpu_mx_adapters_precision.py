"""What of p reaches the adapted product where C is bf16: the shared weight is zero, so that C is up p alone.

All 24 bits of it: rank + 8 additions in fp32, U of the sizes each (those of zeros are exact), and bf16's half step."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
import mxref
from test_gpu_mx_adapters import PRODUCT, U, Case, close

pytestmark = pytest.mark.gpu
# 128 x 128 tiles with two and with four buffers, 256 x 256 ones, with a tail of quadrants; few rows.  The projection row
# by row, in tiles, in runs.
SHAPES = [(300, 128, 2100), (300, 1536, 2100), (700, 1536, 2100), (2049, 128, 4100), (4100, 128, 4352), (37, 256, 300)]


def adds(c, y, p, count):
    """y against up p in 64 bits, p as it came out, `count` of whose products are not zero."""
    p64 = p.cpu().numpy().astype(np.float64)
    exact, tol = np.zeros(y.shape), np.zeros(y.shape)
    for n in range(c.adapters):
        rows, u = c.own(n), c.up[n].astype(np.float64)
        exact[rows] = p64[rows] @ u.T
        tol[rows] = (count + 8) * U * (np.abs(p64[rows]) @ np.abs(u).T)
    close(y, exact, tol + 2.0 ** -8 * (np.abs(exact) + tol))


@pytest.mark.parametrize("M,K,N,rank,adapters,order", [s for s in PRODUCT if s[0] * s[2] < 3e6])
def test_what_the_adapter_adds_in_bf16(M, K, N, rank, adapters, order):
    c = Case(M, K, N, mx.E4M3, rank, adapters, order, seed=5)
    c.b[:], c.sb[:] = 0, 127
    c.put()
    y, p = c.product(out_dtype=torch.bfloat16)
    adds(c, y, p, rank)


@pytest.mark.parametrize("rank", [8, 16, 24, 64, 136])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_what_is_left_when_ranks_cancel(M, K, N, rank):
    """Four pairs of ranks whose first 16 bits are the same and cancel: 2^-17 to 2^-15 of p is all that is left.  p is put
    together from eight bits each of three columns, whose scales are 1, 2^-8 and 2^-16."""
    c = Case(M, K, N, mx.E4M3, rank, 2, "mixed", alpha=False)
    rng = np.random.default_rng(rank + M)
    c.b[:], c.sb[:] = 0, 127
    c.a[:], c.sa[:] = 0, 127
    c.a[:, [0, 32, 64]] = 0x38  # 1
    c.sa[:, 1], c.sa[:, 2] = 119, 111
    c.down[:], c.up[:] = 0, 0
    ranks = rng.permutation(rank)[:8]
    for n in range(2):
        for i, j in zip(ranks[0::2], ranks[1::2]):
            c.down[n, [i, j], 0] = 1 + rng.integers(0, 128) / 128
            c.down[n, [i, j], 32] = rng.integers(128, 256) / 128
            c.down[n, i, 64] = rng.integers(224, 256) / 128
            c.up[n, :, i] = 2.0 ** rng.integers(-2, 3)
            c.up[n, :, j] = -c.up[n, :, i]
    c.put()
    y, p = c.product(out_dtype=torch.bfloat16)
    x = mxref.dequantize(c.a, c.sa, c.fmt)
    for n in range(2):
        rows = c.own(n)
        assert np.array_equal(p.cpu().numpy()[rows].astype(np.float64), x[rows] @ c.down[n].astype(np.float64).T)
    adds(c, y, p, 8)
