"""Infinities and NaN in some columns of up, at ranks of one step of 16 and of several: those columns of the adapter's own
rows are not finite, and every other value of C has the bits that it has with zeros there."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
from test_gpu_mx_adapters import Case

pytestmark = pytest.mark.gpu
# few rows (1, 2 and 4 tiles wide), 128 x 128 tiles with two and four buffers, 256 x 256 ones, with a tail of quadrants
SHAPES = [(7, 128, 96), (40, 256, 520), (64, 512, 9000), (300, 256, 2100), (300, 1536, 2100), (2049, 128, 4100),
          (4100, 128, 4352)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rank", [16, 24, 64, 136])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_columns_of_up(M, K, N, rank, dtype):
    c = Case(M, K, N, mx.E4M3, rank, 3, "mixed")
    c.ids[:3] = 2, 1, 0
    rng = np.random.default_rng(rank + N)
    columns = np.unique(np.concatenate([[0, 31, N - 1], rng.integers(0, N, 5)]))
    at = rng.integers(0, rank, len(columns))
    at[0], at[-1] = 0, rank - 1
    c.up[2, columns, at] = 0
    c.put()
    want, want_p = c.product(out_dtype=dtype)
    c.up[2, columns, at] = rng.choice([np.inf, -np.inf, np.nan], len(columns))
    c.put()
    y, p = c.product(out_dtype=dtype)
    assert torch.equal(p, want_p)
    spoilt = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    spoilt[torch.from_numpy(c.own(2)).cuda()[:, None], torch.from_numpy(columns).cuda()[None, :]] = True
    assert torch.equal(~torch.isfinite(y), spoilt)
    assert torch.equal(y[~spoilt], want[~spoilt])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_rows_whose_p_is_not_finite(M, K, N, dtype):
    """An alpha that is not finite, at a rank of several steps: its adapter's rows alone."""
    c = Case(M, K, N, mx.E4M3, 40, 3, "mixed")
    c.ids[:3] = 2, 1, 0
    c.put()
    want, want_p = c.product(out_dtype=dtype)
    for bad in (np.inf, np.nan):
        c.alpha[1] = bad
        c.put()
        y, p = c.product(out_dtype=dtype)
        own = torch.from_numpy(c.ids == 1).cuda()
        assert not torch.isfinite(p[own]).any() and not torch.isfinite(y[own]).any()
        assert torch.equal(p[~own], want_p[~own]) and torch.equal(y[~own], want[~own])
