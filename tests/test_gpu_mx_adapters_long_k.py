"""The adapted product where K decides between the few-row kernel and the tiles: that kernel holds its rows' scales in
LDS, 32 rows' up to K = 76800 or, in the form of 32 x 64, 51200.  Tolerances as in test_gpu_mx_adapters."""
import numpy as np
import pytest
import torch

import mx_block_scaled_x128_amd as mx
from test_gpu_mx_adapters import Case, close

pytestmark = pytest.mark.gpu


# rows 1 to 16; 17 to 64 with few and with many columns (the 32 x 64 form from 256 workgroups of 32 x 32 on)
@pytest.mark.parametrize("M,N,K", [(M, 70, K) for M in (1, 8, 16, 40, 64) for K in (76800, 76928)]
                         + [(33, 4160, 51200), (33, 4160, 51328)])
def test_lengths_on_both_sides_of_lds(M, N, K):
    fmt, rank = (mx.E2M1, 24) if M % 16 else (mx.E4M3, 16)
    c = Case(M, K, N, fmt, rank, 3, "mixed" if M > 1 else "one")
    y, p = c.product()
    exact, tol = c.exact_p()
    close(p, exact, tol)
    exact, tol = c.exact_c()
    close(y, exact, tol)
    half, p16 = c.product(out_dtype=torch.bfloat16)
    assert torch.equal(p16, p) and torch.equal(p, c.project())
    close(half, exact, tol + 2.0 ** -8 * (np.abs(exact) + tol))
    none = torch.from_numpy((c.ids < 0) | (c.ids >= 3)).cuda()
    assert torch.equal(y[none], c.base()[none]) and torch.equal(half[none], c.base(out_dtype=torch.bfloat16)[none])
