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


@pytest.mark.parametrize("M,N,tiles", [(17, 70, False), (64, 1536, False), (300, 4160, True)])
def test_a_packed_p_is_written_for_the_tiles_alone(M, N, tiles):
    """Rows that the few-row kernel takes leave the packed p's part of the workspace as it was."""
    K, rank = 256, 16
    c = Case(M, K, N, mx.E4M3, rank, 1, "one")
    want, want_p = c.product()
    n = mx.mxfp4_gemm_adapted_workspace(M, N, K, rank)
    assert n == (M + 31) // 32 * 3 * 1024  # no runs of the projection
    work = torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
    y, p = torch.empty((M, (N + 15) // 16 * 16), device="cuda"), torch.empty_like(want_p)
    st = mx.mxfp4_gemm_adapted(M, N, K, c.a_d.data_ptr(), c.a_d.stride(0), c.fmt, c.sa_d.data_ptr(), c.b_d.data_ptr(),
                               c.b_d.stride(0), c.sb_d.data_ptr(), c.ids_d.data_ptr(), 1, rank, c.down_d.data_ptr(), K,
                               rank * K, c.up_d.data_ptr(), rank, N * rank, c.alpha_d.data_ptr(), p.data_ptr(), y.data_ptr(),
                               y.stride(0), mx.F32, work.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(y[:, :N], want) and torch.equal(p, want_p)
    assert bool((work != 0x5A).any()) == tiles
