"""Workspaces of the adapted product and of the adapters' gradients by their extents (no GPU)."""
import pytest

import mx_block_scaled_x128_amd as mx

# the few-row kernel holds the scales of 32 rows of either operand in 150 KB of LDS: K / 32 bytes a row
LAST = 76800


def packed(M, rank):
    """Three bf16 parts of p for whole strips of 32 rows and 16 ranks."""
    return (M + 31) // 32 * ((rank + 15) // 16) * 3 * 512 * 2


@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("rank", [8, 16, 64])
def test_rows_that_go_to_the_tiles_for_their_length_have_a_packed_p(M, rank):
    N = 4096
    assert mx.mxfp4_gemm_adapted_workspace(M, N, LAST, rank) == mx.mx_adapter_project_workspace(M, LAST, rank)
    for K in (LAST + 128, 81920, 1 << 20, 1 << 23, (1 << 30) - 128):
        assert mx.mxfp4_gemm_adapted_workspace(M, N, K, rank) == packed(M, rank) + mx.mx_adapter_project_workspace(M, K, rank)


def test_more_rows_have_a_packed_p_whichever_kernel_takes_them():
    """The query's device need not be the call's, and from 17 rows on the kernel goes by the device's compute units."""
    for M, K in ((17, 256), (64, 3584), (64, LAST + 128), (300, 256), (8192, 3584)):
        assert mx.mxfp4_gemm_adapted_workspace(M, 1536, K, 16) == packed(M, 16) + mx.mx_adapter_project_workspace(M, K, 16)
    assert mx.mxfp4_gemm_adapted_workspace(16, (1 << 26) + 1, 128, 16) == packed(16, 16)
    assert mx.mxfp4_gemm_adapted_workspace(16, 1 << 26, 128, 16) == 0
    assert mx.mxfp4_gemm_adapted_workspace(300, 0, 256, 16) == mx.mx_adapter_project_workspace(300, 256, 16)


def test_a_call_without_that_workspace_is_refused():
    A, B, P, C, D, U, I, S, T = (0x100000 * i for i in range(1, 10))

    def call(K, work):
        return mx.mxfp4_gemm_adapted(8, 4096, K, A, K, mx.E4M3, S, B, K // 2, T, I, 4, 16, D, K, 16 * K, U, 16, 4096 * 16, None,
                                     P, C, 4096, 0, work, None)
    assert call(LAST + 128, None) == 1 and call(81920, None) == 1  # MXFP8_ERR_NULL
    assert call(81920, A) == 6 and call(81920, C) == 6  # MXFP8_ERR_ALIAS
