"""Which kernel a call's shape takes, and what the binding asks for it, on the host."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from weight_only_int4_stats_b200 import build
    build.build()
    import weight_only_int4_stats_b200 as awq
    return awq.lib()


@pytest.mark.parametrize("N,K", [(14336, 4096), (4096, 14336), (37, 384)])
@pytest.mark.parametrize("bits", [4, 3])
def test_up_to_8_fp16_rows_with_inv_s_are_held_in_two_parts(L, N, K, bits):
    """The workspace of 1 to 8 rows holds two fp16 rows of each (the kernel that rounds nothing
    before the output); 9 rows need no such copy of fp16 activations."""
    def need(M):
        return L.awq_gemm_epilogue_workspace_size(M, N, K, bits, 1, 0)
    for M in range(1, 9):
        assert M * 4 * K <= need(M)
    splits = (need(9) + 256) // (9 * N * 4)   # partial sums of slices of K alone
    assert need(9) <= splits * 9 * N * 4 + 255
    for E in (2, 128):
        for T in (1, 4 * E, 4 * E + 1, 8 * E):
            assert L.awq_gemm_grouped_workspace_size(T, E, N, K, bits, 1, 0) >= T * 4 * K
        assert L.awq_gemm_grouped_workspace_size(8 * E + 1, E, N, K, bits, 1, 0) == 0
