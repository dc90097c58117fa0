"""Sizes that the block norm's gradient takes, without a GPU."""

import pytest

from layout_aware_gemm_amd import tgemm

UNS = tgemm.TGEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("M,K,gates", [
    (65536, 5120, 65536),            # a gate per token
    (300000, 4096, 100000),          # groups of three, some across workgroups
    (1 << 22, 16384, 1 << 22), (1 << 30, 512, 1 << 29), ((1 << 31) - 1, 1, (1 << 31) - 1),
    (1 << 20, 16384, 1), (1 << 20, 16384, 0)])
def test_any_number_of_gates(M, K, gates):
    """What the forward takes the backward takes too: the number of gate rows is
    not limited, and does not change the workspace (sums of at most 512 groups
    of rows)."""
    need = tgemm.lib().tgemm_block_norm_backward_workspace_bytes
    for post in (0, 1):
        rows = 1 + post + (2 if gates else 0)
        n = need(M, K, post, gates)
        assert 0 < n <= 512 * rows * K * 4
        assert n == need(M, K, post, min(gates, 1))
    assert need(M, 16385, 0, gates) == UNS
