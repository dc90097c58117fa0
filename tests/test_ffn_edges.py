"""The feed-forward entry points without a GPU, beside test_ffn: sizes that no
launch can hold are refused by the calls themselves."""

from layout_aware_gemm_amd import tgemm

UNS = tgemm.TGEMM_ERR_UNSUPPORTED
P = 0x1000  # a fake non-NULL address: nothing is enqueued


def test_calls_refuse_grids_past_the_limit():
    """Before anything is enqueued, so no device is needed."""
    L, rows = tgemm.lib(), 1 << 23          # of 512 or 1024 threads: 2^32 and more
    assert L.tgemm_quantize_i8(P, 8192, rows, 8192, P, 8192, P, None) == UNS
    assert L.tgemm_rms_norm_i8(P, 4096, None, 0, P, 1e-6, rows, 4096, None, 0, P, 4096, P,
                               None) == UNS
    # a workgroup per row and 2048 columns
    assert L.tgemm_gated_grad(1 << 24, 8, P, 8, P, 16, 0, 0, P, 16, None) == UNS
    assert L.tgemm_gated_grad(1 << 23, 4096, P, 4096, P, 8192, 0, 0, P, 8192, None) == UNS
