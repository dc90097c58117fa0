"""Linear layers at the edges of the kernels' choice: few rows beside the
widths where the blocks of weight rows change, tiled products whose last round
goes to smaller tiles, and captured calls that copy their operands first."""

import pytest
import torch

from layout_aware_gemm_amd import tgemm
from test_gpu_ffn import BF, replay, rows
from test_gpu_linear import F32, check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 8, 9, 17, 32, 33, 64])
@pytest.mark.parametrize("N", [4096, 4097, 6656, 6657, 8192, 8193])
@pytest.mark.parametrize("K", [40, 33])
def test_few_rows(M, N, K):
    print(f"linear edges {M}x{N}x{K}", flush=True)
    x, w = rows(M, K, M), rows(N, K, N, 1.5 * K ** -0.5)
    b, r = rows(1, N, 7, 0.5)[0], rows(M, N, 8, 2.0)
    y, z = tgemm.linear(x, w.t(), b, "silu", r, save=True)
    check_forward(y, z, x, w.t(), b, r, "silu")


@pytest.mark.parametrize("M,N,K", [(1979, 9280, 72), (1437, 13120, 40), (3834, 9600, 33),
                                   (3399, 9664, 64)])
def test_tails(M, N, K):
    print(f"linear tails {M}x{N}x{K}", flush=True)
    x, w = rows(M, K, M), rows(N, K, N, 1.5 * K ** -0.5)
    b, r = rows(1, N, 7, 0.5)[0], rows(M, N, 8, 2.0)
    y, z = tgemm.linear(x, w.t(), b, "relu", r, save=BF)
    check_forward(y, z, x, w.t(), b, r, "relu")


@pytest.mark.parametrize("M,N,K", [(96, 201, 263), (300, 131, 521), (7, 200, 33)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_captured_copies(M, N, K, layout):
    """Operands off the 16-byte grid or not K-contiguous, copied inside the graph."""
    print(f"linear captured {layout} {M}x{N}x{K}", flush=True)
    x = rows(M, K, 1, off=1) if layout[0] == "N" else rows(K, M, 1, off=1).t()
    w = rows(K, N, 2, 0.1, off=1) if layout[1] == "N" else rows(N, K, 2, 0.1, off=1).t()
    b, dy = rows(1, N, 3)[0], rows(M, N, 5)

    def step():
        y, z = tgemm.linear(x, w, b, "gelu_tanh", save=True)
        return (y, z) + tgemm.linear_backward(dy, x, w, z, "gelu_tanh", bias=True, dw_dtype=F32)

    def change():
        x.mul_(-0.5)
        dy.mul_(2.0)

    y, z, dx, dw, db = step()
    check_forward(y, z, x, w, b, None, "gelu_tanh")
    check_backward(dx, dw, db, dy, x, w, z, "gelu_tanh")
    replay(step, change)
    assert not torch.equal(step()[0], y)
