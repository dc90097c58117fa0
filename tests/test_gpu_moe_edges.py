"""Expert layers on both sides of the sizes where the down product's kernel
changes (32 workgroups of 16 columns per token, up to 8 tokens)."""

import pytest
import torch

from layout_aware_gemm_amd import tgemm
from parity_util import dev
from test_gpu_moe import check_layer, check_routing, layer

pytestmark = pytest.mark.gpu

CASES = [(1, 511, 2), (1, 512, 2), (1, 1000, 8), (2, 1023, 3), (2, 1024, 3), (3, 1535, 2),
         (3, 1536, 4), (5, 2559, 2), (5, 2560, 7), (8, 2048, 2), (8, 4095, 16), (8, 4096, 16),
         (7, 4099, 5), (9, 4096, 2)]


@pytest.mark.parametrize("M,K,top", CASES)
@pytest.mark.parametrize("F,E", [(40, 6), (72, 20)])
def test_down_product(M, K, top, F, E):
    print(f"moe edges {M}x{K}x{F} {top} of {E}", flush=True)
    x, r, w1, w2 = layer(M, K, F, E)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    if top <= E:
        y, ids, p = tgemm.moe(x, r.t(), u, d, top, routing=True)
        check_routing(ids, p, x, r, top)
        check_layer(y, x, ids, p, w1, w2, "silu")
    # experts listed more than once, and outside
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, E + 1, (M, top), generator=g, dtype=torch.int32).to(dev())
    p = torch.randn(M, top, generator=g).to(dev())
    y = tgemm.moe_experts(x, ids, p, u, d)
    check_layer(y, x, ids, p, w1, w2, "silu")
    for _ in range(4):
        assert torch.equal(tgemm.moe_experts(x, ids, p, u, d), y)
