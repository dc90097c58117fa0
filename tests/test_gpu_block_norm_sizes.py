"""The block norm's gradient for many gate rows and for the most rows."""

import pytest
import torch

from layout_aware_gemm_amd import tgemm
from parity_util import dev
from test_gpu_block_norm import BF, F32, check_backward, inputs, rows
from test_gpu_ffn import U32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("post", [False, True])
def test_gate_per_token(post):
    """Many tokens with a gate each: every row's results are those of the same
    rows in a small call, bit for bit."""
    m, rep, K = 600, 110, 5120
    y, h, w, wp, gate = inputs(m, K, m, post, BF)
    dn, ds = rows(m, K, 8), rows(m, K, 9)

    def both(*ts):
        y, h, gate, dn, ds = ts
        kw = {"post_weight": wp, "gate": gate, "scale": 0.5}
        rstd = tgemm.block_norm(y, h, w, save=True, **kw)[2]
        return tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)

    want = both(y, h, gate, dn, ds)
    got = both(*(t.repeat(rep, 1) for t in (y, h, gate, dn, ds)))
    for i in (0, 1, 4):                       # dresidual, dy, dgate
        assert torch.equal(got[i].view(rep, m, K), want[i].expand(rep, m, K))


# (groups of rows that end inside a workgroup's, more of them than workgroups or
# fewer, one that spans several workgroups)
@pytest.mark.parametrize("M,K,G", [(3003, 72, 1001), (5120, 40, 1024), (2600, 264, 520),
                                   (2055, 33, 685), (1028, 8200, 257), (2052, 40, 513),
                                   (2565, 40, 513), (1536, 40, 511 * 3 + 3), (1030, 40, 5)])
@pytest.mark.parametrize("post", [False, True])
def test_groups_across_workgroups(M, K, G, post):
    print(f"block norm groups {M}x{K} gates {G} post {post}", flush=True)
    args = inputs(M, K, G, post, BF)
    y, h, w, wp, gate = args
    dn, ds = rows(M, K, 8), rows(M, K, 9)
    kw = {"post_weight": wp, "gate": gate, "scale": 0.75}
    rstd = tgemm.block_norm(y, h, w, save=True, **kw)[2]
    got = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)
    check_backward(got, dn, ds, args, 0.75)
    again = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)
    assert all(u is v or torch.equal(u, v) for u, v in zip(got, again))


@pytest.mark.parametrize("post", [False, True])
def test_most_rows(post):
    """2^31 - 1 rows, of which the last 5,000,000 are not zero: their results are
    those of a call of their own (in the columns' sums, n fp32 terms are within
    n U32 of the sum of their sizes)."""
    print(f"block norm 2^31 - 1 rows post {post}", flush=True)
    M, K, n = (1 << 31) - 1, 1, 5_000_000
    y, h, dn = (torch.zeros(M, K, dtype=BF, device=dev()) for _ in range(3))
    for i, t in enumerate((y, h, dn)):
        g = torch.Generator(device=dev()).manual_seed(i)
        t[-n:] = torch.randn(n, K, generator=g, device=dev()).to(BF)
    w = torch.ones(K, dtype=BF, device=dev())
    kw = {"post_weight": w if post else None, "scale": 0.5}
    sy, sh, sdn = (t[-n:].clone() for t in (y, h, dn))
    small = tgemm.block_norm(sy, sh, w, save=True, **kw)[2]
    rstd = torch.full((1 + post, M), 1000.0, dtype=F32, device=dev())   # (1 / sqrt(eps))
    rstd[:, -n:] = small
    want = tgemm.block_norm_backward(sdn, sy, sh, small, w, **kw)
    got = tgemm.block_norm_backward(dn, y, h, rstd, w, **kw)
    for i in (0, 1):                          # dresidual, dy
        assert torch.equal(got[i][-n:], want[i])
        assert not got[i][:1000].any() and not got[i][M // 2: M // 2 + 1000].any()
    p = sy.double() * (small[1, :, None].double() if post else 1.0)
    s = sh.double() + 0.5 * p
    terms = sdn.double() * s * small[0, :, None].double()
    bound = 1.01 * U32 * (n + 8) * terms.abs().sum()
    assert (got[2].double() - terms.sum(dim=0)).abs().item() <= bound.item()
