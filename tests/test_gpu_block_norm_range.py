"""The block norms' gradient over the range that their forward supports: rows
whose squares leave fp32 on either side, by value against the fp64 oracle, under
the bounds of the ordinary rows (test_gpu_block_norm.py).

What those bounds count holds for normalised terms: rs enters once through s rs
inside the reduced sum, once in its factor and once where that meets s rs again
(3 er), the roundings of s rs and y ry are among the K + 6 and 8 units of the
sums.  Below 2^-126 fp32 has fewer bits; no compared value of a case is
between that and the comparison's floor of 1e-35."""

import pytest
import torch

import test_gpu_block_norm as plain
from layout_aware_gemm_amd import tgemm
from test_gpu_block_norm import BF, F32, check_backward, check_forward, inputs, rows

pytestmark = pytest.mark.gpu


def scaled(t, exponents):
    """Row i times 2^exponents[i]."""
    e = torch.tensor(exponents, dtype=torch.float64, device=t.device)
    return (t.double() * torch.exp2(e)[:, None]).to(t.dtype)


def step(args, dn, ds, scale, eps):
    y, h, w, wp, gate = args
    kw = {"post_weight": wp, "gate": gate, "scale": scale}
    n, s, rstd = tgemm.block_norm(y, h, w, eps=eps, save=True, **kw)
    check_forward(n, s, args, scale)
    got = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)
    check_backward(got, dn, ds, args, scale)
    again = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)
    assert all(u is v or torch.equal(u, v) for u, v in zip(got, again))


# exponents of y's and of the residual's rows
LARGE = [(0, 0), (80, 0), (0, 80), (64, 64), (100, 100), (80, -40), (-40, 80), (62, 76)]


@pytest.mark.parametrize("K", [5, 264, 2049, 8200, 9001])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("G", [0, 2])
@pytest.mark.parametrize("res", [BF, F32])
def test_large_rows(K, post, G, res):
    """Large y, large residual, both, and one far above the other."""
    print(f"block norm large rows K {K} post {post} gates {G} {res}", flush=True)
    M = len(LARGE)
    y, h, w, wp, gate = inputs(M, K, G, post, res)
    y, h = scaled(y, [a for a, _ in LARGE]), scaled(h, [b for _, b in LARGE])
    dn = rows(M, K, 8)
    for ds in (rows(M, K, 9).to(res), None):
        step((y, h, w, wp, gate), dn, ds, 0.5, plain.EPS)


@pytest.mark.parametrize("K", [264, 9001])
@pytest.mark.parametrize("res", [BF, F32])
def test_gradient_along_a_large_row(K, res):
    """ds along y: what the projection has to take away is as large as the rest."""
    M = 4
    y, h, w, wp, gate = inputs(M, K, 1, True, res)
    ds = y.clone().to(res)
    y = scaled(y, [80, 70, 100, 0])
    step((y, h, w, wp, gate), rows(M, K, 8, 2.0 ** -6), ds, 0.5, plain.EPS)


@pytest.mark.parametrize("K", [264, 2049, 9001])
@pytest.mark.parametrize("res", [BF, F32])
def test_small_rows_without_eps(K, res, monkeypatch):
    """eps = 0: rows whose squares underflow keep their direction."""
    monkeypatch.setattr(plain, "EPS", 0.0)
    M = 4
    dn, ds = rows(M, K, 8), rows(M, K, 9).to(res)
    # a small block's output, normed onto an ordinary stream
    y, h, w, wp, gate = inputs(M, K, 2, True, res)
    step((scaled(y, [0, -40, -80, -100]), h, w, wp, gate), dn, ds, 0.5, 0.0)
    # both small, without a post-norm
    y, h, w, wp, gate = inputs(M, K, 2, False, res)
    tiny = [0, -40, -70, -90]
    step((scaled(y, tiny), scaled(h, tiny), w, wp, gate), dn, ds, 0.5, 0.0)
    # a small stream and a small share of an ordinary block's output
    y, h, w, wp, gate = inputs(M, K, 2, True, res)
    step((y, scaled(h, [-80] * M), w, wp, gate), dn, ds, 2.0 ** -80, 0.0)
