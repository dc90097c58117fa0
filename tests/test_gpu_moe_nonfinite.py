"""Routing by logits that are not finite, in both places where the choice is
made: inside the up product (up to 8 tokens, few logits) and by a kernel of its
own.  NaN counts as largest, the lowest index goes first among equals, and a
token that has such a logit spoils no other.  (Weights: as in test_gpu_moe.py;
exp(-inf) is 0, and an infinite or NaN l_0 makes all of a token's weights NaN.)"""

import numpy as np
import pytest
import torch

from layout_aware_gemm_amd import tgemm
from parity_util import dev
from test_gpu_ffn import BF, U32, f64, within
from test_gpu_moe import F32, check_layer, layer

pytestmark = pytest.mark.gpu


def expected(x, r, top, renorm):
    """(ids, weights) in fp64."""
    with np.errstate(all="ignore"):
        logits = np.stack([(f64(x)[:, None, :] * f64(r)[None, i:i + 1, :]).sum(axis=2)[:, 0]
                           for i in range(r.shape[0])], axis=1)
        ids = np.stack([sorted(range(len(l)), key=lambda e: (not np.isnan(l[e]), -l[e] if not
                                                            np.isnan(l[e]) else 0.0, e))[:top]
                        for l in logits])
        chosen = np.take_along_axis(logits, ids, axis=1)
        e = np.exp(chosen - chosen[:, :1])
        total = (e if renorm else np.exp(logits - chosen[:, :1])).sum(axis=1, keepdims=True)
        return ids, e / total, chosen


@pytest.mark.parametrize("M", [1, 2, 5, 8, 40])
@pytest.mark.parametrize("E,top", [(9, 4), (9, 9), (120, 8)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("router", [BF, F32])
def test_choice(M, E, top, renorm, router):
    """Infinite and NaN values in a token's x, or in one expert's router row."""
    print(f"routing {M} tokens {top} of {E} {renorm} {router}", flush=True)
    K, F, bad_token = 16, 8, M // 2
    g = torch.Generator().manual_seed(M + E)
    x = torch.randint(-2, 3, (M, K), generator=g).to(BF).to(dev())
    x[:, 3] = torch.where(torch.arange(M, device=dev()) % 2 == 0, 1.0, -1.0).to(BF)
    r = torch.randint(-1, 2, (E, K), generator=g).to(router).to(dev())
    _, _, w1, w2 = layer(M, K, F, E)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    base = tgemm.moe(x, r.t(), u, d, top, renormalize=renorm, routing=True)

    def check(z, q):
        y, ids, p = tgemm.moe(z, q.t(), u, d, top, renormalize=renorm, routing=True)
        want, weights, l = expected(z, q, top, renorm)
        assert np.array_equal(ids.cpu().numpy(), want)
        good = np.isfinite(weights).all(axis=1)
        assert np.array_equal(np.isfinite(f64(p)).all(axis=1), good)
        rows = np.nonzero(good)[0]
        if rows.size:
            # (a weight of exp(-inf) is 0 exactly)
            far = np.where(np.isfinite(l), l, l[:, :1])[rows]
            far = np.abs(far - far[:, :1])
            n = top if renorm else E
            within(f64(p)[rows], weights[rows], weights[rows] * (far + n + 10) * 2.02 * U32)
            t = torch.as_tensor(rows, device=dev())
            check_layer(y[t], z[t], ids[t], p[t], w1, w2, "silu")
        for m in set(range(M)) - set(rows.tolist()):
            assert torch.isnan(p[m]).all() and torch.isnan(y[m]).all()
        again = tgemm.moe(z, q.t(), u, d, top, renormalize=renorm, routing=True)
        assert torch.equal(again[1], ids) and torch.equal(again[0][good], y[good])
        return y, ids, p

    check(x, r)
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = x.clone()
        z[bad_token, 2] = bad
        got = check(z, r)
        keep = [m for m in range(M) if m != bad_token]
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, base))
        # a router row: the logit is infinite with x's sign, one expert of all
        q = r.clone()
        q[E // 2, 3] = bad
        check(x, q)
    # all logits of a token -inf or NaN, zeros of either sign
    z = x.clone()
    z[bad_token] = 0.0
    z[bad_token, ::2] = -0.0
    check(z, r)
