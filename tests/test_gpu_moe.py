"""Mixture-of-experts layers on the GPU against the fp64 oracle.

Bounds (u = 2^-24, ub = 2^-8: half a step of fp32, of bf16):

* ids: those of the fp64 logits, exactly (both sums carry 64 bits; equal logits
  come from small integers, whose sums are exact).
* weights: the logits' difference rounds to fp32 once, exp, the sum of n terms,
  the quotient and the scale follow: (|l - l_0| + n + 10) 2 u relative.
* H: the gated product's fp32 errors (act_bounds of its test, its rounding to
  bf16 taken off), and 2^-16 for its two parts (each rounds to half a step of
  2^-8 of what it holds).
* y: the errors of H and of the F-term sums through |W2| and the weights, their
  sum over the choices, and ub for the store.
"""

import numpy as np
import pytest
import torch

import oracle
from layout_aware_gemm_amd import tgemm
from parity_util import dev
from test_gpu_ffn import BF, U32, UB, Guarded, act_bounds, f64, replay, rows, within

pytestmark = pytest.mark.gpu

F32 = torch.float32


def stack(E, R, K, seed, std, pad=0, off=0, gap=0):
    """bf16 [E, R, K] with padded rows, experts ``gap`` elements further apart."""
    ld, size = K + pad, R * (K + pad) + gap
    buf = rows(1, E * size + off + 16, seed, std)[0]
    return torch.as_strided(buf, (E, R, K), (size, ld, 1), off)


def layer(M, K, F, E, seed=1, pad=0, off=0, gap=0, router=BF):
    x = rows(M, K, seed, ld=K + pad, off=off)
    if M > 2:
        x[M // 2] = 0.0                    # every expert ties
    r = rows(E, K, seed + 1, 1.5 / np.sqrt(K), ld=K + pad, off=off).to(router)
    w1 = stack(E, 2 * F, K, seed + 2, 1 / np.sqrt(K), pad, off, gap)
    w2 = stack(E, K, F, seed + 3, 1 / np.sqrt(F), pad, off, gap)
    return x, r, w1, w2


def check_routing(ids, p, x, r, top, renorm=True, scale=1.0):
    want, q, logits = oracle.block.route(f64(x), f64(r).T, top, renorm, scale)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), want)
    l = np.take_along_axis(logits, want, axis=1)
    n = top if renorm else r.shape[0]
    within(p, q, np.abs(q) * (np.abs(l - l[:, :1]) + n + 10) * 2.02 * U32)


def check_layer(y, x, ids, p, w1, w2, act):
    """y for the routing (ids, p) that the GPU used."""
    X, P, I = f64(x), f64(p), ids.cpu().numpy()
    M, top = I.shape
    E, K, F = w2.shape
    H, EH = np.zeros((M, top, F)), np.zeros((M, top, F))
    out, err = np.zeros((M, K)), np.zeros((M, K))
    for e in range(E):
        m, j = np.where(I == e)
        if m.size == 0:
            continue
        W1, W2 = f64(w1[e].contiguous()), f64(w2[e].contiguous())
        gu, size = X[m] @ W1.T, np.abs(X[m]) @ np.abs(W1).T
        eg = K * 1.01 * U32 * size
        h, eh = act_bounds(gu, eg[:, :F], eg[:, F:], act)
        e = (eh - 1.01 * UB * np.abs(h)) / (1 + 1.01 * UB)
        eh = e + 2.0 ** -16 * (np.abs(h) + e) + 1e-38
        q = P[m, j][:, None]
        np.add.at(out, m, q * (h @ W2.T))
        np.add.at(err, m, np.abs(q) * (eh * 1.01 + (F + 2 * top + 12) * 1.01 * U32 * np.abs(h))
                  @ np.abs(W2).T)
    within(y, out, err * 1.01 + UB * (np.abs(out) + err))


# (tokens at a time 8, 16 and 64; experts fewer and more than choices; more
# choices of one expert than tokens at a time; two passes; K and F off the
# vectors; weights past the cache)
CASES = [(1, 64, 64, 4, 2), (1, 2048, 96, 64, 8), (1, 1, 1, 1, 1), (3, 40, 33, 5, 5),
         (5, 1000, 333, 10, 3), (8, 72, 100, 1, 1), (9, 512, 160, 8, 2), (13, 264, 72, 8, 2),
         (16, 136, 65, 3, 3), (17, 520, 128, 4, 2), (33, 72, 1000, 30, 1), (64, 256, 96, 128, 8),
         (64, 72, 40, 2, 1), (64, 136, 200, 4, 4), (64, 64, 64, 1, 1), (65, 48, 16, 6, 2),
         (130, 200, 24, 9, 4), (2, 8200, 64, 3, 2), (40, 64, 16, 1024, 16), (3, 31, 7, 300, 2),
         (4, 2048, 1024, 8, 4), (64, 520, 24, 70, 8), (20, 33, 2049, 2, 2), (8, 2049, 513, 20, 6),
         (7, 2048, 2048, 9, 1), (33, 200, 136, 33, 3)]


@pytest.mark.parametrize("M,K,F,E,top", CASES)
@pytest.mark.parametrize("act,router,renorm", [("silu", BF, True), ("gelu_tanh", F32, False)])
def test_moe(M, K, F, E, top, act, router, renorm):
    print(f"moe {M}x{K}x{F} {top} of {E} {act} {router}", flush=True)
    x, r, w1, w2 = layer(M, K, F, E, router=router)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    scale = 1.0 if renorm else 2.5
    y, ids, p = tgemm.moe(x, r.t(), u, d, top, act, renorm, scale, routing=True)
    check_routing(ids, p, x, r, top, renorm, scale)
    check_layer(y, x, ids, p, w1, w2, act)
    # the same bits again, and from the routing as the caller's
    assert torch.equal(tgemm.moe(x, r.t(), u, d, top, act, renorm, scale), y)
    assert torch.equal(tgemm.moe_experts(x, ids, p, u, d, act), y)


@pytest.mark.parametrize("pad,off,gap", [(8, 8, 64), (3, 5, 7), (0, 1, 0), (8, 0, 3)])
@pytest.mark.parametrize("M,K,F,E,top", [(1, 64, 32, 4, 2), (7, 129, 65, 5, 2), (30, 200, 40, 3, 2)])
def test_strides(M, K, F, E, top, pad, off, gap):
    """Rows, experts and bases of any stride and alignment."""
    x, r, w1, w2 = layer(M, K, F, E, 1, pad, off, gap)
    y, ids, p = tgemm.moe(x, r.t(), w1.transpose(1, 2), w2.transpose(1, 2), top, routing=True)
    check_routing(ids, p, x, r, top)
    check_layer(y, x, ids, p, w1, w2, "silu")


def test_tokens_are_independent():
    """A token's row does not depend on the batch it comes in, as far as the
    same kernel computes it."""
    x, r, w1, w2 = layer(13, 264, 72, 8)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    y, ids, p = tgemm.moe(x, r.t(), u, d, 2, routing=True)
    order = torch.tensor([12, 3, 7, 0, 5, 9, 1, 2, 4, 6, 8, 10, 11], device=dev())
    y2, ids2, p2 = tgemm.moe(x[order].contiguous(), r.t(), u, d, 2, routing=True)
    assert torch.equal(ids2, ids[order]) and torch.equal(p2, p[order]) and torch.equal(y2, y[order])
    x3 = x.view(1, 13, 264)
    y3, ids3, _ = tgemm.moe(x3, r.t(), u, d, 2, routing=True)
    assert ids3.shape == (1, 13, 2) and torch.equal(y3[0], y)


def test_ties_and_infinite_logits():
    """Small integers: equal logits are equal exactly.  NaN and infinite logits
    choose valid experts and spoil their own token only."""
    K, F, E, top = 16, 8, 9, 4
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-1, 2, (40, K), generator=g).to(BF).to(dev())
    r = torch.randint(-1, 2, (E, K), generator=g).to(BF).to(dev())
    r[5] = r[2]
    _, _, w1, w2 = layer(40, K, F, E)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    y, ids, p = tgemm.moe(x, r.t(), u, d, top, routing=True)
    check_routing(ids, p, x, r, top)
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = x.clone()
        z[3, 2] = bad
        y2, ids2, p2 = tgemm.moe(z, r.t(), u, d, top, routing=True)
        keep = [i for i in range(40) if i != 3]
        assert torch.equal(y2[keep], y[keep]) and torch.equal(ids2[keep], ids[keep])
        i3 = ids2[3].tolist()
        assert len(set(i3)) == top and all(0 <= e < E for e in i3)
        assert torch.isnan(y2[3]).any()


@pytest.mark.parametrize("M,E,K", [(6, 40, 72), (30, 4, 72), (6, 40, 2056), (5, 4, 2049)])
def test_routing_of_the_callers(M, E, K):
    """Experts listed twice by a token, out of range, negative, none at all;
    weights of either sign and zero."""
    F, top = 40, 5
    x, _, w1, w2 = layer(M, K, F, E)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(0, E, (M, top), generator=g, dtype=torch.int32).to(dev())
    p = torch.randn(M, top, generator=g).to(dev())
    ids[0] = torch.tensor([1, 1, 1, 2, 1])
    ids[1] = torch.tensor([-1, E, 2, 2 ** 31 - 1, -2 ** 31])
    ids[2] = -1
    ids[3] = ids[0]
    p[4, 1] = 0.0
    y = tgemm.moe_experts(x, ids, p, u, d)
    check_layer(y, x, ids, p, w1, w2, "silu")
    assert bool((y[2] == 0).all())
    assert torch.equal(tgemm.moe_experts(x, ids, p, u, d), y)
    assert bool((tgemm.moe_experts(x, torch.full_like(ids, -1), p, u, d) == 0).all())
    # every choice the same expert: more columns than tokens
    one = torch.full_like(ids, E - 1)
    check_layer(tgemm.moe_experts(x, one, p, u, d), x, one, p, w1, w2, "silu")


@pytest.mark.parametrize("M,K,F,E,top", [(8, 264, 520, 5, 11), (7, 72, 2100, 3, 13),
                                         (2, 33, 40, 2, 16), (20, 264, 72, 5, 11),
                                         (8, 2056, 520, 5, 11), (7, 2049, 72, 300, 16),
                                         (8, 2048, 40, 6, 16), (1, 2048, 200, 3, 7)])
def test_experts_listed_again(M, K, F, E, top):
    """Every token lists its experts more than once, with weights of their own:
    the same bits every time."""
    x, _, w1, w2 = layer(M, K, F, E, seed=30)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, E, (M, top), generator=g, dtype=torch.int32).to(dev())
    p = torch.randn(M, top, generator=g).to(dev())
    y = tgemm.moe_experts(x, ids, p, u, d)
    check_layer(y, x, ids, p, w1, w2, "silu")
    for _ in range(8):
        assert torch.equal(tgemm.moe_experts(x, ids, p, u, d), y)
    one = ids[:, :1].expand(M, top).contiguous()
    check_layer(tgemm.moe_experts(x, one, p, u, d), x, one, p, w1, w2, "silu")


@pytest.mark.parametrize("M,K,F,E,top", [(1, 64, 64, 4, 2), (5, 33, 17, 10, 3), (64, 72, 40, 6, 2),
                                         (70, 40, 9, 100, 16), (1, 1, 1, 1, 1)])
@pytest.mark.parametrize("routed", [0, 1])
def test_stays_inside(M, K, F, E, top, routed):
    print(f"moe guarded {M}x{K}x{F} {top} of {E}", flush=True)
    x, r, w1, w2 = layer(M, K, F, E)
    need = tgemm.lib().tgemm_moe_workspace_bytes(M, K, F, E, top, routed)
    ws, Y, ids, p = Guarded(need), Guarded(2 * M * K), Guarded(4 * M * top), Guarded(4 * M * top)
    if not routed:
        at = Guarded.PAD
        ids.buf[at: at + 4 * M * top].view(torch.int32).copy_(
            torch.randint(-1, E + 1, (M * top,), generator=torch.Generator().manual_seed(3),
                          dtype=torch.int32))
        p.buf[at: at + 4 * M * top].view(F32).fill_(0.5)
    args = (M, K, F, E, top, x.data_ptr(), K, r.data_ptr() if routed else None, K, 0, 1, 1.0,
            ids.ptr(), p.ptr(), w1.data_ptr(), K, 2 * F * K, w2.data_ptr(), F, F * K, 0, Y.ptr(), K)
    run, stream = tgemm.lib().tgemm_run_moe, torch.cuda.current_stream().cuda_stream
    assert run(*args, ws.ptr(), need - 1, stream) == tgemm.TGEMM_ERR_WORKSPACE_LIMIT
    assert run(*args, ws.ptr() + 8, need, stream) == tgemm.TGEMM_ERR_INVALID_ARG
    assert run(*args, ws.ptr(), need, stream) == 0
    torch.cuda.synchronize()
    assert all(b.intact() for b in (ws, Y, ids, p))
    # the library's own workspace gives the same
    at = Guarded.PAD
    y = Y.buf[at: at + 2 * M * K].view(BF).clone()
    assert run(*args, None, -1, stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(Y.buf[at: at + 2 * M * K].view(BF), y)


@pytest.mark.parametrize("M,K,F,E,top", [(1, 256, 96, 16, 2), (20, 264, 72, 8, 2)])
def test_replays(M, K, F, E, top):
    """Captured, with other tokens (and so other experts) at each replay."""
    x, r, w1, w2 = layer(M, K, F, E)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    replay(lambda: tgemm.moe(x, r.t(), u, d, top, routing=True), lambda: x.mul_(-0.5))


def test_two_graphs_at_once():
    """Two captured layers replayed on two streams do not share memory."""
    x, r, w1, w2 = layer(20, 264, 72, 8)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    xs = [x, (x * 2).contiguous()]
    want = [tgemm.moe(v, r.t(), u, d, 2) for v in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for v in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tgemm.moe(v, r.t(), u, d, 2))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))


def test_streams():
    x, r, w1, w2 = layer(20, 264, 72, 8)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    want = tgemm.moe(x, r.t(), u, d, 2, routing=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream, 0):
        got = tgemm.moe(x, r.t(), u, d, 2, routing=True, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_far_experts():
    """Experts more than 2^32 bytes apart."""
    K, F, E = 64, 32, 3
    x, r, w1, w2 = layer(5, K, F, E)
    gap = 1_200_000_000
    far = torch.empty(2 * gap + 3 * F * K + 64, dtype=BF, device=dev())
    f1 = torch.as_strided(far, (E, 2 * F, K), (gap, K, 1))
    f2 = torch.as_strided(far, (E, K, F), (gap, F, 1), 2 * F * K)
    f1.copy_(w1)
    f2.copy_(w2)
    want = tgemm.moe(x, r.t(), w1.transpose(1, 2), w2.transpose(1, 2), 2)
    assert torch.equal(tgemm.moe(x, r.t(), f1.transpose(1, 2), f2.transpose(1, 2), 2), want)
