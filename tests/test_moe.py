"""Mixture-of-experts layers without a GPU: the oracle against its definition,
the arguments the entry points refuse, the binding's checks."""

import numpy as np
import pytest
import torch

import oracle
from layout_aware_gemm_amd import tgemm

OK, INV, UNS = tgemm.TGEMM_OK, tgemm.TGEMM_ERR_INVALID_ARG, tgemm.TGEMM_ERR_UNSUPPORTED
P = 0x1000  # a fake non-NULL address: validation never dereferences pointers


def test_routing():
    x = np.array([[1.0, 0.0], [0.0, 0.0]])
    r = np.array([[1.0, 3.0, 3.0, 2.0], [9.0, 9.0, 9.0, 9.0]])
    ids, p, _ = oracle.block.route(x, r, 3)
    assert ids.tolist() == [[1, 2, 3], [0, 1, 2]]     # the lowest index of equals first
    e = np.exp([0.0, 0.0, -1.0])
    assert np.allclose(p[0], e / e.sum()) and np.allclose(p[1], 1 / 3)
    q = oracle.block.route(x, r, 3, renormalize=False, scale=2.0)[1]
    assert np.allclose(q[0], 2 * e / (e.sum() + np.exp(-2.0))) and np.allclose(q[1], 0.5)


def test_all_experts_make_a_dense_layer():
    """With every expert chosen the layer is the weighted sum of all of them."""
    rng = np.random.default_rng(8)
    x, w1, w2 = rng.normal(0, 1, (3, 5)), rng.normal(0, 1, (4, 5, 6)), rng.normal(0, 1, (4, 3, 5))
    ids, p, _ = oracle.block.route(x, rng.normal(0, 1, (5, 4)), 4)
    y = oracle.block.experts(x, ids, p, w1, w2)
    want = np.zeros_like(y)
    for e in range(4):
        share = np.sum(np.where(ids == e, p, 0), axis=1, keepdims=True)
        want += share * (oracle.ffn.gated(x @ w1[e], "silu") @ w2[e])
    assert np.allclose(y, want)
    assert np.array_equal(oracle.block.experts(x, np.full_like(ids, -1), p, w1, w2), 0 * y)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(rt=1), OK), (dict(router=None, ldr=0, rt=9), OK), (dict(act=1), OK),
    (dict(top=6), OK), (dict(top=7), INV), (dict(top=0), INV), (dict(M=0), INV), (dict(K=0), INV),
    (dict(F=0), INV), (dict(E=0), INV), (dict(act=2), INV), (dict(act=-1), INV), (dict(rt=2), INV),
    (dict(x=None), INV), (dict(ids=None), INV), (dict(p=None), INV), (dict(w1=None), INV),
    (dict(w2=None), INV), (dict(y=None), INV), (dict(ldx=7), INV), (dict(ldr=7), INV),
    (dict(ld1=7), INV), (dict(ld2=4), INV), (dict(ldy=7), INV), (dict(s1=79), INV),
    (dict(s2=39), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(router=None, scale=float("nan")), OK), (dict(router=None, top=7), OK),
    (dict(E=1, top=1, s1=0, s2=0), OK), (dict(E=1024), OK), (dict(E=1025), UNS),
    (dict(E=64, top=16), OK), (dict(E=64, top=17), UNS), (dict(M=1 << 31), UNS),
    (dict(ld1=1 << 22, s1=1 << 40), UNS), (dict(ld2=1 << 22, s2=1 << 40), UNS),
    (dict(ldx=1 << 22), UNS), (dict(ldx=1 << 22, M=1), OK), (dict(s1=1 << 61), UNS),
    (dict(ldr=1 << 62), UNS),
])
def test_validate(kw, expect):
    a = dict(M=3, K=8, F=5, E=6, top=2, x=P, ldx=8, router=P, ldr=8, rt=0, norm=1, scale=1.0, ids=P,
             p=P, w1=P, ld1=8, s1=80, w2=P, ld2=5, s2=40, act=0, y=P, ldy=8)
    a.update(kw)
    assert tgemm.lib().tgemm_validate_moe(
        a["M"], a["K"], a["F"], a["E"], a["top"], a["x"], a["ldx"], a["router"], a["ldr"], a["rt"],
        a["norm"], a["scale"], a["ids"], a["p"], a["w1"], a["ld1"], a["s1"], a["w2"], a["ld2"],
        a["s2"], a["act"], a["y"], a["ldy"]) == expect


def test_workspace_queries():
    need = tgemm.lib().tgemm_moe_workspace_bytes
    assert need(1, 8, 5, 6, 2, 1) >= 6 * 8 + 2 * 64 * 4
    assert need(64, 2048, 768, 128, 8, 1) >= 64 * 128 * 8 + 64 * 8 * 768 * 4
    assert need(1000, 2048, 768, 128, 8, 1) == need(64, 2048, 768, 128, 8, 1)
    assert need(64, 2048, 768, 128, 8, 0) < need(64, 2048, 768, 128, 8, 1)
    assert need(1, 8, 5, 6, 7, 1) == INV and need(1, 8, 5, 2000, 1, 1) == UNS


def test_binding_refuses():
    bf = torch.bfloat16
    x, r = torch.zeros(3, 8, dtype=bf), torch.zeros(6, 8, dtype=bf)
    w1, w2 = torch.zeros(6, 10, 8, dtype=bf), torch.zeros(6, 8, 5, dtype=bf)
    u, d = w1.transpose(1, 2), w2.transpose(1, 2)
    ids, p = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, 2)
    cpu = [lambda: tgemm.moe(x, r.t(), u, d, 2), lambda: tgemm.moe_experts(x, ids, p, u, d),
           lambda: tgemm.moe_experts(x, ids[:2], p[:2], u, d),
           lambda: tgemm.moe_experts(x, ids, p[:, :1], u, d),
           lambda: tgemm.moe_experts(x, ids[0], p[0], u, d),
           lambda: tgemm.moe_experts(x, ids[:, ::2], p[:, ::2], u, d)]
    for bad in cpu:
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tgemm._experts(w1, "w"), lambda: tgemm._experts(u[0], "w"),
                lambda: tgemm._experts(u[:, :, :0], "w"),
                lambda: tgemm._experts(w1[:, :1].expand(6, 10, 8).transpose(1, 2), "w")):
        with pytest.raises(ValueError):
            bad()
    assert tgemm._experts(u, "w") == (80, 8)
    with pytest.raises(TypeError):
        tgemm._experts(u.float(), "w")
    for bad in (lambda: tgemm.moe_experts(x, ids.long(), p, u, d),
                lambda: tgemm.moe_experts(x, ids, p.double(), u, d)):
        with pytest.raises(TypeError):
            bad()
