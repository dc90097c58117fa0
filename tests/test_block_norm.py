"""The norms around a residual sum without a GPU: the oracle's gradient against
differences, the arguments the entry points refuse, the binding's checks."""

import numpy as np
import pytest
import torch

import oracle
from layout_aware_gemm_amd import tgemm

OK, INV, UNS = tgemm.TGEMM_OK, tgemm.TGEMM_ERR_INVALID_ARG, tgemm.TGEMM_ERR_UNSUPPORTED
P = 0x1000  # a fake non-NULL address: validation never dereferences pointers


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("G", [0, 1, 2, 6])
def test_gradient_against_differences(post, G):
    """Central differences in fp64 (step 1e-5: third derivatives of order 1
    give 1e-10, the rounding 1e-11 per term; a few dozen terms)."""
    rng = np.random.default_rng(6)
    M, K = 6, 7
    a = {"y": rng.normal(0, 1, (M, K)), "h": rng.normal(0, 2, (M, K)), "w": rng.normal(1, 0.2, K),
         "post": rng.normal(1, 0.2, K) if post else None,
         "gate": rng.normal(0.4, 0.2, (G, K)) if G else None}
    dn, ds = rng.normal(0, 1, (M, K)), rng.normal(0, 1, (M, K))
    grads = oracle.block.block_norm_grad(dn, scale=0.5, eps=1e-3, ds=ds, **a)

    def loss():
        n, s, _ = oracle.block.block_norm(scale=0.5, eps=1e-3, **a)
        return np.sum(n * dn) + np.sum(s * ds)

    step = 1e-5
    for name, grad in zip(("h", "y", "w", "post", "gate"), grads):
        arg = a[name]
        if arg is None:
            assert grad is None
            continue
        assert grad.shape == arg.shape
        for i in np.ndindex(arg.shape):
            keep = arg[i]
            arg[i] = keep + step
            up = loss()
            arg[i] = keep - step
            down = loss()
            arg[i] = keep
            assert abs((up - down) / (2 * step) - grad[i]) < 1e-7


def test_group_rows_serve_their_tokens():
    g = np.array([[1.0, 2.0], [3.0, 4.0]])
    assert oracle.block.spread(g, 6).tolist() == [[1, 2]] * 3 + [[3, 4]] * 3


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(st=1), OK), (dict(post=None), OK), (dict(gate=None, ldg=0, G=0), OK),
    (dict(G=3), OK), (dict(G=1), OK), (dict(rstd=None), OK), (dict(eps=0.0), OK),
    (dict(scale=-2.0), OK), (dict(st=2), INV), (dict(st=-1), INV), (dict(G=4), INV),
    (dict(G=0), INV), (dict(G=-1), INV), (dict(G=12), INV), (dict(eps=-1e-6), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(M=0), INV), (dict(K=0), INV), (dict(y=None), INV),
    (dict(h=None), INV), (dict(w=None), INV), (dict(s=None), INV), (dict(n=None), INV),
    (dict(ldy=7), INV), (dict(ldh=7), INV), (dict(lds=7), INV), (dict(ldn=7), INV),
    (dict(ldg=7), INV), (dict(M=1 << 31, G=1), UNS), (dict(ldy=1 << 62), UNS),
    (dict(ldg=1 << 62), UNS),
])
def test_validate(kw, expect):
    a = dict(y=P, ldy=8, h=P, ldh=8, st=0, post=P, gate=P, ldg=8, G=6, scale=0.5, w=P, eps=1e-6,
             M=6, K=8, s=P, lds=8, n=P, ldn=8, rstd=P)
    a.update(kw)
    L = tgemm.lib()
    common = (a["y"], a["ldy"], a["h"], a["ldh"], a["st"], a["post"], a["gate"], a["ldg"], a["G"],
              a["scale"], a["w"])
    assert L.tgemm_validate_block_norm(*common, a["eps"], a["M"], a["K"], a["s"], a["lds"], a["n"],
                                       a["ldn"], a["rstd"]) == expect
    if "eps" not in kw:
        # the same rules for the backward call, with dn for s and dy for n
        st = L.tgemm_validate_block_norm_backward(
            a["s"], a["lds"], None, 0, *common, P, a["M"], a["K"], P, 8, a["n"], a["ldn"], P, P, P)
        assert st == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(ds=P, ldds=8), OK), (dict(ds=P, ldds=7), INV), (dict(rstd=None), INV),
    (dict(dw=None), INV), (dict(dp=None), INV), (dict(dg=None), INV), (dict(dh=None), INV),
    (dict(lddh=7), INV), (dict(post=None, dp=None), OK), (dict(gate=None, dg=None), OK),
])
def test_validate_backward(kw, expect):
    a = dict(ds=None, ldds=0, post=P, gate=P, rstd=P, dh=P, lddh=8, dw=P, dp=P, dg=P)
    a.update(kw)
    st = tgemm.lib().tgemm_validate_block_norm_backward(
        P, 8, a["ds"], a["ldds"], P, 8, P, 8, 0, a["post"], a["gate"], 8, 2, 1.0, P, a["rstd"], 6, 8,
        a["dh"], a["lddh"], P, 8, a["dw"], a["dp"], a["dg"])
    assert st == expect


def test_sizes():
    need = tgemm.lib().tgemm_block_norm_backward_workspace_bytes
    assert need(1, 8, 0, 0) == 4 * 8
    assert need(6, 8, 1, 2) == 6 * 4 * 8 * 4
    assert need(100000, 4096, 1, 1) <= 16 * 512 * 4096
    assert need(1, 16384, 1, 1) > 0 and need(1, 16385, 1, 1) == UNS
    assert need(0, 8, 0, 0) == INV and need(6, 8, 0, 4) == INV and need(6, 8, 0, -1) == INV
    assert need(1 << 31, 8, 0, 0) == UNS
    run = tgemm.lib().tgemm_block_norm   # refused before any device call
    assert run(P, 16385, P, 16385, 0, None, None, 0, 0, 1.0, P, 1e-6, 1, 16385, P, 16385, P, 16385,
               None, None) == UNS
    assert run(P, 16384, P, 16384, 0, None, None, 0, 0, 1.0, P, 1e-6, 1 << 23, 16384, P, 16384, P,
               16384, None, None) == UNS


def test_binding_refuses():
    bf = torch.bfloat16
    y, w = torch.zeros(6, 8, dtype=bf), torch.ones(8, dtype=bf)
    rstd = torch.ones(1, 6)
    for bad in (lambda: tgemm.block_norm(y, y, w),                         # CPU tensors
                lambda: tgemm.block_norm_backward(y, y, y, rstd, w),
                lambda: tgemm.block_norm(y, y[:5], w),
                lambda: tgemm.block_norm(y, y, w[:7]),
                lambda: tgemm.block_norm(y, y, w, post_weight=w[:7]),
                lambda: tgemm.block_norm(y, y, w, gate=w[:7]),
                lambda: tgemm.block_norm(y, y, w, gate=y[:4]),             # 4 does not divide 6
                lambda: tgemm.block_norm(y, y, w, gate=y.view(1, 6, 8)),
                lambda: tgemm.block_norm(y[:, ::2], y[:, ::2], w[:4]),
                lambda: tgemm.block_norm_backward(y[:5], y, y, rstd, w),
                lambda: tgemm.block_norm_backward(y, y, y, rstd, w, ds=y[:5]),
                lambda: tgemm.block_norm_backward(y, y, y, rstd, w, post_weight=w),
                lambda: tgemm.block_norm_backward(y, y, y, rstd.double(), w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tgemm.block_norm(y.float(), y, w),
                lambda: tgemm.block_norm(y, y.half(), w),
                lambda: tgemm.block_norm(y, y, w, gate=w.float()),
                lambda: tgemm.block_norm_backward(y.float(), y, y, rstd, w),
                lambda: tgemm.block_norm_backward(y, y, y, rstd, w, ds=y.float())):
        with pytest.raises(TypeError):
            bad()
