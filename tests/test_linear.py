"""Linear layers without a GPU: the oracle's gradient against differences, the
arguments the entry points refuse, the binding's checks."""

import numpy as np
import pytest
import torch

import oracle
from layout_aware_gemm_amd import tgemm

OK, INV, UNS = tgemm.TGEMM_OK, tgemm.TGEMM_ERR_INVALID_ARG, tgemm.TGEMM_ERR_UNSUPPORTED
P = 0x1000  # a fake non-NULL address: validation never dereferences pointers


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu_tanh"])
def test_gradient_against_differences(kind):
    """Central differences in fp64, as for the gated product: 1e-10 from the
    third derivative and 1e-11 of rounding per term, a few dozen terms.  (relu:
    no z within a step of its kink.)"""
    rng = np.random.default_rng(5)
    x, w, b = rng.normal(0, 1, (4, 6)), rng.normal(0, 1, (6, 5)), rng.normal(0, 1, 5)
    dy = rng.normal(0, 1, (4, 5))
    z = oracle.block.linear(x, w, b)[1]
    assert np.abs(z).min() > 1e-3
    dx, dw, db, _ = oracle.block.linear_grad(dy, x, w, z, kind)
    step = 1e-5
    for arg, grad in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(arg.shape):
            keep = arg[i]
            arg[i] = keep + step
            up = np.sum(dy * oracle.block.linear(x, w, b, kind)[0])
            arg[i] = keep - step
            down = np.sum(dy * oracle.block.linear(x, w, b, kind)[0])
            arg[i] = keep
            assert abs((up - down) / (2 * step) - grad[i]) < 1e-8


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(epi=1), OK), (dict(act=0), OK), (dict(act=1), OK), (dict(act=3), OK),
    (dict(ta="T"), OK), (dict(tb="N"), OK), (dict(bias=None), OK), (dict(r=None, ldr=0), OK),
    (dict(z=None, ldz=0, zt=9), OK), (dict(zt=1), OK),
    (dict(act=4), INV), (dict(act=-1), INV), (dict(epi=2), INV), (dict(epi=-1), INV),
    (dict(zt=2), INV), (dict(M=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(lda=10), INV),
    (dict(ldb=10), INV), (dict(ldr=6), INV), (dict(ldy=6), INV), (dict(ldz=6), INV),
    (dict(A=None), INV), (dict(B=None), INV), (dict(y=None), INV), (dict(ta="q"), INV),
    (dict(M=1 << 31), UNS), (dict(N=(1 << 31) - 100), UNS), (dict(ldy=1 << 62), UNS),
    (dict(ldr=1 << 62), UNS), (dict(ldz=1 << 62), UNS),
])
def test_validate_linear(kw, expect):
    a = dict(ta="N", tb="T", M=3, N=7, K=11, A=P, lda=None, B=P, ldb=None, bias=P, act=2, r=P,
             ldr=None, y=P, ldy=None, epi=0, z=P, ldz=None, zt=0)
    a.update(kw)
    M, N, K = a["M"], a["N"], a["K"]
    st = tgemm.lib().tgemm_validate_linear(
        a["ta"].encode(), a["tb"].encode(), M, N, K, a["A"],
        a["lda"] or (K if a["ta"] == "N" else M), a["B"], a["ldb"] or (N if a["tb"] == "N" else K),
        a["bias"], a["act"], a["r"], N if a["ldr"] is None else a["ldr"], a["y"],
        N if a["ldy"] is None else a["ldy"], a["epi"], a["z"], N if a["ldz"] is None else a["ldz"],
        a["zt"])
    assert st == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(epi=1), OK), (dict(tb="N"), OK), (dict(ta="T"), OK), (dict(epi=2), INV),
    (dict(zt=1), OK), (dict(zt=3), INV), (dict(act=2, z=None, ldz=0, zt=3), OK),
    (dict(act=4), INV), (dict(act=0, z=None), INV), (dict(M=0), INV), (dict(N=0), INV),
    (dict(K=0), INV), (dict(A=None), INV), (dict(B=None), INV), (dict(dy=None), INV),
    (dict(da=None), INV), (dict(db=None), INV), (dict(dbias=None), OK), (dict(lda=10), INV),
    (dict(lddy=6), INV), (dict(ldz=6), INV), (dict(ldda=10), INV), (dict(lddb=10), INV),
    (dict(tb="N", lddb=6), INV), (dict(tb="N", lddb=7), OK), (dict(ldda=1 << 62), UNS),
    (dict(M=1 << 31), UNS),
])
def test_validate_linear_backward(kw, expect):
    a = dict(ta="N", tb="T", M=3, N=7, K=11, A=P, lda=None, B=P, ldb=None, dy=P, lddy=None, z=P,
             ldz=None, zt=0, act=0, da=P, ldda=None, db=P, lddb=None, epi=0, dbias=P)
    a.update(kw)
    M, N, K = a["M"], a["N"], a["K"]
    ldb = N if a["tb"] == "N" else K
    st = tgemm.lib().tgemm_validate_linear_backward(
        a["ta"].encode(), a["tb"].encode(), M, N, K, a["A"],
        a["lda"] or (K if a["ta"] == "N" else M), a["B"], a["ldb"] or ldb, a["dy"], a["lddy"] or N,
        a["z"], N if a["ldz"] is None else a["ldz"], a["zt"], a["act"], a["da"], a["ldda"] or K,
        a["db"], a["lddb"] or ldb, a["epi"], a["dbias"])
    assert st == expect


def test_workspace_queries():
    L, N, T = tgemm.lib(), b"N", b"T"
    assert L.tgemm_linear_workspace_bytes(N, T, 4, 4096, 4096, P, 4096, P, 4096) == 0
    # few rows of a K-contiguous weight are read at any alignment, others copied
    assert L.tgemm_linear_workspace_bytes(N, T, 4, 40, 33, P, 33, P + 2, 35) == 0
    assert L.tgemm_linear_workspace_bytes(N, T, 70, 40, 33, P, 33, P, 33) >= (70 + 40) * 40 * 2
    assert L.tgemm_linear_workspace_bytes(N, T, 70, 40, 64, P + 2, 64, P, 64) >= 70 * 64 * 2
    assert L.tgemm_linear_workspace_bytes(N, N, 4, 40, 64, P, 64, P, 40) >= 40 * 64 * 2
    assert L.tgemm_linear_workspace_bytes(N, T, 128, 128, 8192, P, 8192, P, 8192) >= 2 * 4 * 128 * 128
    assert L.tgemm_linear_workspace_bytes(N, T, 0, 40, 64, P, 64, P, 64) == INV
    assert L.tgemm_linear_backward_workspace_bytes(N, T, 4, 40, 64, P, 64, P, 64) >= (256 * 64 * 2
                                                                                      + 40 * 4)
    assert L.tgemm_linear_backward_workspace_bytes(N, T, 4, 0, 64, P, 64, P, 64) == INV
    assert L.tgemm_linear_backward_workspace_bytes(N, T, 1 << 30, 8, 8, P, 8, P, 8) == UNS


def test_binding_refuses():
    bf = torch.bfloat16
    x, w, b, y = (torch.zeros(3, 8, dtype=bf), torch.zeros(8, 6, dtype=bf),
                  torch.zeros(6, dtype=bf), torch.zeros(3, 6, dtype=bf))
    for bad in (lambda: tgemm.linear(x, w),                                # CPU tensors
                lambda: tgemm.linear_backward(y, x, w),
                lambda: tgemm.linear(x, w[:7]),
                lambda: tgemm.linear(x, w, bias=b[:5]),
                lambda: tgemm.linear(x, w, bias=b.float()),
                lambda: tgemm.linear(x, w, residual=y[:2]),
                lambda: tgemm.linear(x, w, residual=torch.zeros(6, dtype=bf).expand(3, 6)),
                lambda: tgemm.linear(x, w, act="tanh"),
                lambda: tgemm.linear_backward(y[:2], x, w),
                lambda: tgemm.linear_backward(y, x, w, act="silu"),        # no z
                lambda: tgemm.linear_backward(y, x, w, z=y[:, :5], act="silu")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tgemm.linear(x.float(), w),
                lambda: tgemm.linear(x, w, out_dtype=torch.float16),
                lambda: tgemm.linear(x, w, residual=y, out_dtype=torch.float32),
                lambda: tgemm.linear(x, w, save=torch.float16),
                lambda: tgemm.linear_backward(y.float(), x, w),
                lambda: tgemm.linear_backward(y, x, w, dw_dtype=torch.float16),
                lambda: tgemm.linear_backward(y, x, w, z=y.half(), act="silu")):
        with pytest.raises(TypeError):
            bad()
