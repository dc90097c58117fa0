"""The feed-forward operators without a GPU: the oracle's own pins, the
arguments the entry points refuse (checked before any device call), and the
binding's checks."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from layout_aware_gemm_amd import tgemm

OK, INV, UNS = tgemm.TGEMM_OK, tgemm.TGEMM_ERR_INVALID_ARG, tgemm.TGEMM_ERR_UNSUPPORTED
P = 0x1000  # a fake non-NULL address: validation never dereferences pointers


# ---- the oracle --------------------------------------------------------------


def test_codes_are_rounded_quotients():
    """Against exact rational arithmetic (Python's round of a Fraction is to
    nearest, ties to even), ties included: t = T/2 is 63.5."""
    rng = np.random.default_rng(3)
    for _ in range(20):
        h = oracle.bf16_bits_to_f64(rng.integers(0x3e00, 0x4300, 40).astype(np.uint16))
        w = oracle.bf16_bits_to_f64(rng.integers(0x3f00, 0x4000, 40).astype(np.uint16))
        t = h * w * rng.choice([-1.0, 1.0], 40)
        t[:3] = [np.abs(t).max(), np.abs(t).max() / 2, -np.abs(t).max() / 2]
        q, scale = oracle.ffn.quantize_rows(t[None])
        top = Fraction(float(np.abs(t).max()))
        want = [round(Fraction(float(v)) * 127 / top) for v in t]
        assert q[0].tolist() == want
        assert scale[0] == float(np.abs(t).max()) / 127.0
    assert q[0, 1] == 64 and q[0, 2] == -64


def test_special_rows():
    t = np.array([[0.0, 0.0], [1.0, np.nan], [np.inf, 1.0], [-2.0, 1.0]])
    q, scale = oracle.ffn.quantize_rows(t)
    assert q[:3].tolist() == [[0, 0]] * 3 and q[3].tolist() == [-127, 64]
    assert scale[0] == 0 and np.isnan(scale[1:3]).all() and scale[3] == 2 / 127


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_gradient_against_differences(kind):
    """Central differences in fp64: error ~ step^2 |third derivative| / 6
    (below 1e-10 for step 1e-5) plus 1e-16 / step = 1e-11 of rounding."""
    rng = np.random.default_rng(4)
    gu, dh = rng.normal(0, 2, (5, 14)), rng.normal(0, 1, (5, 7))
    got = oracle.ffn.gated_grad(dh, gu, kind)
    step = 1e-5
    for i in range(5):
        for j in range(14):
            e = np.zeros_like(gu)
            e[i, j] = step
            d = (oracle.ffn.gated(gu + e, kind) - oracle.ffn.gated(gu - e, kind)) / (2 * step)
            assert abs(np.sum(d * dh) - got[i, j]) < 1e-8


def test_activations_closed_forms():
    g = np.linspace(-20, 20, 401)
    assert np.allclose(oracle.ffn.act(g, "silu")[0], g / (1 + np.exp(-g)), rtol=1e-12, atol=0)
    z = np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    assert np.allclose(oracle.ffn.act(g, "gelu_tanh")[0], g / 2 * (1 + np.tanh(z)), rtol=1e-12,
                       atol=1e-15)


# ---- refused arguments -------------------------------------------------------


def v_i8(ta="N", tb="T", M=4, N=5, K=32, A=P, lda=None, B=P, ldb=None, sa=P, sb=P, C=P, ldc=None,
         epi=0):
    lda = (K if ta == "N" else M) if lda is None else lda
    ldb = (N if tb == "N" else K) if ldb is None else ldb
    return tgemm.lib().tgemm_validate_i8(ta.encode(), tb.encode(), M, N, K, A, lda, B, ldb, sa, sb,
                                         C, N if ldc is None else ldc, epi)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(epi=1), OK), (dict(ta="T", tb="N"), OK), (dict(K=131071), OK),
    (dict(K=131072), UNS), (dict(M=1 << 31), UNS), (dict(lda=1 << 62), UNS),
    (dict(M=(1 << 31) - 100), UNS), (dict(N=(1 << 31) - 100), UNS),
    (dict(epi=2), INV), (dict(epi=-1), INV), (dict(ta="x"), INV),
    (dict(M=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(lda=31), INV), (dict(ldb=31), INV),
    (dict(ldc=4), INV), (dict(A=None), INV), (dict(B=None), INV), (dict(C=None), INV),
    (dict(sa=None), INV), (dict(sb=None), INV),
])
def test_validate_i8(kw, expect):
    assert v_i8(**kw) == expect


def v_gated(ta="N", tb="T", M=4, F=5, K=32, A=P, lda=None, B=P, ldb=None, act=0, H=P, ldh=None,
            GU=P, ldgu=None, i8=False, sa=P, sb=P):
    lda = (K if ta == "N" else M) if lda is None else lda
    ldb = (2 * F if tb == "N" else K) if ldb is None else ldb
    ldh = F if ldh is None else ldh
    if i8:
        return tgemm.lib().tgemm_validate_gated_i8(ta.encode(), tb.encode(), M, F, K, A, lda, B,
                                                   ldb, sa, sb, act, H, ldh)
    return tgemm.lib().tgemm_validate_gated(ta.encode(), tb.encode(), M, F, K, A, lda, B, ldb, act,
                                            H, ldh, GU, 2 * F if ldgu is None else ldgu)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(act=1), OK), (dict(GU=None), OK), (dict(GU=None, ldgu=0), OK),
    (dict(M=(1 << 31) - 100), UNS), (dict(F=(1 << 30) - 100), UNS),
    (dict(ta="T", tb="N"), OK), (dict(i8=True), OK), (dict(i8=True, K=131071), OK),
    (dict(i8=True, K=131072), UNS), (dict(K=131072), OK), (dict(F=1 << 30), UNS),
    (dict(act=2), INV), (dict(act=-1), INV), (dict(M=0), INV), (dict(F=0), INV), (dict(K=0), INV),
    (dict(ldh=4), INV), (dict(ldgu=9), INV), (dict(tb="N", ldb=9), INV), (dict(lda=31), INV),
    (dict(A=None), INV), (dict(B=None), INV), (dict(H=None), INV), (dict(ldh=1 << 61), UNS),
    (dict(i8=True, sa=None), INV), (dict(i8=True, sb=None), INV), (dict(i8=True, act=7), INV),
])
def test_validate_gated(kw, expect):
    assert v_gated(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(act=1), OK), (dict(M=0), INV), (dict(F=0), INV), (dict(act=3), INV),
    (dict(gut=1), OK), (dict(gut=-1), INV),
    (dict(dh=None), INV), (dict(gu=None), INV), (dict(dgu=None), INV), (dict(lddh=6), INV),
    (dict(ldgu=13), INV), (dict(lddgu=13), INV), (dict(F=1 << 30), UNS), (dict(M=1 << 31), UNS),
])
def test_validate_gated_grad(kw, expect):
    a = dict(M=3, F=7, dh=P, lddh=None, gu=P, ldgu=None, gut=0, act=0, dgu=P, lddgu=None)
    a.update(kw)
    F = a["F"]
    st = tgemm.lib().tgemm_validate_gated_grad(
        a["M"], F, a["dh"], a["lddh"] or F, a["gu"], a["ldgu"] or 2 * F, a["gut"], a["act"],
        a["dgu"],
        a["lddgu"] or 2 * F)
    assert st == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(epi=1), OK), (dict(tb="N"), OK), (dict(ta="T"), OK), (dict(epi=2), INV),
    (dict(gut=1), OK), (dict(gut=3), INV), (dict(act=2), INV), (dict(M=0), INV), (dict(F=0), INV), (dict(K=0), INV), (dict(F=1 << 30), UNS),
    (dict(A=None), INV), (dict(B=None), INV), (dict(dh=None), INV), (dict(gu=None), INV),
    (dict(da=None), INV), (dict(db=None), INV), (dict(lda=10), INV), (dict(ldb=10), INV),
    (dict(lddh=6), INV), (dict(ldgu=13), INV), (dict(ldda=10), INV), (dict(lddb=10), INV),
    (dict(tb="N", lddb=13), INV), (dict(tb="N", lddb=14), OK), (dict(ldda=1 << 62), UNS),
])
def test_validate_gated_backward(kw, expect):
    a = dict(ta="N", tb="T", M=3, F=7, K=11, A=P, lda=None, B=P, ldb=None, dh=P, lddh=None, gu=P,
             ldgu=None, gut=0, act=0, da=P, ldda=None, db=P, lddb=None, epi=0)
    a.update(kw)
    M, F, K = a["M"], a["F"], a["K"]
    ldb = 2 * F if a["tb"] == "N" else K
    st = tgemm.lib().tgemm_validate_gated_backward(
        a["ta"].encode(), a["tb"].encode(), M, F, K, a["A"],
        a["lda"] or (K if a["ta"] == "N" else M), a["B"], a["ldb"] or ldb, a["dh"], a["lddh"] or F,
        a["gu"], a["ldgu"] or 2 * F, a["gut"], a["act"], a["da"], a["ldda"] or K, a["db"], a["lddb"] or ldb,
        a["epi"])
    assert st == expect


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(r=P, s=P), OK), (dict(eps=0.0), OK), (dict(r=P), INV), (dict(s=P), INV),
    (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(x=None), INV), (dict(w=None), INV), (dict(q=None), INV), (dict(scale=None), INV),
    (dict(M=0), INV), (dict(K=0), INV), (dict(ldx=7), INV), (dict(ldq=7), INV),
    (dict(r=P, s=P, ldr=7), INV), (dict(r=P, s=P, lds=7), INV), (dict(M=1 << 31), UNS),
    (dict(ldx=1 << 61), UNS),
])
def test_validate_rms_norm_i8(kw, expect):
    a = dict(x=P, ldx=8, r=None, ldr=8, w=P, eps=1e-6, M=3, K=8, s=None, lds=8, q=P, ldq=8, scale=P)
    a.update(kw)
    st = tgemm.lib().tgemm_validate_rms_norm_i8(
        a["x"], a["ldx"], a["r"], a["ldr"], a["w"], a["eps"], a["M"], a["K"], a["s"], a["lds"],
        a["q"], a["ldq"], a["scale"])
    assert st == expect
    if not {"r", "s", "eps", "w"} & set(kw):
        assert tgemm.lib().tgemm_validate_quantize_i8(a["x"], a["ldx"], a["M"], a["K"], a["q"],
                                                      a["ldq"], a["scale"]) == expect


def test_workspace_queries():
    """Host-only: nothing for operands read in place, room for the copies of
    others and for partial sums, a status for invalid arguments."""
    L, N, T = tgemm.lib(), b"N", b"T"
    assert L.tgemm_i8_workspace_bytes(N, T, 4, 4096, 4096, P, 4096, P, 4096) == 0
    assert L.tgemm_i8_workspace_bytes(N, T, 4, 40, 33, P, 33, P, 33) >= (4 + 40) * 48
    assert L.tgemm_i8_workspace_bytes(N, N, 4, 40, 64, P, 64, P, 40) >= 40 * 64
    assert L.tgemm_i8_workspace_bytes(N, T, 4, 40, 64, P + 1, 64, P, 64) >= 4 * 64
    assert L.tgemm_i8_workspace_bytes(N, T, 128, 128, 8192, P, 8192, P, 8192) == 4 * 4 * 128 * 128
    assert L.tgemm_i8_workspace_bytes(N, T, 0, 40, 64, P, 64, P, 64) == INV
    assert L.tgemm_i8_workspace_bytes(N, T, 4, 40, 1 << 20, P, 1 << 20, P, 1 << 20) == UNS
    assert L.tgemm_gated_i8_workspace_bytes(N, T, 4, 64, 64, P, 64, P, 64) == 0
    assert L.tgemm_gated_i8_workspace_bytes(N, T, 4, 64, 65, P, 65, P, 65) >= (4 + 128) * 80
    assert L.tgemm_gated_workspace_bytes(N, T, 4, 64, 64, P, 64, P, 64) == 0
    assert L.tgemm_gated_workspace_bytes(T, T, 4, 64, 64, P, 4, P, 64) == 4 * 64 * 2
    assert L.tgemm_gated_workspace_bytes(N, T, 4, 64, 64, None, 64, P, 64) == INV
    # dGU padded to whole tiles of rows, and 64 columns
    assert L.tgemm_gated_backward_workspace_bytes(N, T, 4, 40, 64, P, 64, P, 64) >= 256 * 128 * 2
    assert L.tgemm_gated_backward_workspace_bytes(N, N, 4, 40, 64, P, 64, P, 80) >= 4 * 80 * 2
    assert L.tgemm_gated_backward_workspace_bytes(N, T, 4, 0, 64, P, 64, P, 64) == INV


def test_binding_refuses():
    """Shapes, types and devices are checked before the library is called."""
    bf, i8 = torch.bfloat16, torch.int8
    x, w = torch.zeros(3, 8, dtype=bf), torch.ones(8, dtype=bf)
    a, b = torch.zeros(3, 8, dtype=i8), torch.zeros(8, 6, dtype=i8)
    s3, s6 = torch.ones(3), torch.ones(6)
    for bad in (lambda: tgemm.rms_norm_i8(x, w),                      # CPU tensors
                lambda: tgemm.quantize_i8(x),
                lambda: tgemm.matmul_i8(a, b, s3, s6),
                lambda: tgemm.gated_matmul_i8(a, b, s3, s6),
                lambda: tgemm.gated_matmul(x, torch.zeros(8, 6, dtype=bf)),
                lambda: tgemm.rms_norm_i8(x, torch.ones(7, dtype=bf)),
                lambda: tgemm.rms_norm_i8(x, w, out_residual=x),
                lambda: tgemm.rms_norm_i8(x, w, residual=torch.zeros(2, 8, dtype=bf)),
                lambda: tgemm.quantize_i8(x[:, ::2]),
                lambda: tgemm.quantize_i8(x[:1].expand(3, 8)),
                lambda: tgemm.matmul_i8(a, torch.zeros(7, 6, dtype=i8), s3, s6),
                lambda: tgemm.matmul_i8(a, b, s6, s6),
                lambda: tgemm.matmul_i8(a, b, s3, s3),
                lambda: tgemm.gated_matmul_i8(a, torch.zeros(8, 5, dtype=i8), s3, torch.ones(5)),
                lambda: tgemm.gated_matmul(x, torch.zeros(8, 5, dtype=bf)),
                lambda: tgemm.gated_backward(x, x, x, torch.zeros(8, 6, dtype=bf))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tgemm.quantize_i8(x.float()),
                lambda: tgemm.matmul_i8(x, b, s3, s6),
                lambda: tgemm.matmul_i8(a, b, s3, s6, out_dtype=torch.float16),
                lambda: tgemm.gated_matmul(a, b)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        tgemm._act("relu")


def test_grids_past_the_limit_are_refused():
    """Copies and gradient passes too large for one launch: the calls say so
    before anything is enqueued (the queries run the same checks)."""
    L = tgemm.lib()
    N, T, P = tgemm._flag("N"), tgemm._flag("T"), 1 << 20
    big = 1 << 25
    assert L.tgemm_i8_workspace_bytes(N, N, 4, big, 131071, P, 131071, P, big) == UNS
    assert L.tgemm_i8_workspace_bytes(N, T, 4, 1 << 17, 131071, P, 131071, P, 131071) > 0
    assert L.tgemm_gated_workspace_bytes(N, N, 4, big, 131072, P, 131072, P, 2 * big) == UNS
    assert L.tgemm_gated_backward_workspace_bytes(N, T, (1 << 24) + 64, 8, 8, P, 8, P, 8) == UNS
    assert L.tgemm_gated_backward_workspace_bytes(N, T, 1 << 23, 8, 8, P, 8, P, 8) > 0
