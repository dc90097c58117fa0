"""The feed-forward operators where their other tests do not reach: the
gradient's large tiles in every layout, what its error is made of, the
statuses of the calls, gates far below zero, block sizes of few rows, and rows
of the smallest values.

Bounds as in test_gpu_ffn (u32 = 2^-24, ub = 2^-8).
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import workloads
from layout_aware_gemm_amd import tgemm
from parity_util import dev
from test_gpu_ffn import (BF, U32, UB, act_bounds, check_quant, codes, f64, gen, scales,
                          within)

pytestmark = pytest.mark.gpu


def framed(n, k, seed, std):
    """bf16 [n, k] on the GPU between NaNs: what lies behind each row."""
    buf = torch.full((n, (k + 15) // 8 * 8), float("nan"), dtype=BF)
    buf[:, :k] = workloads.randn_bf16((n, k), std, gen(seed))
    return buf.to(dev())[:, :k]


def operands(M, F, K, layout):
    x = framed(M, K, 1, 1.0) if layout[0] == "N" else framed(K, M, 1, 1.0).t()
    w = framed(K, 2 * F, 2, K ** -0.5) if layout[1] == "N" else framed(2 * F, K, 2, K ** -0.5).t()
    return x, w, framed(M, F, 3, 1.0)


def rounded_dgu(dh, gu, kind):
    """dGU in bf16 as the elementwise gradient leaves it."""
    M, F = dh.shape
    out = torch.empty(M, 2 * F, dtype=BF, device=dev())
    tgemm._call("tgemm_gated_grad", dev(), M, F, dh.data_ptr(), dh.stride(0), gu.data_ptr(), 2 * F,
                tgemm.EPI_STORE_F32, tgemm._act(kind), out.data_ptr(), 2 * F)
    return out


def product(got, p, ep, q, n, out_u):
    """got against p @ q for |p error| <= ep and an fp32 sum of n terms."""
    r, m = p @ q, (ep * 1.01 + n * 1.01 * U32 * np.abs(p)) @ np.abs(q)
    within(got, r, m * 1.01 + out_u * (np.abs(r) + m))


# 256x256 tiles from 60 k-steps of them per compute unit on: 15360 in all.
# These have 15487 (3 x 17 tiles of 157 and 40 x 17 of 11), 15807 and 16065.
@pytest.mark.parametrize("M,F,K", [(707, 5003, 4101), (4099, 5000, 700), (65, 20100, 4100)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN", "TT"])
def test_gradient_large_tiles(M, F, K, layout):
    """Both gradient products by value on the large tiles: dB stored [K][2F]
    is the product with its operands exchanged."""
    print(f"gradient {layout} {M}x{F}x{K}", flush=True)
    x, w, dh = operands(M, F, K, layout)
    gu = tgemm.gated_matmul(x, w, save=True)[1]
    dx, dw = tgemm.gated_backward(dh, gu, x, w, dw_dtype=torch.float32)
    G, D, X, W = f64(gu), f64(dh), f64(x), f64(w)
    dgu = oracle.ffn.gated_grad(D, G, "silu")
    # dgu: ub of itself, and fp32 terms below 2^-18 of |dh| (|u| + |act|):
    # |s| < 30 here, so (3 |s| + 12) 2 u32 (1 + |g|) < 2^-18 (1 + |g|)
    big = np.abs(D) * (1 + np.abs(G[:, :F])) * (np.abs(G[:, F:]) + np.abs(G[:, :F]))
    eg = UB * np.abs(dgu) + 2.0 ** -18 * np.concatenate([big, big], 1)
    product(dx, dgu, eg, W.T, 2 * F, UB)
    product(dw.t(), dgu.T, eg.T, X, M, U32)
    dx2, dw2 = tgemm.gated_backward(dh, gu, x, w)
    assert torch.equal(dx, dx2) and torch.equal(dw.to(BF), dw2)


@pytest.mark.parametrize("M,F,K,layout", [(333, 1000, 520, "NT"), (130, 70, 72, "TN"),
                                          (707, 5003, 4101, "NT")])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gradient_is_the_product_of_the_rounded_dgu(M, F, K, layout, kind):
    """dX and dW against exact products of the bf16 dGU: beside that one
    rounding there are the fp32 sums and the outputs' own rounding, no more."""
    print(f"rounded dgu {layout} {M}x{F}x{K} {kind}", flush=True)
    x, w, dh = operands(M, F, K, layout)
    gu = tgemm.gated_matmul(x, w, act=kind, save=True)[1]
    dx, dw = tgemm.gated_backward(dh, gu, x, w, act=kind, dw_dtype=torch.float32)
    dgu = f64(rounded_dgu(dh, gu, kind))
    product(dx, dgu, 0 * dgu, f64(w).T, 2 * F, UB)
    product(dw.t(), dgu.T, 0 * dgu.T, f64(x), M, U32)


# ---- statuses ----------------------------------------------------------------


def test_errors_of_other_calls_are_left_alone():
    """A HIP error that the caller's thread left behind is neither reported
    by the feed-forward calls nor taken from the caller."""
    M, F, K = 70, 40, 72
    x, w, dh = framed(M, K, 1, 1.0), framed(2 * F, K, 2, 0.2), framed(M, F, 3, 1.0)
    (q, s), (qw, sw) = tgemm.quantize_i8(x), tgemm.quantize_i8(w)
    h, gu = tgemm.gated_matmul(x, w.t(), save=True)
    dx, dw = tgemm.gated_backward(dh, gu, x, w.t())
    c = tgemm.matmul_i8(q, qw.t(), s, sw)
    h8 = tgemm.gated_matmul_i8(q, qw.t(), s, sw)
    out = [torch.zeros_like(t) for t in (q, s, h, gu, dx, dw.t(), c, h8)]
    Q, S, H, GU, DX, DW, C, H8 = (t.data_ptr() for t in out)
    n, t = tgemm._flag("N"), tgemm._flag("T")
    prod = (n, t, M, F, K, x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0))
    i8 = (K, q.data_ptr(), K, qw.data_ptr(), K, s.data_ptr(), sw.data_ptr())
    L = tgemm.lib()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    assert ws.numel() >= max(L.tgemm_gated_backward_workspace_bytes(*prod),
                             L.tgemm_i8_workspace_bytes(n, t, M, 2 * F, *i8[:-2]))
    work = (ws.data_ptr(), ws.numel())
    calls = [
        ("tgemm_quantize_i8", (x.data_ptr(), x.stride(0), M, K, Q, K, S)),
        ("tgemm_run_gated", prod + (0, H, F, GU, 2 * F) + work),
        ("tgemm_run_gated_backward",
         prod + (dh.data_ptr(), dh.stride(0), gu.data_ptr(), 2 * F, tgemm.EPI_STORE_F32, 0, DX, K,
                 DW, K, tgemm.EPI_STORE_BF16) + work),
        ("tgemm_run_i8", (n, t, M, 2 * F) + i8 + (C, 2 * F, tgemm.EPI_STORE_BF16) + work),
        ("tgemm_run_gated_i8", (n, t, M, F) + i8 + (0, H8, F) + work),
    ]
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    L.hipMalloc.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    got = []
    for name, args in calls:
        assert L.hipMalloc(None, 16) == 1      # hipErrorInvalidValue, left pending
        got.append((name, getattr(L, name)(*args, stream), L.hipGetLastError()))
    torch.cuda.synchronize()
    assert got == [(name, tgemm.TGEMM_OK, 1) for name, _ in calls]
    for i, (o, r) in enumerate(zip(out, (q, s, h, gu, dx, dw.t(), c, h8))):
        assert torch.equal(o, r), i


# ---- gates far below zero ----------------------------------------------------


def far_gates(kind, n):
    """Gates whose sigmoid runs from e^-55 to e^-150, past where 1 / (1 + e^-s)
    leaves fp32; the argument s of the last is -150."""
    lo = 150.0 if kind == "silu" else 12.23  # s(-12.23) = -150
    return -np.linspace(0.37 * lo if kind == "silu" else 0.67 * lo, lo, n)


def relative(s):
    """Of act(g) v in fp32: the exponent's argument (3 roundings of s, one of
    the constant, one of the product: each |s| u32, doubled), exp2 and the
    products; then the store's ub."""
    return ((10 * np.abs(s) + 24) * U32 + UB) * 1.05


def check_far(got, ref, rel):
    assert np.min(np.abs(ref)) > 2.0 ** -120
    within(got, ref, rel * np.abs(ref))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_far_gates_gradient(kind):
    """dgu where dh brings the gate's tail back into range (by 2^127 at most)."""
    F = 333
    g = np.float32(far_gates(kind, F))
    a, d, s = oracle.ffn.act(g.astype(np.float64), kind)
    assert s.min() > -153 and s.max() < -50
    up = np.exp2(np.minimum(127, np.round(-np.log2(np.abs(a)))))
    sign = np.array([[1.0], [-1.0], [1.0]])
    u = 1 + np.arange(3 * F).reshape(3, F) % 7 / 8
    dh = torch.tensor(sign * up, dtype=torch.float32).to(BF).to(dev())
    gu = torch.tensor(np.concatenate([np.tile(g, (3, 1)), u], 1), dtype=torch.float32).to(dev())
    got = f64(rounded_dgu(dh, gu, kind))
    check_far(got[:, :F], sign * up * u * d, relative(s))
    check_far(got[:, F:], sign * up * a, relative(s))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,K", [(9, 64), (100, 64), (70, 4096)])
@pytest.mark.parametrize("op", ["i8", "bf16", "bf16 keep"])
def test_far_gates_products(kind, M, K, op):
    """h for gates in the tail and large u, on the few-row kernel, the tiles
    and the sum of K chunks.  Row m holds one value, so g and u are products
    of two numbers, exact in fp32."""
    print(f"far gates {kind} {op} {M} {K}", flush=True)
    F = 50
    big = 2.0 ** 100
    if op == "i8":
        # g = code * step: the code's column scale carries the step
        code = np.round(np.linspace(45, 127, F) if kind == "silu" else np.linspace(83, 127, F))
        step = np.float32(150 / 127 if kind == "silu" else 12.23 / 127)
        a, b = torch.zeros(M, K, dtype=torch.int8), torch.zeros(2 * F, K, dtype=torch.int8)
        a[:, 3] = 1
        b[:F, 3] = torch.tensor(-code).to(torch.int8)
        b[F:, 3] = torch.arange(1, F + 1)
        sb = torch.cat([torch.full((F,), float(step)), torch.full((F,), big)]).to(dev())
        h = tgemm.gated_matmul_i8(a.to(dev()), b.to(dev()).t(), torch.ones(M, device=dev()), sb,
                                  act=kind)
        g, u = (-code * step).astype(np.float32), np.arange(1, F + 1) * big
    else:
        g = f64(torch.tensor(far_gates(kind, F)).to(BF))
        u = f64(torch.tensor(np.linspace(1, 3, F) * big).to(BF))
        x, w = torch.zeros(M, K, dtype=BF), torch.zeros(2 * F, K, dtype=BF)
        x[:, 3] = 1
        w[:, 3] = torch.tensor(np.concatenate([g, u])).to(BF)
        keep = op == "bf16 keep"
        h = tgemm.gated_matmul(x.to(dev()), w.to(dev()).t(), act=kind, save=keep)
        h = h[0] if keep else h
    act, _, s = oracle.ffn.act(np.asarray(g, np.float64), kind)
    check_far(h, np.tile(act * u, (M, 1)), relative(s))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_far_gates_leave_others_alone(kind):
    """One far gate per 8 columns: the others' bits do not change."""
    M, F = 5, 333
    gu = torch.randn(M, 2 * F, generator=gen(1)) * 3
    dh = workloads.randn_bf16((M, F), 1.0, gen(2)).to(dev())
    far = gu.clone()
    far[:, 5:F:8] = -100.0
    near = torch.ones(2 * F, dtype=torch.bool)
    near[5:F:8] = near[F + 5::8] = False
    a, b = rounded_dgu(dh, gu.to(dev()), kind), rounded_dgu(dh, far.to(dev()), kind)
    assert torch.equal(a[:, near.to(dev())], b[:, near.to(dev())])
    x, w = framed(M, 64, 1, 1.0), framed(2 * F, 64, 2, 0.1)
    w2 = w.clone()
    w2[5:F:8] = 0
    w2[5:F:8, 0] = -200.0
    x[:, 0] = 1
    keep = near[:F].to(dev())
    for rows in (x, x.repeat(40, 1)):
        h = tgemm.gated_matmul(rows, w.t(), act=kind)
        h2 = tgemm.gated_matmul(rows, w2.t(), act=kind)
        assert torch.equal(h[:, keep], h2[:, keep])


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gates_without_a_finite_value(kind):
    """NaN gates make dg, du and h NaN, infinite ones give the limits, and
    their neighbours keep their values."""
    M, F = 3, 40
    gu = torch.randn(M, 2 * F, generator=gen(1))
    dh = workloads.randn_bf16((M, F), 1.0, gen(2)).to(dev())
    want = rounded_dgu(dh, gu.to(dev()), kind)
    gu[1, 7], gu[2, 9] = float("nan"), float("inf")
    got = rounded_dgu(dh, gu.to(dev()), kind)
    bad = torch.zeros(M, 2 * F, dtype=torch.bool, device=dev())
    bad[1, 7] = bad[1, F + 7] = bad[2, 9] = bad[2, F + 9] = True
    assert torch.equal(got[~bad], want[~bad])
    assert torch.isnan(got[1, [7, F + 7]]).all()
    assert got[2, F + 9].item() == float("inf") * np.sign(dh[2, 9].item())
    assert got[2, 9] == (dh[2, 9].float() * gu[2, F + 9].item()).to(BF)
    # forward: one token's NaN in x reaches its own row only
    x, w = framed(70, 64, 1, 1.0), framed(2 * F, 64, 2, 0.1)
    h = tgemm.gated_matmul(x, w.t(), act=kind)
    x[13, 3] = float("nan")
    for m in (70, 20):
        h2 = tgemm.gated_matmul(x[:m], w.t(), act=kind)
        assert torch.isnan(h2[13]).all() and torch.isfinite(h2[:13]).all()
        assert torch.isfinite(h2[14:]).all()
    assert torch.equal(tgemm.gated_matmul(x, w.t(), act=kind)[14:], h[14:])


# ---- few rows ----------------------------------------------------------------


@pytest.mark.parametrize("M", [33, 64])
@pytest.mark.parametrize("N", [4065, 4096, 4097])
def test_few_rows_around_half_the_compute_units(M, N):
    """127.03, 128 and 128.03 blocks of 32 outputs: both block sizes for 33
    to 64 rows."""
    K = 208
    a, w = codes(M, K, 1, full=True), codes(N, K, 2, full=True)
    sa, sb = scales(M, 1), scales(N, 2)
    ref = oracle.ffn.matmul_i8(a.cpu().numpy(), w.t().cpu().numpy(), f64(sa), f64(sb))
    within(tgemm.matmul_i8(a, w.t(), sa, sb, out_dtype=torch.float32), ref,
           np.abs(ref) * 3.01 * U32)
    x, v = framed(M, K, 1, 1.0), framed(2 * N, K, 2, 0.1)
    h, gu = tgemm.gated_matmul(x, v.t(), save=True)
    X, V = f64(x), f64(v).T
    e = K * U32 * 1.01 * (np.abs(X) @ np.abs(V))
    within(gu, X @ V, e)
    within(h, *act_bounds(X @ V, e[:, :N], e[:, N:], "silu"))


# ---- rows of the smallest values ---------------------------------------------


@pytest.mark.parametrize("K", [5, 513, 9000, 40001])
def test_rows_below_the_normal_range(K):
    """Rows of bf16 subnormals (multiples of 2^-133), alone and beside a
    normal value: exact codes, scales to their own rounding."""
    n = torch.randint(-127, 128, (4, K), generator=gen(K)).double()
    n[0, 0], n[1, 0] = 127, 1
    n[1, 1:] = 0
    n[2, 0], n[2, 2] = 64.0, -3
    x = (n * 2.0 ** -133).to(BF)
    x[3, 1] = 2.0 ** -126
    assert torch.equal(x.double()[:3], n[:3] * 2.0 ** -133)
    q, scale = tgemm.quantize_i8(x.to(dev()))
    check_quant(q, scale, *oracle.ffn.quantize_rows(f64(x)))
    # the norm's scale is of order 1 whatever the row's size
    w = torch.ones(K, dtype=BF, device=dev())
    q2, s2 = tgemm.rms_norm_i8(x.to(dev()), w, eps=0.0)
    h = f64(x)
    check_quant(q2, s2, *oracle.ffn.quantize_rows(h, 1 / np.sqrt(np.mean(h * h, 1))))
