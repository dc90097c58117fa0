"""The feed-forward operators where their other tests do not reach: the
gradient's large tiles in every layout, what its error is made of, and the
statuses of the calls.

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
from test_gpu_ffn import BF, U32, UB, f64, gen, within

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
