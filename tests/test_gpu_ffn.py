"""The feed-forward operators on the GPU against the fp64 oracle.

Bounds (u32 = 2^-24, the half step of fp32; ub = 2^-8, of bf16):

* codes and the stored residual sum: equal, bit for bit.  Scales: one
  rounding of an fp64 value whose own error is of the order 2^-50: u32.
* 8-bit products: the integer sum is exact; its conversion and the two scale
  products round once each, so fp32 outputs are within 3 u32 (1 + u32)^2 <
  3.01 u32 relative, bf16 ones within ub more.
* gates: with |g error| <= eg and |u error| <= eu, h moves by at most
  |act'| eg |u| + |act| eu with |act'| <= 1.13 for both activations (doubled
  where the errors are second order); the fp32 evaluation of act adds, per
  unit, the exponent's argument (3 roundings of s) and exp2, 1 + e, rcp and
  the product (1 ulp each): (3 |s| + 8) 2 u32.  Then ub for the store.
* bf16 products in fp32: K u32 (|a| @ |b|), as for the library's GEMM.
* gradients: dgu within ub of its formula plus fp32 terms; the products sum
  those errors and round once more.
"""

import numpy as np
import pytest
import torch

import oracle
import workloads
from layout_aware_gemm_amd import tgemm
from parity_util import bf16_to_f64, bits, dev

pytestmark = pytest.mark.gpu

U32, UB = 2.0 ** -24, 2.0 ** -8
BF, I8 = torch.bfloat16, torch.int8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(M, K, seed, std=1.0, ld=None, off=0):
    """bf16 [M, K] on the GPU inside a larger buffer: row stride ld, first
    element ``off`` elements past an aligned address."""
    ld = K if ld is None else ld
    buf = workloads.randn_bf16((M * ld + off + 16,), std, gen(seed))
    return torch.as_strided(buf.to(dev()), (M, K), (ld, 1), off)


def codes(M, K, seed, ld=None, off=0, full=False):
    ld = K if ld is None else ld
    n = M * ld + off + 32
    lo = -128 if full else -127
    buf = torch.randint(lo, 128, (n,), generator=gen(seed), dtype=torch.int32).to(I8)
    return torch.as_strided(buf.to(dev()), (M, K), (ld, 1), off)


def scales(n, seed):
    return (torch.rand(n, generator=gen(seed)) * 0.02 + 0.001).to(dev())


def f64(t):
    return bf16_to_f64(t) if t.dtype == BF else t.detach().cpu().numpy().astype(np.float64)


def within(got, ref, bound):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - ref) / (bound + 1e-35))
    assert worst <= 1.0, worst


# ---- rows to 8-bit codes -----------------------------------------------------

ROWS = [(1, 1), (3, 5), (2, 8), (1, 64), (7, 511), (2, 512), (3, 513), (5, 2048), (3, 2049),
        (2, 4096), (2, 5120), (1, 8191), (2, 8200), (2, 13824), (1, 16385), (2, 32768), (2, 32776),
        (1, 70001), (600, 264), (513, 2057), (520, 5000), (515, 8000), (515, 8201), (513, 33001)]


def check_quant(q, scale, ref_q, ref_scale):
    assert np.array_equal(q.cpu().numpy(), ref_q)
    s = scale.cpu().numpy().astype(np.float64)
    nan = np.isnan(ref_scale)
    assert np.array_equal(np.isnan(s), nan)
    assert np.all(np.abs(s - ref_scale)[~nan] <= 1.01 * U32 * ref_scale[~nan] + 2.0 ** -150)


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
def test_quantize(M, K, pad, off):
    print(f"quantize {M}x{K} pad {pad} off {off}", flush=True)
    x = rows(M, K, K + M, ld=K + pad, off=off)
    q, scale = tgemm.quantize_i8(x)
    check_quant(q, scale, *oracle.ffn.quantize_rows(f64(x)))


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("pad,off", [(0, 0), (5, 3)])
def test_rms_norm(M, K, res, pad, off):
    print(f"rms norm {M}x{K} residual {res} pad {pad} off {off}", flush=True)
    x = rows(M, K, K + M, ld=K + pad, off=off)
    r = rows(M, K, K + M + 1, 3.0, ld=K + 2 * pad, off=2 * off) if res else None
    w = (1 + 0.2 * torch.randn(K, generator=gen(K))).to(BF).to(dev())
    out = tgemm.rms_norm_i8(x, w, eps=1e-5, residual=r)
    ref_q, ref_s, ref_h = oracle.ffn.rms_norm_i8(bits(x), bits(w), np.float32(1e-5),
                                                 None if r is None else bits(r))
    check_quant(out[0], out[1], ref_q, ref_s)
    if res:
        assert np.array_equal(bits(out[2]), ref_h)


def test_rms_norm_special_rows():
    """Zeros, NaN, infinity, squares past fp32, products past fp32, tiny
    values, ties (T/2 is 63.5 levels), a single value."""
    K = 600
    x = workloads.randn_bf16((9, K), 1.0, gen(5))
    x[0] = 0
    x[1, 17] = float("nan")
    x[2, 599] = float("-inf")
    x[3] = 2.0 ** 100 * x[3].float()
    x[4, 3] = 2.0 ** 127
    x[5] = (2.0 ** -90 * x[5].float()).to(BF)
    x[6] = 0
    x[6, ::2] = 1.0
    x[6, 1::4] = -0.5
    x[7] = 0
    x[7, 300] = -3.0
    w = torch.ones(K, dtype=BF)
    w[3] = 4.0
    q, scale = tgemm.rms_norm_i8(x.to(dev()), w.to(dev()), eps=0.0 + 1e-30)
    h, t = f64(x), f64(x) * f64(w)
    t[4, 3] = np.inf                        # 2^129 is past fp32
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        ref_q, ref_s = oracle.ffn.quantize_rows(t, 1 / np.sqrt(np.mean(h * h, 1) + np.float32(1e-30)))
    check_quant(q, scale, ref_q, ref_s)
    assert q[6, 1].item() == -64 and q[6, 0].item() == 127
    assert torch.isnan(scale[[1, 2, 4]]).all() and scale[0] == 0


def test_rms_norm_in_place_and_3d():
    """The sum written over the residual; leading dimensions kept."""
    x, r = rows(6, 1000, 1), rows(6, 1000, 2, 2.0)
    w = torch.ones(1000, dtype=BF, device=dev())
    ref = tgemm.rms_norm_i8(x, w, residual=r)
    r2 = r.clone()
    q, s, h = tgemm.rms_norm_i8(x.view(2, 3, 1000), w, residual=r2.view(2, 3, 1000),
                                out_residual=r2.view(2, 3, 1000))
    assert h.data_ptr() == r2.data_ptr() and q.shape == (2, 3, 1000) and s.shape == (2, 3)
    assert torch.equal(r2, ref[2]) and torch.equal(q.view(6, 1000), ref[0])
    assert torch.equal(s.view(6), ref[1])


def test_quantize_leaves_the_rest_alone():
    """Codes in rows of a wider buffer: the bytes between the rows stay."""
    x = rows(5, 77, 3)
    buf = torch.full((5 * 90 + 8,), 99, dtype=I8, device=dev())
    scale = torch.empty(5, device=dev())
    q = torch.as_strided(buf, (5, 77), (90, 1), 1)
    tgemm._call("tgemm_quantize_i8", dev(), x.data_ptr(), 77, 5, 77, q.data_ptr(), 90, scale.data_ptr())
    ref, _ = oracle.ffn.quantize_rows(f64(x))
    assert np.array_equal(q.cpu().numpy(), ref)
    q.fill_(99)
    assert bool((buf == 99).all())


# ---- 8-bit products ----------------------------------------------------------

# (skinny blocks of 16 / 32 / 64 rows, 128- and 256-row tiles, split K, edges)
I8_SHAPES = [(1, 1, 16), (1, 16, 48), (1, 1000, 4096), (1, 300, 13824), (5, 17, 64), (16, 33, 512),
             (17, 130, 1040), (32, 64, 256), (33, 257, 80), (64, 129, 2048), (65, 128, 128),
             (66, 1, 16), (127, 255, 144), (129, 129, 272), (200, 300, 4096), (300, 520, 8208),
             (257, 513, 1008), (768, 640, 4096), (1100, 4000, 192), (2100, 4100, 80),
             (2050, 4200, 400), (520, 32000, 144),  # (256x256 tiles; a tail of smaller ones)
             (100, 20001, 144), (100, 5503, 10256),  # (128x128 tiles, whole and in K chunks)
             (130, 5003, 20496),  # (128x256 tiles in K chunks)
             (5, 6151, 16400),  # (a weight loaded past the cache)
             # few rows: whole and half blocks of weight rows, and wide ones
             (1, 4200, 80), (16, 4200, 80), (30, 5001, 48), (64, 4200, 80), (50, 17001, 48),
             (2300, 7268, 1040), (2300, 8418, 1040), (2300, 9698, 1040)]  # (each size of tail)


def i8_ref(a, b, sa, sb):
    return oracle.ffn.matmul_i8(a.cpu().numpy(), b.cpu().numpy(), f64(sa), f64(sb))


@pytest.mark.parametrize("M,N,K", I8_SHAPES)
@pytest.mark.parametrize("out", [torch.float32, BF])
def test_i8(M, N, K, out):
    print(f"i8 {M}x{N}x{K} {out}", flush=True)
    a, w = codes(M, K, M + K, full=True), codes(N, K, N + K, full=True)
    sa, sb = scales(M, 1), scales(N, 2)
    c = tgemm.matmul_i8(a, w.t(), sa, sb, out_dtype=out)
    ref = i8_ref(a, w.t(), sa, sb)
    within(c, ref, np.abs(ref) * (3.01 * U32 + (1.01 * UB if out == BF else 0)))


@pytest.mark.parametrize("M,N,K", [(1, 70, 33), (3, 65, 129), (20, 100, 500), (70, 130, 31),
                                   (150, 140, 1001), (1, 1, 1), (80, 3, 1)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("pad,off", [(0, 0), (16, 16), (3, 5)])
def test_i8_layouts(M, N, K, layout, pad, off):
    """Lengths, strides and bases off the 16-byte grid, every layout."""
    print(f"i8 {layout} {M}x{N}x{K} pad {pad} off {off}", flush=True)
    a = (codes(M, K, 1, ld=K + pad, off=off) if layout[0] == "N"
         else codes(K, M, 1, ld=M + pad, off=off).t())
    b = (codes(K, N, 2, ld=N + pad, off=off) if layout[1] == "N"
         else codes(N, K, 2, ld=K + pad, off=off).t())
    sa, sb = scales(M, 1), scales(N, 2)
    c = tgemm.matmul_i8(a, b, sa, sb, out_dtype=torch.float32)
    ref = i8_ref(a, b, sa, sb)
    within(c, ref, np.abs(ref) * 3.01 * U32)


@pytest.mark.parametrize("M", [2, 70])
def test_i8_largest_sum(M):
    """K = 131071 codes of -128: sums of 2^31 - 2^14, the largest allowed."""
    K = 131071
    a = torch.full((M, K), -128, dtype=I8, device=dev())
    b = torch.full((3, K), -128, dtype=I8, device=dev())
    one = torch.ones(M, device=dev())
    c = tgemm.matmul_i8(a, b.t(), one, torch.ones(3, device=dev()), out_dtype=torch.float32)
    assert bool((c == float(K * 16384)).all())


def test_i8_nan_scale_and_bounds():
    """A NaN scale (a row the quantiser could not hold) makes its row NaN and
    no other; a wider C keeps what lies between its rows."""
    for M in (5, 80):
        a, w = codes(M, 64, 1), codes(30, 64, 2)
        sa, sb = scales(M, 1), scales(30, 2)
        sa[3] = float("nan")
        C = torch.full((M + 1, 41), 7.0, device=dev())
        tgemm._call("tgemm_run_i8", dev(), tgemm._flag("N"), tgemm._flag("T"), M, 30, 64, a.data_ptr(), 64,
                    w.data_ptr(), 64, sa.data_ptr(), sb.data_ptr(), C.data_ptr(), 41,
                    tgemm.EPI_STORE_F32, None, -1)
        c = C[:M, :30]
        assert torch.isnan(c[3]).all() and torch.isfinite(c[:3]).all()
        assert torch.isfinite(c[4:]).all()
        assert bool((C[:, 30:] == 7).all()) and bool((C[M] == 7).all())


# ---- gated products ----------------------------------------------------------


def act_bounds(gu, eg, eu, kind):
    """h and its bound for errors eg, eu of g, u (module docstring)."""
    F = gu.shape[1] // 2
    g, u = gu[:, :F], gu[:, F:]
    a, d, s = oracle.ffn.act(g, kind)
    h = a * u
    fp32 = (3 * np.abs(s) + 8) * 2 * U32
    # (sigmoid of a large argument is flat: its argument's error counts at
    # most e^-|s| |s|, folded into the same term)
    e = (1.13 * eg * np.abs(u) + (np.abs(a) + 1.13 * eg) * eu + np.abs(h) * fp32)
    return h, UB * (np.abs(h) + e) * 1.01 + e


@pytest.mark.parametrize("M,F,K", [(1, 1, 16), (1, 100, 2048), (1, 1000, 8192), (16, 33, 64),
                                   (17, 16, 80), (40, 31, 272), (64, 129, 512), (65, 64, 128),
                                   (130, 65, 144), (300, 200, 4112), (513, 300, 1040),
                                   (1030, 2100, 96), (3, 20, 33), (90, 70, 65), (24, 12300, 48),
                                   (64, 12289, 144), (2100, 2060, 160), (4096, 2100, 48),
                                   (100, 10001, 144), (100, 2751, 10256), (2300, 3634, 1040),
                                   (2300, 4849, 1040), (130, 2501, 20496),
                                   (3, 3079, 16400), (20, 10250, 4912), (2, 4200, 12000),
                                   (1, 4201, 80), (9, 8300, 80), (30, 4200, 80), (50, 4200, 144),
                                   (7, 7001, 272)])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_i8(M, F, K, kind):
    print(f"gated i8 {M}x{F}x{K} {kind}", flush=True)
    a, w = codes(M, K, M), codes(2 * F, K, F)
    sa = scales(M, 1) / np.sqrt(K)
    sb = scales(2 * F, 2) * 0.5
    h = tgemm.gated_matmul_i8(a, w.t(), sa, sb, act=kind)
    gu = i8_ref(a, w.t(), sa, sb)
    eg = 3.01 * U32 * np.abs(gu)
    within(h, *act_bounds(gu, eg[:, :F], eg[:, F:], kind))


GATED = [(1, 1, 8, "NT", 0), (1, 1000, 2048, "NT", 0), (1, 500, 8192, "NT", 0),
         (7, 33, 40, "NT", 8), (16, 64, 520, "NT", 0), (17, 100, 1000, "NT", 0),
         (64, 31, 136, "NT", 0), (65, 65, 64, "NT", 0), (128, 128, 192, "NT", 0),
         (200, 300, 2056, "NT", 8), (300, 77, 4096, "NT", 0), (520, 300, 520, "NT", 0),
         (1030, 2100, 72, "NT", 0), (5, 9, 7, "NT", 0), (70, 33, 65, "NT", 3),
         (1, 64, 64, "NN", 0), (33, 20, 48, "NN", 0), (130, 150, 200, "TN", 0),
         (100, 64, 136, "TT", 0), (2, 3, 1, "NT", 0), (30, 12300, 40, "NT", 0),
         (2100, 2060, 72, "NT", 0), (4096, 2100, 24, "NT", 0), (100, 10001, 72, "NT", 0),
         (100, 2751, 5128, "NT", 0), (2300, 3634, 520, "NT", 0), (2300, 4849, 520, "NT", 0),
         (130, 2501, 10248, "NT", 0), (3, 3079, 8200, "NT", 0), (20, 10250, 2456, "NT", 0),
         (1, 4201, 40, "NT", 0), (9, 8300, 40, "NT", 0), (30, 4200, 40, "NT", 0),
         (50, 4200, 72, "NT", 0), (7, 7001, 136, "NT", 0)]


@pytest.mark.parametrize("M,F,K,layout,pad", GATED)
@pytest.mark.parametrize("kind,keep", [("silu", torch.float32), ("gelu_tanh", torch.float32),
                                       ("silu", BF)])
def test_gated_and_gradient(M, F, K, layout, pad, kind, keep):
    print(f"gated {layout} {M}x{F}x{K} pad {pad} {kind} {keep}", flush=True)
    x = rows(M, K, M, ld=K + pad) if layout[0] == "N" else rows(K, M, M, ld=M + pad).t()
    std = 1.5 / np.sqrt(K)
    w = (rows(K, 2 * F, F, std, ld=2 * F + pad) if layout[1] == "N"
         else rows(2 * F, K, F, std, ld=K + pad).t())
    h, gu = tgemm.gated_matmul(x, w, act=kind, save=True)
    assert torch.equal(h, tgemm.gated_matmul(x, w, act=kind))
    X, W = f64(x), f64(w)
    ref = X @ W
    e = K * U32 * 1.01 * (np.abs(X) @ np.abs(W))
    within(gu, ref, e)
    within(h, *act_bounds(ref, e[:, :F], e[:, F:], kind))

    dh, gu = rows(M, F, 9, ld=F + pad), gu.to(keep)
    dx, dw = tgemm.gated_backward(dh, gu, x, w, act=kind, dw_dtype=torch.float32)
    G, D = f64(gu), f64(dh)
    dgu = oracle.ffn.gated_grad(D, G, kind)
    # dgu: its rounding, and the fp32 terms of act and act' (the derivative
    # is a sum of two terms; each is within the argument's error)
    g, u = G[:, :F], G[:, F:]
    a, _, s = oracle.ffn.act(g, kind)
    slope = np.abs(g) * (1.0 if kind == "silu" else 1.6 * (1 + 0.135 * g * g))
    ed = (3 * np.abs(s) + 12) * 2 * U32 * (1 + slope)
    ef = np.concatenate([np.abs(D * u) * ed, np.abs(D * a) * (3 * np.abs(s) + 8) * 2 * U32], axis=1)
    eg = UB * (np.abs(dgu) + ef) + ef + 1e-38
    S = 1.01 * U32

    def product(got, p, ep, q, n, out_u):
        r = p @ q
        b = (ep + n * S * (np.abs(p) + ep)) @ np.abs(q)
        within(got, r, b * 1.01 + out_u * (np.abs(r) + b))

    product(dx, dgu, eg, W.T, 2 * F, UB)
    product(dw.t(), dgu.T, eg.T, X, M, U32)
    assert dw.stride() == ((1, K) if layout[1] == "T" else (2 * F, 1)) or 1 in (K, 2 * F)
    dw16 = tgemm.gated_backward(dh, gu, x, w, act=kind)[1]
    product(dw16.t(), dgu.T, eg.T, X, M, UB)


@pytest.mark.parametrize("M,F,K", [(300, 1000, 520), (2000, 33, 72), (70, 5000, 136),
                                   (513, 260, 264), (1, 300, 40), (4099, 31, 8), (255, 129, 1000),
                                   (100, 90, 67), (257, 33, 257), (64, 32, 1),
                                   (700, 5000, 4100), (4099, 5000, 700), (65, 20100, 4100)])
def test_gradient_shapes(M, F, K):
    """The joint launch of both gradient products: K dimensions (2F and M)
    off the 64-element step, split or not, tiles cut in every direction.
    What lies between the stored rows of x, w and dh is NaN."""
    print(f"gradient {M}x{F}x{K}", flush=True)

    def framed(n, k, seed, std):
        buf = torch.full((n, (k + 15) // 8 * 8), float("nan"), dtype=BF)
        buf[:, :k] = workloads.randn_bf16((n, k), std, gen(seed))
        return buf.to(dev())[:, :k]

    x, w, dh = framed(M, K, 1, 1.0), framed(2 * F, K, 2, K ** -0.5), framed(M, F, 3, 1.0)
    gu = tgemm.gated_matmul(x, w.t(), save=True)[1]
    dx, dw = tgemm.gated_backward(dh, gu, x, w.t(), dw_dtype=torch.float32)
    G, D, X, W = f64(gu), f64(dh), f64(x), f64(w)
    dgu = oracle.ffn.gated_grad(D, G, "silu")
    # dgu: ub of itself, and fp32 terms below 2^-18 of |dh| (|u| + |act|)
    # (|s| < 30 here: (3 |s| + 12) 2 u32 (1 + |g|) < 2^-18 (1 + |g|))
    big = np.abs(D) * (1 + np.abs(G[:, :F])) * (np.abs(G[:, F:]) + np.abs(G[:, :F]))
    eg = UB * np.abs(dgu) + 2.0 ** -18 * np.concatenate([big, big], 1)

    def product(got, p, ep, q, n, out_u):
        r, m = p @ q, (ep * 1.01 + n * 1.01 * U32 * np.abs(p)) @ np.abs(q)
        within(got, r, m * 1.01 + out_u * (np.abs(r) + m))

    product(dx, dgu, eg, W, 2 * F, UB)
    product(dw.t(), dgu.T, eg.T, X, M, U32)
    # the same bits again, and with bf16 weights' gradient the rounding of it
    dx2, dw2 = tgemm.gated_backward(dh, gu, x, w.t())
    assert torch.equal(dx, dx2) and torch.equal(dw.to(BF), dw2)


def test_gradient_writes_nothing_else():
    """dA and dB in wider buffers."""
    M, F, K = 130, 70, 72
    x, w, dh = rows(M, K, 1), rows(2 * F, K, 2, 0.1), rows(M, F, 3)
    gu = tgemm.gated_matmul(x, w.t(), save=True)[1]
    dx, dw = tgemm.gated_backward(dh, gu, x, w.t())
    dA = torch.full((M + 1, K + 5), 3.0, dtype=BF, device=dev())
    dB = torch.full((2 * F + 1, K + 9), 4.0, dtype=BF, device=dev())
    tgemm._call("tgemm_run_gated_backward", dev(), tgemm._flag("N"), tgemm._flag("T"), M, F, K,
                x.data_ptr(), K, w.data_ptr(), K, dh.data_ptr(), F, gu.data_ptr(), 2 * F,
                tgemm.EPI_STORE_F32, 0,
                dA.data_ptr(), K + 5, dB.data_ptr(), K + 9, tgemm.EPI_STORE_BF16, None, -1)
    assert torch.equal(dA[:M, :K], dx) and torch.equal(dB[: 2 * F, :K], dw.t())
    assert bool((dA[:, K:] == 3).all()) and bool((dA[M] == 3).all())
    assert bool((dB[:, K:] == 4).all()) and bool((dB[2 * F] == 4).all())


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_grad_values(kind):
    """The elementwise gradient over the whole range of g, saturated ends
    and infinities included, F off the vector width."""
    F = 333
    g = torch.cat([torch.linspace(-30, 30, 300), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 200.0,
                   -200.0, 1e4, -1e4, 3e38, -3e38]), torch.linspace(-3, 3, 23)]).to(BF)
    gu = torch.cat([g.repeat(3, 1), workloads.randn_bf16((3, F), 1.0, gen(1))], 1).to(dev())
    dh = workloads.randn_bf16((3, F), 1.0, gen(2)).to(dev())
    out = torch.full((3, 2 * F + 5), 7.0, dtype=BF, device=dev())
    tgemm._call("tgemm_gated_grad", dev(), 3, F, dh.data_ptr(), F, gu.data_ptr(), 2 * F,
                tgemm.EPI_STORE_BF16, tgemm._act(kind), out.data_ptr(), 2 * F + 5)
    assert bool((out[:, 2 * F:] == 7).all())
    G, D = f64(gu), f64(dh)
    with np.errstate(over="ignore", invalid="ignore"):
        p = 1 / (1 + np.exp(-oracle.ffn.act(np.clip(G[:, :F], -1e4, 1e4), kind)[2]))
        ref = oracle.ffn.gated_grad(D, np.clip(G, -1e4, 1e4), kind)
    # past 1e4 the sigmoid is 0 or 1: act' = p and act = g p
    big = np.abs(G[:, :F]) > 1e4
    ref[:, F:][big] = (D * G[:, :F] * p)[big]
    a, _, s = oracle.ffn.act(np.clip(G[:, :F], -30, 30), kind)
    slope = np.abs(a) + np.abs(np.clip(G[:, :F], -30, 30)) * (1 if kind == "silu" else 1.6 * 122)
    # (terms with |s| past 100 have saturated: their error is the tail e^-100)
    ed = (3 * np.minimum(np.abs(s), 100) + 12) * 2 * U32 * (1 + np.minimum(slope, 40))
    e = np.concatenate([np.abs(D * G[:, F:]) * ed,
                        np.abs(ref[:, F:]) * (3 * np.minimum(np.abs(s), 100) + 8) * 2 * U32], 1)
    got = f64(out[:, : 2 * F])
    # products past the largest bf16 value, (2 - 2^-7) 2^127: infinite, as
    # any rounding of them is
    over = np.abs(ref) > (2 - 2.0 ** -8) * 2.0 ** 127
    assert over.any() and np.array_equal(got[over], np.sign(ref[over]) * np.inf)
    within(np.where(over, 0, got), np.where(over, 0, ref),
           np.where(over, 0, UB * (np.abs(ref) + e) + e + 1e-36))


def test_gated_writes_nothing_else():
    """H and GU in wider buffers, both kernels (few rows, tiles)."""
    for M in (9, 100):
        F, K = 50, 64
        x, w = rows(M, K, 1), rows(2 * F, K, 2, 0.2)
        H = torch.full((M + 1, F + 7), 3.0, dtype=BF, device=dev())
        GU = torch.full((M + 1, 2 * F + 9), 4.0, device=dev())
        tgemm._call("tgemm_run_gated", dev(), tgemm._flag("N"), tgemm._flag("T"), M, F, K, x.data_ptr(), K,
                    w.data_ptr(), K, 0, H.data_ptr(), F + 7, GU.data_ptr(), 2 * F + 9,
                    None, -1)
        h, gu = tgemm.gated_matmul(x, w.t(), save=True)
        assert torch.equal(H[:M, :F], h) and torch.equal(GU[:M, : 2 * F], gu)
        assert bool((H[:, F:] == 3).all()) and bool((H[M] == 3).all())
        assert bool((GU[:, 2 * F:] == 4).all()) and bool((GU[M] == 4).all())


# ---- together, streams, graphs -----------------------------------------------


def block(x, res, wn, q1, s1, q2, s2):
    """Norm, gated projection, quantiser, down projection, as served."""
    q, s, h = tgemm.rms_norm_i8(x, wn, residual=res)
    a = tgemm.gated_matmul_i8(q, q1.t(), s, s1)
    qa, sa = tgemm.quantize_i8(a)
    return tgemm.matmul_i8(qa, q2.t(), sa, s2), h, a


def block_inputs(M, D, F):
    x, res = rows(M, D, 1), rows(M, D, 2, 2.0)
    wn = (1 + 0.1 * torch.randn(D, generator=gen(3))).to(BF).to(dev())
    q1, s1 = tgemm.quantize_i8(rows(2 * F, D, 4, 1 / np.sqrt(D)))
    q2, s2 = tgemm.quantize_i8(rows(D, F, 5, 1 / np.sqrt(F)))
    return x, res, wn, q1, s1, q2, s2


@pytest.mark.parametrize("M,D,F", [(1, 512, 1376), (48, 264, 500), (200, 512, 1376)])
def test_served_block(M, D, F):
    """The run of four operators against the oracle's, each step fed with
    the GPU's own previous output (so a step's bound is its own)."""
    x, res, wn, q1, s1, q2, s2 = block_inputs(M, D, F)
    y, h, a = block(x, res, wn, q1, s1, q2, s2)
    rq, rs, rh = oracle.ffn.rms_norm_i8(bits(x), bits(wn), np.float32(1e-6), bits(res))
    assert np.array_equal(bits(h), rh)
    gu = oracle.ffn.matmul_i8(rq, q1.cpu().numpy().T, rs, f64(s1))
    eg = 4.02 * U32 * np.abs(gu)            # (one rounding more: the scale)
    within(a, *act_bounds(gu, eg[:, :F], eg[:, F:], "silu"))
    aq, asc = oracle.ffn.quantize_rows(f64(a))
    ref = oracle.ffn.matmul_i8(aq, q2.cpu().numpy().T, asc, f64(s2))
    within(y, ref, np.abs(ref) * (4.02 * U32 + 1.01 * UB))


def test_block_on_another_stream():
    """Helpers called under a side stream, and with the stream passed by
    object and by handle, give the default stream's bits."""
    args = block_inputs(80, 256, 300)
    want = block(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = block(*args)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    x, w = rows(90, 72, 1), rows(100, 72, 2, 0.2)
    dh = rows(90, 50, 3)
    h, gu = tgemm.gated_matmul(x, w.t(), save=True)
    dx, dw = tgemm.gated_backward(dh, gu, x, w.t())
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream, 0):
        h2, gu2 = tgemm.gated_matmul(x, w.t(), save=True, stream=s)
        dx2, dw2 = tgemm.gated_backward(dh, gu2, x, w.t(), stream=s)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.skip(reason="aborted on the GPU (memory aperture violation in a replay) while calls under "
                  "capture allocated their workspace inside the graph and the backward's kernel used "
                  "scratch memory; neither is done any more, the cause was not shown")
@pytest.mark.parametrize("M", [4, 100])
def test_graph_replays(M):
    """A captured block and a captured training step (both with K split over
    workgroups and packed operands among their calls), replayed between eager
    calls of the same and with new input values."""
    D, F = 4104, 96                          # K long: split; D % 16 != 0: packed
    args = block_inputs(M, D, F)
    x, w = rows(M, 4096, 1), rows(2 * 40, 4096, 2, 0.02)
    dh = rows(M, 40, 3)

    def calls():
        y, h, a = block(*args)
        hh, gu = tgemm.gated_matmul(x, w.t(), save=True)
        dx, dw = tgemm.gated_backward(dh, gu, x, w.t())
        return y, h, a, hh, gu, dx, dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = calls()
    for rep in range(3):
        args[0].mul_(-0.5)
        x.mul_(-0.5)
        dh.mul_(2.0)
        want = calls()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (o, r) in enumerate(zip(outs, want)):
            assert torch.equal(o, r), (rep, i)


def replay(calls, change):
    """Capture calls(), then replay it three times, each between eager calls
    of the same after change() has altered the inputs."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = calls()
    for rep in range(3):
        change()
        want = calls()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (o, r) in enumerate(zip(outs, want)):
            assert torch.equal(o, r), (rep, i)


@pytest.mark.parametrize("M,D,F", [(3, 512, 1376), (130, 4096, 96)])
def test_served_block_replays(M, D, F):
    """(130 rows, K = 4096: K split over workgroups, the partial sums in a
    workspace of the caller's.)"""
    args = block_inputs(M, D, F)
    replay(lambda: block(*args), lambda: args[0].mul_(-0.5))


@pytest.mark.parametrize("M,F,K", [(96, 200, 264), (300, 130, 520)])
def test_training_step_replays(M, F, K):
    x, w, dh = rows(M, K, 1), rows(2 * F, K, 2, 0.05), rows(M, F, 3)

    def step():
        h, gu = tgemm.gated_matmul(x, w.t(), save=True)
        dx, dw = tgemm.gated_backward(dh, gu, x, w.t())
        return h, gu, dx, dw

    def change():
        x.mul_(-0.5)
        dh.mul_(2.0)

    replay(step, change)


def test_workspace_contract():
    """The library's own workspace is refused under capture, a caller's that
    is too small always; nothing is written by a refused call, and the
    asked-for size is enough."""
    M, N, K = 70, 40, 4096                   # K split: partial sums
    a, w, sa, sb = codes(M, K, 1), codes(N, K, 2), scales(M, 1), scales(N, 2)
    want = tgemm.matmul_i8(a, w.t(), sa, sb)
    C = torch.full((M, N), 7.0, dtype=BF, device=dev())
    prod = (tgemm._flag("N"), tgemm._flag("T"), M, N, K, a.data_ptr(), K, w.data_ptr(), K)
    need = tgemm.lib().tgemm_i8_workspace_bytes(*prod)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    rest = (sa.data_ptr(), sb.data_ptr(), C.data_ptr(), N, tgemm.EPI_STORE_BF16)
    run, limit = tgemm.lib().tgemm_run_i8, tgemm.TGEMM_ERR_WORKSPACE_LIMIT
    s = torch.cuda.current_stream().cuda_stream
    assert run(*prod, *rest, None, 0, s) == limit
    assert run(*prod, *rest, ws.data_ptr(), need - 1, s) == limit
    assert run(*prod, *rest, ws.data_ptr() + 8, need, s) == tgemm.TGEMM_ERR_INVALID_ARG
    g, st = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(g):
        st.append(run(*prod, *rest, None, -1, torch.cuda.current_stream().cuda_stream))
        C.add_(0)
    torch.cuda.synchronize()
    assert st == [limit] and bool((C == 7).all())
    assert run(*prod, *rest, ws.data_ptr(), need, s) == 0 and torch.equal(C, want)
    C.zero_()
    assert run(*prod, *rest, None, -1, s) == 0 and torch.equal(C, want)


class Guarded:
    """Device bytes inside a larger buffer of 0x5A, which must stay so."""

    PAD = 8192

    def __init__(self, nbytes):
        self.n = nbytes
        self.buf = torch.full((nbytes + 2 * self.PAD,), 0x5A, dtype=torch.uint8, device=dev())

    def ptr(self):
        return self.buf.data_ptr() + self.PAD

    def intact(self):
        return (bool((self.buf[: self.PAD] == 0x5A).all())
                and bool((self.buf[self.PAD + self.n:] == 0x5A).all()))


@pytest.mark.parametrize("M,F,K", [(4, 40, 4096), (1, 1, 8), (70, 33, 72), (300, 130, 520),
                                   (3, 500, 40), (257, 129, 65), (700, 5000, 4100)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_backward_stays_inside(M, F, K, layout):
    """Outputs and workspace of exactly the asked-for size, guarded on both
    sides."""
    print(f"backward guarded {layout} {M}x{F}x{K}", flush=True)
    x = rows(M, K, 1) if layout[0] == "N" else rows(K, M, 1)
    w = rows(2 * F, K, 2, 0.1) if layout[1] == "T" else rows(K, 2 * F, 2, 0.1)
    dh, gu = rows(M, F, 3), rows(M, 2 * F, 4)  # (gu in bf16)
    prod = (tgemm._flag(layout[0]), tgemm._flag(layout[1]), M, F, K, x.data_ptr(), x.stride(0),
            w.data_ptr(), w.stride(0))
    need = tgemm.lib().tgemm_gated_backward_workspace_bytes(*prod)
    ws, dA, dB = Guarded(need), Guarded(2 * M * K), Guarded(8 * F * K)
    tgemm._call("tgemm_run_gated_backward", dev(), *prod, dh.data_ptr(), F, gu.data_ptr(), 2 * F,
                tgemm.EPI_STORE_BF16, 0,
                dA.ptr(), K, dB.ptr(), w.shape[1], tgemm.EPI_STORE_F32, ws.ptr(), need)
    torch.cuda.synchronize()
    assert ws.intact() and dA.intact() and dB.intact()


@pytest.mark.parametrize("M,N,K", [(4, 192, 4104), (4, 4104, 96), (1, 1, 1), (17, 33, 47),
                                   (70, 40, 4096), (130, 260, 129), (300, 500, 100)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("gated", [False, True])
def test_i8_stays_inside(M, N, K, layout, gated):
    print(f"i8 guarded {layout} {M}x{N}x{K} gated {gated}", flush=True)
    n = 2 * N if gated else N
    a = codes(M, K, 1) if layout[0] == "N" else codes(K, M, 1)
    b = codes(n, K, 2) if layout[1] == "T" else codes(K, n, 2)
    sa, sb = scales(M, 1), scales(n, 2)
    prod = (tgemm._flag(layout[0]), tgemm._flag(layout[1]), M, N, K, a.data_ptr(), a.stride(0),
            b.data_ptr(), b.stride(0))
    L = tgemm.lib()
    need = (L.tgemm_gated_i8_workspace_bytes if gated else L.tgemm_i8_workspace_bytes)(*prod)
    ws, C = Guarded(need), Guarded(2 * M * N if gated else 4 * M * N)
    if gated:
        tgemm._call("tgemm_run_gated_i8", dev(), *prod, sa.data_ptr(), sb.data_ptr(), 0, C.ptr(), N,
                    ws.ptr(), need)
    else:
        tgemm._call("tgemm_run_i8", dev(), *prod, sa.data_ptr(), sb.data_ptr(), C.ptr(), N,
                    tgemm.EPI_STORE_F32, ws.ptr(), need)
    torch.cuda.synchronize()
    assert ws.intact() and C.intact()


@pytest.mark.parametrize("M,F,K", [(4, 40, 4096), (1, 1, 8), (70, 33, 72), (70, 16, 8192),
                                   (300, 130, 520), (5, 7, 9)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_gated_stays_inside(M, F, K, layout):
    print(f"gated guarded {layout} {M}x{F}x{K}", flush=True)
    x = rows(M, K, 1) if layout[0] == "N" else rows(K, M, 1)
    w = rows(2 * F, K, 2, 0.1) if layout[1] == "T" else rows(K, 2 * F, 2, 0.1)
    prod = (tgemm._flag(layout[0]), tgemm._flag(layout[1]), M, F, K, x.data_ptr(), x.stride(0),
            w.data_ptr(), w.stride(0))
    need = tgemm.lib().tgemm_gated_workspace_bytes(*prod)
    ws, H, GU = Guarded(need), Guarded(2 * M * F), Guarded(8 * M * F)
    tgemm._call("tgemm_run_gated", dev(), *prod, 0, H.ptr(), F, GU.ptr(), 2 * F, ws.ptr(), need)
    torch.cuda.synchronize()
    assert ws.intact() and H.intact() and GU.intact()


@pytest.mark.parametrize("M,K", [(4, 96), (4, 4104), (1, 1), (3, 511), (2, 8201), (1, 40001)])
def test_rows_stay_inside(M, K):
    print(f"rows guarded {M}x{K}", flush=True)
    x, r, w = rows(M, K, 1), rows(M, K, 2), rows(1, K, 3)
    q, s, h = Guarded(M * K), Guarded(4 * M), Guarded(2 * M * K)
    tgemm._call("tgemm_quantize_i8", dev(), x.data_ptr(), K, M, K, q.ptr(), K, s.ptr())
    torch.cuda.synchronize()
    assert q.intact() and s.intact()
    tgemm._call("tgemm_rms_norm_i8", dev(), x.data_ptr(), K, r.data_ptr(), K, w.data_ptr(), 1e-6, M, K,
                h.ptr(), K, q.ptr(), K, s.ptr())
    torch.cuda.synchronize()
    assert q.intact() and s.intact() and h.intact()


def test_two_captured_graphs_do_not_share():
    """Two graphs of split products, replayed at once on two streams."""
    a1, w1 = codes(70, 8192, 1), codes(64, 8192, 2)
    a2, w2 = codes(90, 8192, 3), codes(64, 8192, 4)
    s1, s2, sw = scales(70, 1), scales(90, 2), scales(64, 3)
    r1, r2 = tgemm.matmul_i8(a1, w1.t(), s1, sw), tgemm.matmul_i8(a2, w2.t(), s2, sw)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = tgemm.matmul_i8(a1, w1.t(), s1, sw)
    with torch.cuda.graph(g2):
        o2 = tgemm.matmul_i8(a2, w2.t(), s2, sw)
    t1, t2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        o1.zero_()
        o2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(t1):
            g1.replay()
        with torch.cuda.stream(t2):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, r1) and torch.equal(o2, r2)


def test_far_offsets():
    """Row offsets past 2^32 bytes (8-bit and bf16 operands, outputs)."""
    M, K, ld = 70, 64, 70_000_000            # 4.9e9 elements of stride
    buf = torch.zeros((M - 1) * ld + K, dtype=I8, device=dev())
    a = torch.as_strided(buf, (M, K), (ld, 1))
    src = codes(M, K, 1)
    a.copy_(src)
    w, sa, sb = codes(40, K, 2), scales(M, 1), scales(40, 2)
    want = tgemm.matmul_i8(src, w.t(), sa, sb)
    assert torch.equal(tgemm.matmul_i8(a, w.t(), sa, sb), want)
    assert torch.equal(tgemm.matmul_i8(a[:30], w.t(), sa[:30], sb),
                       tgemm.matmul_i8(src[:30], w.t(), sa[:30], sb))
    xs = rows(M, K // 2, 3)
    x = torch.as_strided(buf.view(torch.uint8)[: buf.numel() // 2 * 2].view(BF), (M, K // 2),
                         (ld // 2, 1))
    x.copy_(xs)
    ww = rows(80, K // 2, 4, 0.2)
    assert torch.equal(tgemm.gated_matmul(x, ww.t()), tgemm.gated_matmul(xs, ww.t()))
    q, s = tgemm.quantize_i8(x)
    q0, s0 = tgemm.quantize_i8(xs)
    assert torch.equal(q, q0) and torch.equal(s, s0)
