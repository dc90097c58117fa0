"""Linear layers (product, bias, activation, residual) and their gradient on
the GPU against the fp64 oracle.

Bounds (u32 = 2^-24, ub = 2^-8: half a step of fp32, of bf16):

* z: the fp32 sum of K products and the bias, (K + 1) u32 (|a| @ |b| + |bias|).
* y: an error e of z moves act(z) by at most 1.13 e; the fp32 evaluation of
  act adds (3 |s| + 8) 2 u32 of |act| (s the sigmoid's argument), the residual's
  addition u32 of the sum, the store ub (bf16) or u32 (fp32) of the result.
* dz: ub of itself, the type the products read it in, plus the fp32 terms of
  act': (3 |s| + 12) 2 u32 (1 + slope) of |dy|, as for the gated product.  The
  products sum those errors, and round once more.
* db: the fp32 terms of dz and M u32 of the sum of |dz|.
"""

import numpy as np
import pytest
import torch

import oracle
from layout_aware_gemm_amd import tgemm
from parity_util import dev
from test_gpu_ffn import BF, U32, UB, Guarded, f64, replay, rows, within

pytestmark = pytest.mark.gpu

F32 = torch.float32


def act_error(z, ez, kind):
    """Bound on the error of the computed act(z) for |error of z| <= ez."""
    a, _, s = oracle.block.act(z, kind)
    if kind in ("none", "relu"):
        return ez
    return 1.13 * ez + (np.abs(a) + 1.13 * ez) * (3 * np.abs(s) + 8) * 2 * U32


def check_forward(y, z, x, w, b, r, kind):
    X, W = f64(x), f64(w)
    B = 0.0 if b is None else f64(b)
    ref, zr = oracle.block.linear(X, W, B, kind, None if r is None else f64(r))
    ez = (X.shape[1] + 1) * 1.01 * U32 * (np.abs(X) @ np.abs(W) + np.abs(B))
    if z is not None:
        within(z, zr, ez + (UB * (np.abs(zr) + ez) if z.dtype == BF else 0))
    e = act_error(zr, ez, kind)
    if r is not None:
        e = e + 1.01 * U32 * (np.abs(ref) + e)
    within(y, ref, e + (UB if y.dtype == BF else U32) * 1.01 * (np.abs(ref) + e))


def check_backward(dx, dw, db, dy, x, w, z, kind):
    D, X, W, Z = f64(dy), f64(x), f64(w), f64(z)
    (M, K), N = X.shape, W.shape[1]
    rx, rw, rb, dz = oracle.block.linear_grad(D, X, W, Z, kind)
    ef = 0.0
    if kind not in ("none", "relu"):
        s = oracle.block.act(Z, kind)[2]
        slope = np.abs(Z) * (1.0 if kind == "silu" else 1.6 * (1 + 0.135 * Z * Z))
        ef = np.abs(D) * (3 * np.abs(s) + 12) * 2 * U32 * (1 + slope)
    eg = UB * (np.abs(dz) + ef) + ef + 1e-38

    def product(got, p, ep, q, n):
        r = p @ q
        m = (ep * 1.01 + n * 1.01 * U32 * np.abs(p)) @ np.abs(q)
        within(got, r, m * 1.01 + (UB if got.dtype == BF else U32) * (np.abs(r) + m))

    product(dx, dz, eg, W.T, N)
    product(dw.t(), dz.T, eg.T, X, M)
    if db is not None:
        within(db, rb, np.sum(ef + 1.01 * M * U32 * np.abs(dz), axis=0))


# (few-row kernel: whole, half and wide blocks of weight rows; every tile, whole
# and in K chunks; a tail of smaller tiles; edges in every direction)
SHAPES = [(1, 1, 1), (1, 16, 8), (1, 5120, 512), (3, 17, 40), (8, 4200, 72), (9, 33, 4096),
          (16, 257, 520), (17, 64, 128), (33, 300, 1000), (48, 17001, 48), (64, 129, 2048),
          (64, 4200, 40), (65, 64, 64), (100, 20001, 72), (127, 255, 136), (129, 130, 4096),
          (300, 520, 4104), (257, 513, 504), (513, 1000, 520), (130, 5003, 10248),
          (1030, 2100, 72), (2100, 4100, 40), (2300, 7268, 520), (2300, 9698, 520),
          (35, 9001, 40), (64, 16001, 40), (50, 33001, 24), (9, 7001, 136), (30, 8190, 72),
          (41, 130, 2049), (5, 6151, 8200), (5, 9, 7), (70, 33, 65), (1, 1, 300), (200, 1, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind,out,keep", [("none", BF, None), ("relu", F32, BF),
                                           ("silu", BF, F32), ("gelu_tanh", F32, None)])
def test_linear(M, N, K, kind, out, keep):
    print(f"linear {M}x{N}x{K} {kind} {out}", flush=True)
    x, w = rows(M, K, M), rows(N, K, N, 1.5 / np.sqrt(K))
    b, r = rows(1, N, 7, 0.5)[0], rows(M, N, 8, 2.0).to(out)
    got = tgemm.linear(x, w.t(), b, kind, r, out, save=keep or False)
    y, z = got if keep else (got, None)
    check_forward(y, z, x, w.t(), b, r, kind)
    check_forward(tgemm.linear(x, w.t(), act=kind, out_dtype=out), None, x, w.t(), None, None, kind)


@pytest.mark.parametrize("M,N,K", [(1, 70, 33), (3, 65, 129), (20, 100, 500), (70, 130, 31),
                                   (150, 140, 1001), (80, 3, 1)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 8), (3, 5)])
def test_layouts(M, N, K, layout, pad, off):
    """Lengths, strides and bases off the 16-byte grid in every layout; a
    residual with rows of its own stride; both directions."""
    print(f"linear {layout} {M}x{N}x{K} pad {pad} off {off}", flush=True)
    x = (rows(M, K, 1, ld=K + pad, off=off) if layout[0] == "N"
         else rows(K, M, 1, ld=M + pad, off=off).t())
    std = 1.5 / np.sqrt(K)
    w = (rows(K, N, 2, std, ld=N + pad, off=off) if layout[1] == "N"
         else rows(N, K, 2, std, ld=K + pad, off=off).t())
    b, r = rows(1, N, 3, off=off)[0], rows(M, N, 4, ld=N + pad, off=off)
    y, z = tgemm.linear(x, w, b, "silu", r, save=True)
    check_forward(y, z, x, w, b, r, "silu")
    dy = rows(M, N, 5, ld=N + pad, off=off)
    dx, dw, db = tgemm.linear_backward(dy, x, w, z, "silu", bias=True, dw_dtype=F32)
    check_backward(dx, dw, db, dy, x, w, z, "silu")
    assert dw.stride() == ((1, K) if layout[1] == "T" else (N, 1)) or 1 in (K, N)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 300, 40), (64, 64, 64), (70, 5000, 136),
                                   (300, 1000, 520), (513, 260, 264), (257, 33, 257),
                                   (4099, 31, 8), (255, 129, 1000), (2000, 33, 72),
                                   (700, 5000, 4100), (4099, 5000, 700), (65, 20100, 4100)])
@pytest.mark.parametrize("kind,keep", [("none", None), ("relu", BF), ("gelu_tanh", F32),
                                       ("silu", BF)])
def test_backward(M, N, K, kind, keep):
    """What lies between the stored rows of x, w and dy is NaN."""
    print(f"linear backward {M}x{N}x{K} {kind}", flush=True)

    def framed(n, k, seed, std):
        buf = torch.full((n, (k + 15) // 8 * 8), float("nan"), dtype=BF, device=dev())
        buf[:, :k] = rows(n, k, seed, std)
        return buf[:, :k]

    x, w, dy = framed(M, K, 1, 1.0), framed(N, K, 2, 1.5 * K ** -0.5), framed(M, N, 3, 1.0)
    y, z = tgemm.linear(x, w.t(), act=kind, save=F32)
    z = z.to(keep or F32)
    dx, dw, db = tgemm.linear_backward(dy, x, w.t(), None if keep is None else z, kind, bias=True,
                                       dw_dtype=F32)
    check_backward(dx, dw, db, dy, x, w.t(), z, kind)
    # the same bits again, with bf16 weights' gradient the rounding of it
    dx2, dw2, db2 = tgemm.linear_backward(dy, x, w.t(), z, kind)
    assert torch.equal(dx, dx2) and torch.equal(dw.to(BF), dw2) and db2 is None


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh", "relu"])
def test_saturated_and_special(kind):
    """z far out on both sides and zeros through an identity weight, NaN through
    the bias: tails, the kink and NaN as the formulas have them.  (A sigmoid's
    argument s below -174.7 counts as one that gives 0: its error is cut off
    there.)"""
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 40.0, -40.0, -100.0, 120.0, -120.0, 3e4, -3e4,
                      -8.0, 8.0, 1.0, -1.0], dtype=BF, device=dev())
    n = v.numel()
    for M in (1, 80):
        x, eye = v.repeat(M, 1), torch.eye(n, dtype=BF, device=dev())
        y, z = tgemm.linear(x, eye, None, kind, out_dtype=F32, save=True)
        assert torch.equal(z, x.float())
        Z = f64(z)
        a, d, s = oracle.block.act(Z, kind)
        s = np.minimum(np.abs(s), 180)
        within(y, a, np.abs(a) * (3 * s + 9) * 2 * U32 + 1e-37)
        dy = torch.ones(M, n, dtype=BF, device=dev())
        dx, dw, db = tgemm.linear_backward(dy, x, eye, z, kind, bias=True, dw_dtype=F32)
        slope = np.minimum(np.abs(Z) * (1.0 if kind == "silu" else 1.6 * (1 + 0.135 * Z * Z)), 180)
        ef = (3 * s + 12) * 2 * U32 * (1 + slope)
        within(dx, d, UB * (d + ef) + ef)
        within(db, d.sum(axis=0), (ef + 1.01 * M * U32 * np.abs(d)).sum(axis=0))
        nan = torch.zeros(n, dtype=BF, device=dev())
        nan[3] = float("nan")
        bad = tgemm.linear(x, eye, nan, kind)
        assert torch.isnan(bad[:, 3]).all()
        assert torch.isfinite(bad[:, :3]).all() and torch.isfinite(bad[:, 4:]).all()


def test_shapes_and_residual_in_place():
    """Leading dimensions, a 1-D x, and the residual's own buffer as output."""
    x, w, b = rows(12, 64, 1), rows(40, 64, 2, 0.2), rows(1, 40, 3)[0]
    y = tgemm.linear(x, w.t(), b)
    assert torch.equal(tgemm.linear(x.view(3, 4, 64), w.t(), b), y.view(3, 4, 40))
    assert torch.equal(tgemm.linear(x[5], w.t(), b), tgemm.linear(x[5:6], w.t(), b)[0])
    for M, N, K in ((12, 40, 64), (100, 40, 64), (70, 40, 8192), (300, 520, 64)):
        for out in (BF, F32):
            x, w, r = rows(M, K, 1), rows(N, K, 2, K ** -0.5), rows(M, N, 4).to(out)
            want = tgemm.linear(x, w.t(), residual=r, out_dtype=out)
            epi = tgemm._store(out, "out")
            args = (tgemm._flag("N"), tgemm._flag("T"), M, N, K, x.data_ptr(), K, w.data_ptr(), K,
                    None, tgemm.ACT_NONE, r.data_ptr(), N, r.data_ptr(), N, epi, None, 0, 0)
            tgemm._call_ws("tgemm_run_linear", dev(), *args)
            assert torch.equal(r, want), (M, N, K, out)


@pytest.mark.parametrize("M,N,K", [(4, 40, 4096), (1, 1, 8), (70, 33, 72), (300, 130, 520),
                                   (3, 500, 40), (257, 129, 65), (700, 5000, 1032)])
@pytest.mark.parametrize("layout", ["NT", "NN", "TN"])
def test_stays_inside(M, N, K, layout):
    """Outputs and workspaces of exactly the asked-for size, guarded."""
    print(f"linear guarded {layout} {M}x{N}x{K}", flush=True)
    x = rows(M, K, 1) if layout[0] == "N" else rows(K, M, 1)
    w = rows(N, K, 2, 0.1) if layout[1] == "T" else rows(K, N, 2, 0.1)
    b, r, dy = rows(1, N, 3), rows(M, N, 4), rows(M, N, 5)
    prod = (tgemm._flag(layout[0]), tgemm._flag(layout[1]), M, N, K, x.data_ptr(), x.stride(0),
            w.data_ptr(), w.stride(0))
    L = tgemm.lib()
    need = L.tgemm_linear_workspace_bytes(*prod)
    ws, Y, Z = Guarded(need), Guarded(2 * M * N), Guarded(4 * M * N)
    tgemm._call("tgemm_run_linear", dev(), *prod, b.data_ptr(), 0, r.data_ptr(), N, Y.ptr(), N, 0,
                Z.ptr(), N, 1, ws.ptr(), need)
    torch.cuda.synchronize()
    assert ws.intact() and Y.intact() and Z.intact()
    need = L.tgemm_linear_backward_workspace_bytes(*prod)
    ws, dA, dB, db = Guarded(need), Guarded(2 * M * K), Guarded(4 * N * K), Guarded(4 * N)
    tgemm._call("tgemm_run_linear_backward", dev(), *prod, dy.data_ptr(), N, Z.ptr(), N, 1, 0,
                dA.ptr(), K, dB.ptr(), w.shape[1], 1, db.ptr(), ws.ptr(), need)
    torch.cuda.synchronize()
    assert ws.intact() and dA.intact() and dB.intact() and db.intact()
    # the library's own workspace gives the same
    Y2 = torch.empty(M, N, dtype=BF, device=dev())
    tgemm._call("tgemm_run_linear", dev(), *prod, b.data_ptr(), 0, r.data_ptr(), N, Y2.data_ptr(),
                N, 0, None, 0, 0, None, -1)
    at = Guarded.PAD
    assert torch.equal(Y2, Y.buf[at: at + 2 * M * N].view(BF).view(M, N))


@pytest.mark.parametrize("M,N,K", [(3, 200, 264), (96, 200, 264), (300, 130, 520)])
def test_training_step_replays(M, N, K):
    x, w, b, r = rows(M, K, 1), rows(N, K, 2, 0.05), rows(1, N, 3)[0], rows(M, N, 4)
    dy = rows(M, N, 5)

    def step():
        y, z = tgemm.linear(x, w.t(), b, "silu", r, save=True)
        return (y, z) + tgemm.linear_backward(dy, x, w.t(), z, "silu", bias=True)

    def change():
        x.mul_(-0.5)
        dy.mul_(2.0)

    replay(step, change)


def test_streams():
    x, w, r = rows(90, 72, 1), rows(100, 72, 2, 0.2), rows(90, 100, 3)
    y, z = tgemm.linear(x, w.t(), act="gelu_tanh", residual=r, save=True)
    want = tgemm.linear_backward(r, x, w.t(), z, "gelu_tanh", bias=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream, 0):
        y2, z2 = tgemm.linear(x, w.t(), act="gelu_tanh", residual=r, save=True, stream=s)
        got = tgemm.linear_backward(r, x, w.t(), z2, "gelu_tanh", bias=True, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(u, v) for u, v in zip(want, got))


def test_far_offsets():
    """Row offsets past 2^32 bytes of x, the residual and the output."""
    M, K, ld = 70, 64, 35_000_000
    x, w, r = rows(M, K, 1), rows(K, K, 2, 0.2), rows(M, K, 3)
    far = torch.empty((M - 1) * ld + 2 * K, dtype=BF, device=dev())
    fx, fr = torch.as_strided(far, (M, K), (ld, 1)), torch.as_strided(far, (M, K), (ld, 1), K)
    fx.copy_(x)
    fr.copy_(r)
    want = tgemm.linear(x, w.t(), act="silu", residual=r)
    assert torch.equal(tgemm.linear(fx, w.t(), act="silu", residual=fr), want)
    want = tgemm.linear(x[:9], w.t(), act="silu", residual=r[:9])
    assert torch.equal(tgemm.linear(fx[:9], w.t(), act="silu", residual=fr[:9]), want)
