"""The norms around a residual sum, forward and backward, on the GPU against
the fp64 oracle.

Bounds (u = 2^-24, half a step of fp32; ub = 2^-8, of bf16; sums of n terms in
fp32 within n u of the sum of their sizes):

* p: the factor (computed in fp64) and two products, 3 u; a = scale * gate, u;
  s: 4.1 u |a p| + u |s| =: es, then the store.
* 1 / rms of s moves by ||es|| / ||s|| (Cauchy) and one rounding =: er; n by
  rs |w| es + |n| (er + 3 u), then the store.
* the backward pass computes s within es again and reads the kept factors; its
  terms are followed below, step by step.
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
EPS = 1e-6


def unit(t):
    return UB if t.dtype == BF else U32


def vec(n, seed, mean=1.0, std=0.2):
    return (mean + rows(1, n, seed, std)[0].float()).to(BF)


def inputs(M, K, G, post, res, pad=0, off=0):
    y, h = rows(M, K, 1, ld=K + pad, off=off), rows(M, K, 2, 2.0, ld=K + pad, off=off).to(res)
    gate = None if G == 0 else (0.4 + rows(G, K, 3, 0.2, ld=K + pad, off=off).float()).to(BF)
    if gate is not None and pad:
        g = torch.zeros(G, K + pad, dtype=BF, device=dev())
        g[:, :K] = gate
        gate = g[:, :K]
    return y, h, vec(K, 4), vec(K, 5) if post else None, gate


def terms(y, h, w, post, gate, scale):
    """fp64 values, and es, er, ep of the module's docstring."""
    o = {"y": f64(y), "h": f64(h), "w": f64(w), "post": None if post is None else f64(post),
         "gate": None if gate is None else f64(gate.reshape(-1, y.shape[1]))}
    n, s, p = oracle.block.block_norm(**o, scale=scale, eps=EPS)
    a = scale * (np.ones_like(p) if gate is None else oracle.block.spread(o["gate"], p.shape[0]))
    es = 4.1 * U32 * np.abs(a * p) + 1.01 * U32 * np.abs(s)
    norm = np.sqrt(np.sum(s * s, axis=1, keepdims=True) + s.shape[1] * EPS)
    er = np.sqrt(np.sum(es * es, axis=1, keepdims=True)) / norm + 1.01 * U32
    return o, n, s, p, a, es, er


def check_forward(n, s, args, scale):
    o, rn, rs, p, a, es, er = terms(*args, scale)
    within(s, rs, es + unit(s) * (np.abs(rs) + es))
    r = 1 / np.sqrt(np.mean(rs * rs, axis=1, keepdims=True) + EPS)
    en = 1.01 * (r * np.abs(o["w"]) * es + np.abs(rn) * (er + 3 * U32))
    within(n, rn, en + UB * (np.abs(rn) + en))


def check_backward(got, dn, ds, args, scale):
    dh, dy, dw, dp, dg = got
    o, _, s, p, a, es, er = terms(*args, scale)
    D, S = f64(dn), 0.0 if ds is None else f64(ds)
    M, K = D.shape
    rh, ry_, rw, rp, rg = oracle.block.block_norm_grad(D, **o, scale=scale, eps=EPS,
                                                       ds=None if ds is None else S)
    u, y, post = U32, o["y"], 1.0 if o["post"] is None else o["post"]
    r = 1 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + EPS)
    e = D * o["w"]

    def total(x):
        return np.sum(x, axis=1, keepdims=True)

    c1 = total(e * s)
    E1 = total(K * 1.01 * u * np.abs(e * s) + np.abs(e) * es)
    k, Ek = r ** 3 / K * c1, r ** 3 / K * (E1 + np.abs(c1) * (3 * er + 8 * u))
    et = (np.abs(r * e) * (er + 3 * u) + np.abs(k) * es + np.abs(s) * Ek
          + 4 * u * (np.abs(S) + np.abs(r * e) + np.abs(k * s)))
    within(dh, rh, et + unit(dh) * (np.abs(rh) + et))
    x = np.abs(D * s * r)
    within(dw, rw, np.sum(np.abs(D) * r * es + x * (er + (M + 4) * 1.01 * u), axis=0))
    if dg is not None:
        G = o["gate"].shape[0]
        x = np.abs(scale * rh * p)
        b = (np.abs(scale * p) * et + x * (M // G + 8) * 1.01 * u).reshape(G, -1, K).sum(axis=1)
        within(dg.reshape(G, K), rg, b)
    if dp is None:
        e = np.abs(a) * et + 2 * u * np.abs(ry_)
        within(dy, ry_, e + UB * (np.abs(ry_) + e))
        return
    ry = 1 / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + EPS)
    x = np.abs(a * rh * y * ry)
    within(dp, rp, np.sum(np.abs(a * y * ry) * et + x * (M + 8) * 1.01 * u, axis=0))
    q, f = a * post * y, a * rh * post
    part = np.abs(S) + np.abs(r * e)
    EQ = total(np.abs(q) * (np.abs(r * e) * (er + 2 * u) + (K + 6) * 1.01 * u * part)
               + np.abs(k * q) * (es + (K + 6) * 1.01 * u * np.abs(s))
               + np.abs(q * s) * Ek + 4 * u * np.abs(q) * (part + np.abs(k * s)))
    ey = (np.abs(ry * a * post) * et + 6 * u * np.abs(ry * f)
          + np.abs(y) * ry ** 3 / K * (EQ + 8 * u * np.abs(total(f * y))))
    ey = 1.01 * ey
    within(dy, ry_, ey + UB * (np.abs(ry_) + ey))


# (rows of one wave to eight, of one to four chunks per thread; more rows than
# workgroups; odd lengths; gates per channel, sequence and token, groups that
# end inside a workgroup's rows and that span several)
CASES = [(1, 1, 1), (3, 5, 3), (2, 8, 0), (5, 511, 1), (6, 513, 2), (4, 4096, 4), (3, 4100, 1),
         (6, 5120, 3), (2, 8192, 1), (3, 8193, 3), (4, 13824, 2), (2, 16384, 1), (600, 264, 1),
         (1100, 520, 11), (1100, 72, 550), (1026, 136, 1026), (1536, 40, 3), (1536, 33, 512),
         (700, 2049, 7), (520, 5000, 1)]


@pytest.mark.parametrize("M,K,G", CASES)
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("res", [BF, F32])
def test_block_norm(M, K, G, post, res):
    print(f"block norm {M}x{K} gates {G} post {post} {res}", flush=True)
    args = inputs(M, K, G, post, res)
    y, h, w, wp, gate = args
    kw = {"post_weight": wp, "gate": gate, "scale": 0.75}
    n, s, rstd = tgemm.block_norm(y, h, w, eps=EPS, save=True, **kw)
    assert rstd.shape == (1 + post, M)
    check_forward(n, s, args, 0.75)
    n2, s2 = tgemm.block_norm(y, h, w, eps=EPS, **kw)
    assert torch.equal(n, n2) and torch.equal(s, s2)
    dn, ds = rows(M, K, 8), rows(M, K, 9).to(res)
    for d in (ds, None):
        got = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=d, **kw)
        check_backward(got, dn, d, args, 0.75)
        again = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=d, **kw)
        assert all(u is v or torch.equal(u, v) for u, v in zip(got, again))


@pytest.mark.parametrize("pad,off", [(8, 0), (3, 5)])
@pytest.mark.parametrize("M,K,G", [(5, 40, 5), (3, 4099, 1), (600, 129, 3)])
def test_strides(M, K, G, pad, off):
    """Rows of any stride and alignment; a gate [K] is a gate [1, K]."""
    args = inputs(M, K, G, True, BF, pad, off)
    y, h, w, wp, gate = args
    kw = {"post_weight": wp, "gate": gate, "scale": 0.5}
    n, s, rstd = tgemm.block_norm(y, h, w, eps=EPS, save=True, **kw)
    check_forward(n, s, args, 0.5)
    dn, ds = rows(M, K, 8, ld=K + pad, off=off), rows(M, K, 9, ld=K + pad, off=off)
    got = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)
    check_backward(got, dn, ds, args, 0.5)
    if G == 1:
        kw["gate"] = gate[0]
        assert torch.equal(tgemm.block_norm(y, h, w, eps=EPS, **kw)[0], n)
        flat = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)
        assert flat[4].shape == (K,) and torch.equal(flat[4], got[4][0])


def test_leading_dimensions_and_in_place():
    M, K = 12, 264
    y, h, w, wp, gate = inputs(M, K, 3, True, BF)
    kw = {"post_weight": wp, "gate": gate, "scale": 0.5}
    n, s, rstd = tgemm.block_norm(y, h, w, save=True, **kw)
    n3, s3 = tgemm.block_norm(y.view(3, 4, K), h.view(3, 4, K), w, **kw)
    assert torch.equal(n3, n.view(3, 4, K)) and torch.equal(s3, s.view(3, 4, K))
    own = h.clone()
    n2, s2 = tgemm.block_norm(y, own, w, out_residual=own, **kw)
    assert s2 is own and torch.equal(own, s) and torch.equal(n2, n)
    # dresidual over ds and dy over dn
    for K, M in ((264, 12), (520, 1100), (9000, 5)):
        y, h, w, wp, gate = inputs(M, K, 1, True, BF)
        kw = {"post_weight": wp, "gate": gate, "scale": 0.5}
        n, s, rstd = tgemm.block_norm(y, h, w, save=True, **kw)
        dn, ds = rows(M, K, 8), rows(M, K, 9)
        want = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)
        f32 = {"dtype": F32, "device": dev()}
        dw, dp, dg = torch.empty(K, **f32), torch.empty(K, **f32), torch.empty(1, K, **f32)
        tgemm._call("tgemm_block_norm_backward", dev(), dn.data_ptr(), K, ds.data_ptr(), K,
                    y.data_ptr(), K, h.data_ptr(), K, 0, wp.data_ptr(), gate.data_ptr(), K, 1, 0.5,
                    w.data_ptr(), rstd.data_ptr(), M, K, ds.data_ptr(), K, dn.data_ptr(), K,
                    dw.data_ptr(), dp.data_ptr(), dg.data_ptr(), None, -1)
        assert all(torch.equal(u, v) for u, v in zip(want, (ds, dn, dw, dp, dg)))


def test_special_rows():
    """Rows of zeros, of huge and of tiny values, and one that holds NaN, which
    spoils no other."""
    M, K = 6, 520
    y, h, w, wp, gate = inputs(M, K, 1, True, BF)
    y[1], h[1] = 0.0, 0.0
    y[2] *= 2.0 ** 80          # squares past the largest fp32
    y[3] *= 2.0 ** -40
    h[3] *= 2.0 ** -40
    y[4, 7] = float("nan")
    keep = [0, 1, 2, 3, 5]
    kw = {"post_weight": wp, "gate": gate, "scale": 0.5}
    n, s, rstd = tgemm.block_norm(y, h, w, save=True, eps=EPS, **kw)
    assert torch.isnan(n[4]).all()
    part = [t[keep] for t in (y, h)] + [w, wp, gate]
    check_forward(n[keep], s[keep], part, 0.5)
    assert bool((n[1] == 0).all()) and bool((s[1] == 0).all())
    dn, ds = rows(M, K, 8), rows(M, K, 9)
    dh, dy = tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)[:2]
    assert torch.isnan(dh[4]).all() and torch.isnan(dy[4]).all()
    assert torch.isfinite(dh[keep]).all() and torch.isfinite(dy[keep]).all()
    fine = [0, 3, 5]
    part = [t[fine].contiguous() for t in (y, h)] + [w, wp, gate]
    got = tgemm.block_norm_backward(dn[fine].contiguous(), part[0], part[1],
                                    rstd[:, fine].contiguous(), w, ds=ds[fine].contiguous(), **kw)
    check_backward(got, dn[fine], ds[fine], part, 0.5)
    assert torch.equal(got[0], dh[fine]) and torch.equal(got[1], dy[fine])


@pytest.mark.parametrize("M,K,G", [(1, 1, 1), (4, 96, 2), (3, 4104, 0), (2, 8201, 1), (600, 129, 3),
                                   (1100, 72, 550)])
@pytest.mark.parametrize("st", [0, 1])
def test_stays_inside(M, K, G, st):
    print(f"block norm guarded {M}x{K} {G} {st}", flush=True)
    y, h, w, wp, gate = inputs(M, K, G, True, F32 if st else BF)
    size = 4 if st else 2
    s, n, rstd = Guarded(size * M * K), Guarded(2 * M * K), Guarded(8 * M)
    g = None if gate is None else gate.data_ptr()
    common = (y.data_ptr(), K, h.data_ptr(), K, st, wp.data_ptr(), g, K, G, 0.5, w.data_ptr())
    tgemm._call("tgemm_block_norm", dev(), *common, EPS, M, K, s.ptr(), K, n.ptr(), K, rstd.ptr())
    torch.cuda.synchronize()
    assert s.intact() and n.intact() and rstd.intact()
    dn, ds = rows(M, K, 8), rows(M, K, 9).to(h.dtype)
    need = tgemm.lib().tgemm_block_norm_backward_workspace_bytes(M, K, 1, G)
    dh, dy, ws = Guarded(size * M * K), Guarded(2 * M * K), Guarded(need)
    dw, dp, dg = Guarded(4 * K), Guarded(4 * K), Guarded(4 * max(G, 1) * K)
    args = (dn.data_ptr(), K, ds.data_ptr(), K) + common + (rstd.ptr(), M, K, dh.ptr(), K, dy.ptr(),
                                                            K, dw.ptr(), dp.ptr(),
                                                            dg.ptr() if G else None)
    run, stream = tgemm.lib().tgemm_block_norm_backward, torch.cuda.current_stream().cuda_stream
    assert run(*args, ws.ptr(), need - 1, stream) == tgemm.TGEMM_ERR_WORKSPACE_LIMIT
    assert run(*args, ws.ptr() + 4, need, stream) == tgemm.TGEMM_ERR_INVALID_ARG
    assert run(*args, ws.ptr(), need, stream) == 0
    torch.cuda.synchronize()
    assert all(b.intact() for b in (dh, dy, ws, dw, dp, dg))


@pytest.mark.parametrize("M,K,G", [(3, 512, 1), (1100, 264, 11)])
def test_training_step_replays(M, K, G):
    y, h, w, wp, gate = inputs(M, K, G, True, BF)
    dn, ds = rows(M, K, 8), rows(M, K, 9)
    kw = {"post_weight": wp, "gate": gate, "scale": 0.5}

    def step():
        n, s, rstd = tgemm.block_norm(y, h, w, save=True, **kw)
        return (n, s) + tgemm.block_norm_backward(dn, y, h, rstd, w, ds=ds, **kw)

    def change():
        y.mul_(-0.5)
        dn.mul_(2.0)

    replay(step, change)


def test_streams():
    y, h, w, wp, gate = inputs(700, 264, 7, True, BF)
    kw = {"post_weight": wp, "gate": gate, "scale": 0.5}
    n, s, rstd = tgemm.block_norm(y, h, w, save=True, **kw)
    want = tgemm.block_norm_backward(n, y, h, rstd, w, ds=s, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream, 0):
        n2, s2, r2 = tgemm.block_norm(y, h, w, save=True, stream=st, **kw)
        got = tgemm.block_norm_backward(n2, y, h, r2, w, ds=s2, stream=st, **kw)
        torch.cuda.synchronize()
        assert torch.equal(n, n2) and all(torch.equal(u, v) for u, v in zip(want, got))


def test_far_offsets():
    """Row offsets past 2^32 bytes."""
    M, K, ld = 70, 64, 35_000_000
    y, h, w, wp, gate = inputs(M, K, 1, True, BF)
    far = torch.empty((M - 1) * ld + 4 * K, dtype=BF, device=dev())
    fy, fh, fs = (torch.as_strided(far, (M, K), (ld, 1), i * K) for i in range(3))
    fy.copy_(y)
    fh.copy_(h)
    kw = {"post_weight": wp, "gate": gate, "scale": 0.5}
    n, s, rstd = tgemm.block_norm(y, h, w, save=True, **kw)
    n2, _ = tgemm.block_norm(fy, fh, w, out_residual=fs, **kw)
    assert torch.equal(n, n2) and torch.equal(s, fs)
    want = tgemm.block_norm_backward(n, y, h, rstd, w, ds=s, **kw)
    got = tgemm.block_norm_backward(n, fy, fh, rstd, w, ds=fs, **kw)
    assert all(torch.equal(u, v) for u, v in zip(want, got))
