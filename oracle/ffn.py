"""Feed-forward block in fp64: the row quantiser with and without the RMS
norm, 8-bit products, gated projections and their gradient.  NumPy only."""

import numpy as np

from .bf16 import bf16_bits_to_f64, f64_to_bf16_bits


def _codes(t, top):
    """127 t / top to the nearest integer, ties to even, by the remainder of
    a floored division (every term is a short binary fraction: exact)."""
    n = 127.0 * t
    k = np.floor(n / top)
    twice = 2.0 * (n - k * top)
    up = (twice > top) | ((twice == top) & (np.mod(k, 2.0) == 1.0))
    return (k + up).astype(np.int8)


def quantize_rows(t, factor=None):
    """(codes int8 [M, K], scale fp64 [M]) of fp64 rows t; ``factor`` [M]
    multiplies the scales.  Rows of zeros: scale 0; rows with NaN or
    infinity: scale NaN; codes 0 in both."""
    t = np.asarray(t, dtype=np.float64)
    top = np.max(np.abs(t), axis=1)           # NaN propagates
    fine = np.isfinite(top) & (top > 0)
    safe = np.where(fine, top, 1.0)
    q = np.where(fine[:, None], _codes(np.where(fine[:, None], t, 0.0), safe[:, None]), 0)
    scale = top / 127.0 * (1.0 if factor is None else factor)
    scale = np.where(np.isfinite(top), np.where(top > 0, scale, 0.0), np.nan)
    return q.astype(np.int8), scale


def rms_norm_i8(x_bits, weight_bits, eps, residual_bits=None):
    """(codes, scale, h bits) for bf16 bit patterns [M, K], [K]."""
    h_bits = np.asarray(x_bits)
    if residual_bits is not None:
        s = bf16_bits_to_f64(h_bits) + bf16_bits_to_f64(residual_bits)
        with np.errstate(over="ignore", invalid="ignore"):
            h_bits = f64_to_bf16_bits(s.astype(np.float32))  # the sum is an fp32 one
    h = bf16_bits_to_f64(h_bits)
    with np.errstate(invalid="ignore", over="ignore"):
        t = h * bf16_bits_to_f64(weight_bits)[None, :]
        q, scale = quantize_rows(t, 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps))
    return q, scale, h_bits


def matmul_i8(a, b, scale_a, scale_b):
    """fp64 [M, N] of int8 a [M, K], b [K, N]; the sums are exact."""
    s = np.asarray(a, dtype=np.float64) @ np.asarray(b, dtype=np.float64)
    return s * np.asarray(scale_a, np.float64)[:, None] * np.asarray(scale_b, np.float64)[None, :]


def act(g, kind):
    """(act(g), act'(g), s) of act(g) = g * sigmoid(s(g))."""
    if kind == "silu":
        s, ds = g, np.ones_like(g)
    elif kind == "gelu_tanh":
        c = 2.0 * np.sqrt(2.0 / np.pi)
        s, ds = c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g * g)
    else:
        raise ValueError(kind)
    e = np.exp(-np.abs(s))
    p = np.where(s >= 0, 1.0, e) / (1.0 + e)
    pq = e / (1.0 + e) ** 2                  # p (1 - p)
    return g * p, p + g * pq * ds, s


def gated(gu, kind):
    """act(g) * u of [g | u] along the last axis."""
    F = gu.shape[1] // 2
    return act(gu[:, :F], kind)[0] * gu[:, F:]


def gated_grad(dh, gu, kind):
    """d(act(g) * u) . dh with respect to [g | u]."""
    F = gu.shape[1] // 2
    a, d, _ = act(gu[:, :F], kind)
    return np.concatenate([dh * gu[:, F:] * d, dh * a], axis=1)
