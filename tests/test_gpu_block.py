"""The operators around a block's products run together, as a block is trained
and as it is served, on the GPU against the fp64 oracle: each step is fed with
the GPU's own previous output, so a step's bound is its own (those of the
operators' own tests)."""

import numpy as np
import pytest
import torch

from layout_aware_gemm_amd import tgemm
from test_gpu_block_norm import EPS, check_backward as check_norm_backward
from test_gpu_block_norm import check_forward as check_norm
from test_gpu_ffn import BF, replay, rows
from test_gpu_linear import check_backward, check_forward
from test_gpu_moe import check_layer, check_routing, layer

pytestmark = pytest.mark.gpu

F32 = torch.float32


def vec(n, seed, mean=1.0, std=0.1):
    return (mean + rows(1, n, seed, std)[0].float()).to(BF)


class Dense:
    """norm -> up (bias, gelu) -> down (bias), gated onto the stream -> norm"""

    def __init__(self, M, D, F, stream):
        self.y, self.h = rows(M, D, 1), rows(M, D, 2, 2.0).to(stream)
        self.w1, self.w2 = rows(F, D, 3, D ** -0.5), rows(D, F, 4, F ** -0.5)
        self.b1, self.b2 = vec(F, 5, 0.0, 0.5), vec(D, 6, 0.0, 0.5)
        self.n1, self.n2, self.post = vec(D, 7), vec(D, 8), vec(D, 9)
        self.gate = vec(D, 10, 0.3)
        self.dn, self.ds = rows(M, D, 11), rows(M, D, 12).to(stream)

    def forward(self):
        a, h1, r1 = tgemm.block_norm(self.y, self.h, self.n1, save=True)
        u, z1 = tgemm.linear(a, self.w1.t(), self.b1, "gelu_tanh", save=True)
        o = tgemm.linear(u, self.w2.t(), self.b2)
        n, h2, r2 = tgemm.block_norm(o, h1, self.n2, self.post, self.gate, 0.5, save=True)
        return a, h1, r1, u, z1, o, n, h2, r2

    def step(self):
        a, h1, r1, u, z1, o, n, h2, r2 = f = self.forward()
        g2 = tgemm.block_norm_backward(self.dn, o, h1, r2, self.n2, self.post, self.gate, 0.5,
                                       ds=self.ds)
        l2 = tgemm.linear_backward(g2[1], u, self.w2.t(), bias=True, dw_dtype=F32)
        l1 = tgemm.linear_backward(l2[0], a, self.w1.t(), z1, "gelu_tanh", bias=True, dw_dtype=F32)
        g1 = tgemm.block_norm_backward(l1[0], self.y, self.h, r1, self.n1, ds=g2[0])
        return f, g2, l2, l1, g1


@pytest.mark.parametrize("M,D,F,stream", [(96, 264, 520, BF), (333, 520, 1000, F32), (1, 64, 96, BF),
                                          (5, 1000, 333, F32)])
def test_dense_block_trains(M, D, F, stream):
    b = Dense(M, D, F, stream)
    (a, h1, r1, u, z1, o, n, h2, r2), g2, l2, l1, g1 = b.step()
    first, second = (b.y, b.h, b.n1, None, None), (o, h1, b.n2, b.post, b.gate)
    check_norm(a, h1, first, 1.0)
    check_forward(u, z1, a, b.w1.t(), b.b1, None, "gelu_tanh")
    check_forward(o, None, u, b.w2.t(), b.b2, None, "none")
    check_norm(n, h2, second, 0.5)
    check_norm_backward(g2, b.dn, b.ds, second, 0.5)
    check_backward(*l2, g2[1], u, b.w2.t(), z1[:, :1].expand(M, D), "none")
    check_backward(*l1, l2[0], a, b.w1.t(), z1, "gelu_tanh")
    check_norm_backward(g1, l1[0], g2[0], first, 1.0)


@pytest.mark.parametrize("M,D,F", [(96, 264, 200), (3, 512, 128)])
def test_dense_block_replays(M, D, F):
    """A captured training step, its launches in one graph."""
    b = Dense(M, D, F, BF)

    def step():
        f, *grads = b.step()
        return [t for t in f] + [t for g in grads for t in g if t is not None]

    def change():
        b.y.mul_(-0.5)
        b.dn.mul_(2.0)

    replay(step, change)


def served(y, h, n1, n2, post, wo, bo, r, w1, w2):
    """A decode step: projection onto the stream, norm, experts, norm."""
    h1 = tgemm.linear(y, wo.t(), bo, residual=h)
    a, h1 = tgemm.block_norm(y, h1, n1)
    o, ids, p = tgemm.moe(a, r.t(), w1.transpose(1, 2), w2.transpose(1, 2), 2, routing=True)
    n, h2 = tgemm.block_norm(o, h1, n2, post)
    return h1, a, o, ids, p, n, h2


@pytest.mark.parametrize("M", [1, 13, 64])
def test_served_block(M):
    D, F, E = 264, 72, 8
    _, r, w1, w2 = layer(M, D, F, E, seed=20)
    y, h, wo = rows(M, D, 1), rows(M, D, 2, 2.0), rows(D, D, 3, D ** -0.5)
    bo, n1, n2, post = vec(D, 4, 0.0, 0.5), vec(D, 5), vec(D, 6), vec(D, 7)
    args = (y, h, n1, n2, post, wo, bo, r, w1, w2)
    first = tgemm.linear(y, wo.t(), bo, residual=h)
    check_forward(first, None, y, wo.t(), bo, h, "none")
    h1, a, o, ids, p, n, h2 = served(*args)
    check_norm(a, h1, (y, first, n1, None, None), 1.0)
    check_routing(ids, p, a, r, 2)
    check_layer(o, a, ids, p, w1, w2, "silu")
    check_norm(n, h2, (o, h1, n2, post, None), 1.0)
    replay(lambda: served(*args), lambda: y.mul_(-0.5))
    assert EPS == 1e-6 and np.isfinite(n.float().cpu().numpy()).all()
