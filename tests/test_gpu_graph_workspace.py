"""Workspace of captured calls: a graph holds kernels only (nothing in it
allocates, frees or clears memory), calls of one capture share a buffer that
grows between them, and two graphs never share one."""

import ctypes

import pytest
import torch

import workloads
from layout_aware_gemm_amd import tgemm
from parity_util import dev

pytestmark = pytest.mark.gpu

KERNEL, EMPTY = 0, 5  # hipGraphNodeType
BF, F32 = torch.bfloat16, torch.float32


def nt(M, N, K, seed):
    d = workloads.random_operands(M, N, K, "N", "T", seed=seed)
    return d["A"].to(dev()), d["B"].to(dev()), d["lda"], d["ldb"]


def split_product(seed=1, N=512):
    """256 x N x 8192: few tiles, K split into chunks."""
    A, B, lda, ldb = nt(256, N, 8192, seed)
    C = torch.empty(256, N, dtype=BF, device=dev())
    return lambda: tgemm.run("N", "T", 256, N, 8192, A, lda, B, ldb, C, N,
                             tgemm.EPI_STORE_BF16), (C,), (A,)


def row_product():
    """1 x 512 x 8192 of a weight stored [K][N]: partial sums of K chunks."""
    A, B = (torch.randn(1, 8192, device=dev()).to(BF), torch.randn(8192, 512, device=dev()).to(BF))
    C = torch.empty(1, 512, dtype=F32, device=dev())
    return lambda: tgemm.run("N", "N", 1, 512, 8192, A, 8192, B, 512, C, 512,
                             tgemm.EPI_STORE_F32), (C,), (A,)


def ce(grad):
    w = workloads.tiny_ce()
    H, W, lab = w["A"].to(dev()), w["W"].to(dev()), w["labels"].to(dev())
    loss = torch.empty(64, dtype=F32, device=dev())
    g = torch.empty(64, 256, dtype=BF, device=dev()) if grad else None
    return lambda: tgemm.run("N", "T", 64, 256, 128, H, 128, W, 128, None, 256, tgemm.EPI_CE,
                             labels=lab, out_loss=loss, out_grad=g), \
        ((loss, g) if grad else (loss,)), (H,)


def ce_deferred():
    w = workloads.tiny_ce()
    H, W, lab = w["A"].to(dev()), w["W"].to(dev()), w["labels"].to(dev())
    loss = torch.empty(64, dtype=F32, device=dev())
    e = torch.empty(64, 256, dtype=BF, device=dev())
    sc = torch.empty(4, 64, dtype=F32, device=dev())
    return lambda: tgemm.run_ce_deferred("N", "T", 64, 256, 128, H, 128, W, 128, lab, loss, e, 256,
                                         sc), (loss, e, sc), (H,)


def fp8():
    """520 x 536 x 256: both operands cast into the workspace first."""
    A, B, lda, ldb = nt(520, 536, 256, 5)
    sc = torch.tensor([4.0, 8.0, 1.0 / 32], dtype=F32, device=dev())
    C = torch.empty(520, 536, dtype=BF, device=dev())
    return lambda: tgemm.run_fp8("N", "T", 520, 536, 256, A, lda, B, ldb, C, 536,
                                 tgemm.EPI_STORE_BF16, sc), (C,), (A,)


CALLS = {"split": split_product, "row": row_product, "ce": lambda: ce(False),
         "ce_grad": lambda: ce(True), "ce_deferred": ce_deferred, "fp8": fp8}


@pytest.mark.parametrize("name", CALLS)
def test_captured_calls_are_kernels_only(name):
    """The nodes of a captured call.  (The graph is looked at, not run.)"""
    print(name, flush=True)
    call = CALLS[name]()[0]
    call()
    torch.cuda.synchronize()
    L, vp = tgemm.lib(), ctypes.c_void_p
    L.hipStreamBeginCapture.argtypes = [vp, ctypes.c_int]
    L.hipStreamEndCapture.argtypes = [vp, ctypes.POINTER(vp)]
    L.hipGraphGetNodes.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(ctypes.c_size_t)]
    L.hipGraphNodeGetType.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    L.hipGraphDestroy.argtypes = [vp]
    side = torch.cuda.Stream()
    graph, n = vp(), ctypes.c_size_t()
    with torch.cuda.stream(side):
        assert L.hipStreamBeginCapture(side.cuda_stream, 0) == 0
        try:
            call()
        finally:
            assert L.hipStreamEndCapture(side.cuda_stream, ctypes.byref(graph)) == 0
    assert L.hipGraphGetNodes(graph, None, ctypes.byref(n)) == 0 and n.value > 0
    nodes, kinds = (vp * n.value)(), []
    assert L.hipGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        k = ctypes.c_int(-1)
        assert L.hipGraphNodeGetType(node, ctypes.byref(k)) == 0
        kinds.append(k.value)
    assert L.hipGraphDestroy(graph) == 0
    assert kinds.count(KERNEL) >= 1 and set(kinds) <= {KERNEL, EMPTY}, kinds


def captured(calls):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    return g


def test_buffer_grows_within_a_capture():
    """Calls of growing, then shrinking need in one graph, replayed between
    eager calls of the same on changed inputs."""
    made = [row_product(), split_product(2, 256), split_product(3, 512), row_product(), ce(True)]
    calls = [m[0] for m in made]
    g = captured(calls)
    for rep in range(3):
        for m in made:
            m[2][0].mul_(-0.5)
        for c in calls:
            c()
        want = [o.clone() for m in made for o in m[1]]
        for m in made:
            for o in m[1]:
                o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (o, r) in enumerate(zip([o for m in made for o in m[1]], want)):
            assert torch.equal(o, r), (rep, i)


def test_graphs_do_not_share():
    """Two graphs captured one after the other, replayed at once on two
    streams beside eager calls on a third."""
    one, two, three = split_product(7), split_product(8), split_product(9)
    for m in (one, two, three):
        m[0]()
    torch.cuda.synchronize()
    want = [m[1][0].clone() for m in (one, two, three)]
    g1, g2 = captured([one[0]] * 3), captured([two[0]] * 3)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        for m in (one, two, three):
            m[1][0].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        for _ in range(3):
            three[0]()
        torch.cuda.synchronize()
        for i, m in enumerate((one, two, three)):
            assert torch.equal(m[1][0], want[i]), (rep, i)
