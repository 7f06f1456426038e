"""How many blocks a call launches, read from the kernel nodes of a captured call."""
import ctypes

import pytest
import torch

import triangle_attention_biomolecular_b200 as T

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class _Kernel(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("spare", ctypes.c_void_p * 4)]


def launches(call):
    """[(grid, block)] of the kernels that ``call`` launches, in order of capture."""
    call()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    cu = ctypes.CDLL("libcuda.so.1")
    graph, n = ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ctypes.c_int(-1), _Kernel()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append((tuple(p.grid), tuple(p.block)))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("R,C,per_block", [(128, 128, 32), (1024, 16, 256), (100, 128, 32), (32, 512, 8), (4, 1024, 1),
                                           (250, 50, 64), (30, 387, 8)])
def test_norm_backward_uses_one_block_only_to_save_the_sum_of_its_parts(R, C, per_block):
    """Few rows go through one block where that saves the launch that adds up dw and db; the
    gradient of x alone has no such launch and its rows are spread."""
    x = torch.randn(R, C, device="cuda", generator=torch.Generator("cuda").manual_seed(R)).to(BF)
    w = torch.ones(C, device="cuda")
    y, stats, _ = T.norm_forward(x, w)
    both = launches(lambda: T.norm_backward(x, stats, y, w))
    assert [k[0] for k in both] == [(1, 1, 1)]
    alone = launches(lambda: T.norm_backward(x, stats, y, w, need_dw=False))
    assert [k[0] for k in alone] == [((R + per_block - 1) // per_block, 1, 1)]
    assert torch.equal(T.norm_backward(x, stats, y, w)[0], T.norm_backward(x, stats, y, w, need_dw=False)[0])
