"""Kernels of a call, as a captured graph has them: launch sizes, and how many blocks an SM holds at once."""
import ctypes

import torch


class _Params(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


class Kernel:
    def __init__(self, p, cuda):
        self.grid, self.threads, self.shared = tuple(p.grid), p.block[0], p.shared
        func, n = ctypes.c_void_p(p.func), ctypes.c_int(0)
        if not func:
            assert cuda.cuKernelGetFunction(ctypes.byref(func), ctypes.c_void_p(p.kern)) == 0
        assert cuda.cuOccupancyMaxActiveBlocksPerMultiprocessor(ctypes.byref(n), func, self.threads,
                                                                ctypes.c_size_t(self.shared)) == 0
        self.resident = n.value                 # blocks that an SM holds


def kernels(call):
    """The kernels that `call` launches, in no order (it has been called before)."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cuda, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_size_t(0)
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    assert cuda.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ctypes.c_int(-1), _Params()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:                     # a kernel
            assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append(Kernel(p, cuda))
    return out
