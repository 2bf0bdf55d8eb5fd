"""What the kernels of attn_decode_shared wait for, as a captured graph has it: only kernels of the call itself may
start beside one another. (With no groups the call's first kernel stood beside whatever came before it, and could read
what that one, if it let its successor start early, had yet to write.)
"""
import ctypes

import pytest
import torch

from tests import test_attn_shared as shared

pytestmark = pytest.mark.gpu


class Edge(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def programmatic(graph):
    """Of a graph's edges: [whether its end may start beside its beginning] in the order of the nodes."""
    cuda = ctypes.CDLL("libcuda.so.1")
    n = ctypes.c_size_t(0)
    args = (ctypes.c_void_p(graph.raw_cuda_graph()),)
    assert cuda.cuGraphGetEdges_v2(*args, None, None, None, ctypes.byref(n)) == 0
    a, b, e = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (Edge * n.value)()
    assert cuda.cuGraphGetEdges_v2(*args, a, b, e, ctypes.byref(n)) == 0
    after = {a[i]: (b[i], e[i].type != 0) for i in range(n.value)}
    at = next(x for x in after if x not in {y for y, _ in after.values()})
    kinds = []
    while at in after:                       # (a chain: everything is on one stream)
        at, kind = after[at]
        kinds.append(kind)
    assert len(kinds) == n.value
    return kinds


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("groups", [0, 1])
def test_only_the_calls_own_kernels_run_beside_one_another(q8, groups):
    c = shared.Case(31, [(40, [50, 61])] if groups else [], 8, 2, 64, 16, 1, q8, loose=([33], [70]))
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=shared.DEV)
    out = torch.zeros(c.q.shape, device=shared.DEV, dtype=torch.bfloat16)
    c.call(out, workspace=ws)
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        out.zero_()
        c.call(out, workspace=ws)
        out.mul_(1.0)
    kinds = programmatic(graph)
    # zeros; prefixes, if any; own positions; join; product
    assert kinds == ([False, True, True, False] if groups else [False, True, False])
    graph.instantiate()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
