"""What the kernels of attn_decode_shared wait for, as a captured graph has it: only kernels of the call itself may
start beside one another. (With no groups the call's first kernel stood beside whatever came before it, and could read
what that one, if it let its successor start early, had yet to write.)
"""
import ctypes

import pytest
import torch

from state_cached_causal_gb300 import ops
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


def test_calls_at_once_on_two_streams():
    """Each with a workspace of its own; results are those of a call alone."""
    cases = [shared.Case(32, [(3000, [3001 + 5 * i for i in range(70)])], 16, 4, 128, 16, 1, False),
             shared.Case(33, [(900, [950, 1300]), (2000, [2100] * 9)], 16, 4, 128, 16, 2, True)]
    outs, want, spaces = [], [], []
    for c in cases:
        outs.append(torch.zeros(c.q.shape, device=shared.DEV, dtype=torch.bfloat16))
        n = ops.attn_decode_shared_workspace_bytes(len(c.lens), len(c.prefix), c.n - 1, 16, 4, 128)
        spaces.append(torch.empty(n, dtype=torch.uint8, device=shared.DEV))
        c.call(outs[-1], workspace=spaces[-1])
        torch.cuda.synchronize()
        want.append(outs[-1].clone())
        outs[-1].zero_()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    err = torch.zeros(1, dtype=torch.int32, device=shared.DEV)
    for _ in range(20):
        for c, out, ws, st in zip(cases, outs, spaces, streams):
            c.call(out, workspace=ws, stream=st, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for out, w in zip(outs, want):
        assert torch.equal(out, w)
