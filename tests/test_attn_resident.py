"""The blocks that attn_decode and its forms cut their work into are those that the GPU holds at once (the runs are
equal, so a second wave would take as long again), and the workspace is that of either cache."""
import pytest
import torch

from state_cached_causal_gb300 import ops
from tests import _q8, test_attn_decode
from tests._graph import kernels
from tests.test_attn_shared import BF16, DEV, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1), (16, 4), (12, 2), (16, 1), (32, 1), (64, 1)])
def test_one_wave(hq, hkv, D, q8, dtype):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if q8:
        q, kc, vc, ks, vs, table, lens = _q8.case(1, [5000, 300], hq, hkv, D, 16, 1, dtype)
        call = lambda: ops.attn_decode_q8(q, kc, vc, ks, vs, table, lens, 0, 0.1, out, workspace=ws)    # noqa: E731
    else:
        q, kc, vc, table, lens = test_attn_decode.case(1, [5000, 300], hq, hkv, D, 16, 1, dtype)
        call = lambda: ops.attn_decode(q, kc, vc, table, lens, 0, 0.1, out, workspace=ws)               # noqa: E731
    out = torch.zeros(q.shape, device=DEV, dtype=dtype)
    ws = torch.empty(ops.attn_decode_workspace_bytes(2, 0, hq, hkv, D), dtype=torch.uint8, device=DEV)
    grid = [k for k in kernels(call) if k.grid[0] >= sms and k.grid[0] % sms == 0 and k.grid[1:] == (1, 1)]
    assert len(grid) == 1
    # (the plain kernel's blocks of 256 dims leave room for a third, which it does not take)
    assert grid[0].grid[0] == (min(grid[0].resident, 2) if dtype is torch.float32 and D == 256 else grid[0].resident) * sms


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_wave_behind_a_prefix(D, q8):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = Case(2, [(300, [400, 5000])], 16, 4, D, 16, 1, q8)
    out = torch.zeros(c.q.shape, device=DEV, dtype=BF16)
    ws = torch.empty(ops.attn_decode_shared_workspace_bytes(2, 1, 0, 16, 4, D), dtype=torch.uint8, device=DEV)
    grid = [k for k in kernels(lambda: c.call(out, workspace=ws)) if k.grid[0] % sms == 0]
    assert len(grid) == 2                                    # the prefixes' kernel, the other's
    for k in grid:
        assert k.grid[0] <= k.resident * sms
