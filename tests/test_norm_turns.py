"""Head norm, rotation and cache write where the tokens' number decides how many blocks an SM takes, how many warps a
token, and whether the next token's queries are asked for: results as tests/test_norm_rope.py and test_q8_cache.py
hold them, and the launches themselves. (With three blocks for every call, 1900 to 2400 tokens went in two turns,
10.0 us for 8.6, and 33024 tokens in fp32 took 154 us for 131.)
"""
import pytest
import torch

from state_cached_causal_gb300 import ops
from tests import test_norm_rope, test_q8_cache
from tests._graph import kernels
from tests.test_norm_rope import case

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
sizes = pytest.mark.parametrize("T,hq,hkv,D,dtype", [
    (2100, 16, 2, 64, BF16), (4300, 8, 1, 128, BF16),       # four blocks, one turn and two
    (1000, 16, 4, 128, F32), (2400, 5, 3, 64, F32),         # two warps a token; four blocks
    (2600, 3, 1, 64, F32), (3500, 16, 1, 128, F32),         # as many steps with three: four, three
    (5000, 8, 4, 128, BF16), (6000, 16, 8, 64, BF16)])      # the next token's queries asked for


@sizes
def test_results(T, hq, hkv, D, dtype):
    test_norm_rope.check(case(1, T, hq, hkv, D, 16, dtype), False, in_place=T == 6000)


@sizes
def test_results_in_8_bits(T, hq, hkv, D, dtype):
    test_q8_cache.check(case(2, T, hq, hkv, D, 16, dtype), False)


def warps(T, hq, hkv, D, dtype):
    c = case(3, T, hq, hkv, D, 16, dtype)
    (k,) = kernels(lambda: ops.attn_norm_rope_cache(c["q"], c["k"], c["v"], c["qw"], c["kw"], 1e-5, c["cs"], c["pos"],
                                                    False, c["kc"], c["vc"], c["slots"], c["q"]))
    assert k.grid[0] <= k.resident * torch.cuda.get_device_properties(0).multi_processor_count
    return k.grid[0] * k.threads // 32


def test_warps_of_a_launch():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for dtype in (F32, BF16):
        assert warps(sms * 16, 16, 4, 128, dtype) == sms * 16                  # one turn
        assert warps(sms * 12, 16, 4, 128, dtype) >= sms * 12
        assert warps(sms * 14, 16, 4, 128, dtype) >= sms * 14
    # two batches of queries a token: by two warps each where all are at work at once
    assert warps(sms * 8, 16, 4, 128, F32) == sms * 16 and warps(sms * 8, 32, 8, 128, BF16) == sms * 16
    assert warps(sms * 100, 16, 4, 128, F32) == sms * 16                       # many turns
    assert warps(sms * 100, 32, 8, 128, BF16) == sms * 16
    assert warps(sms * 100, 16, 4, 128, BF16) == sms * 12                      # with the next token's queries
