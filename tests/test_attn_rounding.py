"""bf16 attention is rounded once, when it is stored: everything before that carries more bits.

Bound: the weights enter as two bf16 terms (2^-16 of each), scores and sums are fp32, so that a result is off
by 2^-15 of its norm at most before its rounding. An error of d (of the value) turns the rounding of a value
over for a share d / u of them, u the distance of neighbours (2^-7 of the value at most), which makes
sqrt(d u) = 2^-11 of the norm against the rounded result of 64 bits. One bf16 term for the weights makes four
times that.
"""
import pytest
import torch

from state_cached_causal_gb300 import ops
from tests._mixers import attn_ref
from tests.test_attn_decode import case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16


def run(q, kc, vc, table, lens, n, scale):
    out = torch.zeros(q.shape, device=DEV, dtype=BF16)
    ops.attn_decode(q, kc, vc, table, lens, n - 1, scale, out)
    torch.cuda.synchronize()
    want, _ = attn_ref(q.cpu(), kc.cpu(), vc.cpu(), table.cpu(), lens.tolist(), n, scale)
    return out.cpu(), want


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,n", [(16, 4, 1), (4, 2, 4), (8, 1, 4)])
def test_one_rounding(D, hq, hkv, n):
    out, want = run(*case(31, [300, 65, 1000, 9], hq, hkv, D, 16, n, BF16), n, D ** -0.5)
    err = (out.double() - want.to(BF16).double()).norm() / want.norm()
    assert err <= 2.0 ** -11, f"{err:.3g}"


@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 16, 4), (256, 2, 1)])
def test_infinite_values_that_every_row_sees(D, hq, hkv):
    """An infinity among the values of one position makes its column infinite, whatever the weight's
    low bits are, and leaves the other columns; two of opposite signs make NaN."""
    q, kc, vc, table, lens = case(32, [200, 1, 70], hq, hkv, D, 16, 1, BF16)
    for b, pos in ((0, 3), (0, 150), (1, 0), (2, 69)):
        vc[int(table[b, pos // 16]), pos % 16, :, 5 + b] = float("-inf") if b == 1 else float("inf")
    vc[int(table[0, 0]), 7, :, 11], vc[int(table[0, 4]), 9, :, 11] = float("inf"), float("-inf")
    out, want = run(q, kc, vc, table, lens, 1, D ** -0.5)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.isnan(want).any()
    assert torch.isinf(want).any()
    fin = torch.isfinite(want)
    assert torch.equal(out.double()[torch.isinf(want)], want[torch.isinf(want)])
    err = (out.double()[fin] - want[fin].to(BF16).double()).norm() / want[fin].norm()
    assert err <= 2.0 ** -11, f"{err:.3g}"
