"""Chunked outputs of the gated delta rule in bf16 are rounded once, when they are stored.

Bound: states, scores and updates enter the output products as two bf16 terms (2^-17 of each), sums are
fp32, and the state is off by a few of 2^-18, so that an output is off by 2^-15 of its norm at most before
its rounding; against the rounded result of 64 bits that makes 2^-11 of the norm (as in
test_attn_rounding.py). One bf16 term for the scores or the state makes twice to four times that.
"""
import math

import pytest
import torch

from state_cached_causal_gb300 import ops
from tests._mixers import gdn_ref
from tests.test_gdn import DEV, BF16, F32, inputs, pool

pytestmark = pytest.mark.gpu


def errors(seed, lens, hk, hv, st_dtype, scale=128 ** -0.5, **kw):
    """Per sequence: error of the outputs against the rounded ones of 64 bits, over their norm."""
    T = sum(lens)
    inp = inputs(seed, T, hk, hv, 128, 128, BF16, spare=0, **kw)
    st = pool(seed, len(lens), hv, 128, 128, st_dtype)
    S0 = st.double().cpu()
    out = torch.zeros(T, hv, 128, device=DEV, dtype=BF16)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    ops.gdn_fwd_varlen(*inp, st, torch.arange(len(lens), dtype=torch.int32, device=DEV), cu, None, scale,
                       out)
    torch.cuda.synchronize()
    cpu = [t.double().cpu() for t in inp]
    got = []
    for i, n in enumerate(lens):
        a, b = int(cu[i]), int(cu[i + 1])
        want = gdn_ref(*[t[a:b] for t in cpu[:5]], *cpu[5:], S0[i], scale)[0]
        got.append(((out[a:b].double().cpu() - want.to(BF16).double()).norm() / want.norm()).item())
    return got


@pytest.mark.parametrize("st_dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[64], [9, 17, 33, 49, 63], [65, 128, 300]])
def test_one_rounding(lens, st_dtype):
    worst = max(errors(51, lens, 2, 4, st_dtype))
    assert worst <= 2.0 ** -11, f"{worst:.3g}"


def test_one_rounding_with_gates_at_their_ends():
    worst = max(errors(52, [130, 70], 1, 2, F32, gates="ends"))
    assert worst <= 2.0 ** -11, f"{worst:.3g}"


@pytest.mark.parametrize("n", [5, 9, 64, 130])
def test_decays_are_those_of_64_bits(n):
    """Keys of zero leave a state that only decays: its error is the gates' own. Gates far out (a softplus
    of e^-80 under a rate of e^80) by either kernel. The log decay of a token is two exponentials, a
    log1p and two products, each off by 1 or 2 of 2^-24: under 5e-7 of it. The n tokens' sum is 8, so
    that the state is off by 4e-6, and 1e-6 for the last exponential; exponentials whose argument was
    rounded after a product with log2(e) would make 8 * 80 * 2^-24 = 4e-5."""
    hv = 4
    inp = list(inputs(53, n, 2, hv, 128, 128, BF16, spare=0))
    inp[1] = torch.zeros_like(inp[1])
    inp[3] = torch.tensor([-80.0, -76.0, -60.0, -40.0], device=DEV).expand(n, hv).to(BF16).contiguous()
    inp[5] = -inp[3][0].float() - math.log(n / 8)
    inp[6] = torch.zeros(hv, device=DEV)
    st = pool(53, 1, hv, 128, 128, F32)
    S0 = st[0].double().cpu()
    out = torch.zeros(n, hv, 128, device=DEV, dtype=BF16)
    ops.gdn_fwd_varlen(*inp, st, torch.zeros(1, dtype=torch.int32, device=DEV),
                       torch.tensor([0, n], dtype=torch.int32, device=DEV), None, 0.1, out)
    torch.cuda.synchronize()
    cpu = [t.double().cpu() for t in inp]
    want = gdn_ref(*cpu, S0, 0.1)[1][-1]
    err = (st[0].double().cpu() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    assert err.max().item() <= 1e-5, err
