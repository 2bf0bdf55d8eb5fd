"""Rows next to the largest fp32 number through the cache in 8 bits: values from 1.9375 * 2^127 on would round to 2^128,
which reads back as infinity; they are stored as the largest value below it, 1.875 * 2^127."""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests._q8 import DEV, F8, cache_pair, values
from tests.test_norm_rope import case

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_finite_rows_stay_finite(dtype, D):
    c = case(1, 12, 2, 3, D, 16, dtype)
    c["cs"][:, :8], c["cs"][:, 8:] = 1, 0                                # no rotation
    most = torch.finfo(dtype).max
    x = torch.linspace(-1, 1, D, device=DEV, dtype=torch.float64)
    for i, f in enumerate((1.0, 1.0, 0.99, 0.97, 0.9688, 0.96, 0.94, 0.9, 0.88, 0.87, 0.5)):
        c["k"][i], c["v"][i] = (x * most * f).to(dtype), (x.flip(0) * most * f).to(dtype)
    c["v"][1, :, 3] = float("nan")
    c["v"][2, :, 4] = float("-inf")
    kc, vc, ks, vs = cache_pair(synth.generator(8, DEV), tuple(c["kc"].shape))
    ops.attn_norm_rope_cache_q8(c["q"], c["k"], c["v"], None, None, 1e-6, c["cs"], c["pos"], False, kc, vc, ks, vs,
                                c["slots"], torch.zeros_like(c["q"]))
    ko, vo = (torch.zeros(12, 3, D, device=DEV, dtype=F32) for _ in range(2))
    ops.kv_cache_read_q8(kc, vc, ks, vs, c["slots"], ko, vo)
    torch.cuda.synchronize()
    odd = torch.zeros(c["v"].shape, dtype=torch.bool, device=DEV)
    odd[1, :, 3] = odd[2, :, 4] = True
    assert torch.isnan(vo[odd]).all()
    at, page = c["slots"].long(), kc.shape[1]
    for got, want, cache, scale, skip in ((ko, c["k"], kc, ks, ~odd | odd), (vo, c["v"], vc, vs, ~odd)):
        got, want = got[skip].double(), want[skip].double()
        assert torch.isfinite(got).all()
        # half a step, and the last half step of the binade cut: as much again
        assert ((got - want).abs() <= want.abs() * 2.0 ** -4 * (1 + 2.0 ** -10)).all()
        rows = values(cache, scale)[at // page, at % page]
        assert torch.equal(rows[skip].nan_to_num(0), got)
    assert (ks[at // page, at % page][0] == 247).all()                   # e = 120
    assert (ko[0].abs().amax(-1) == 1.875 * 2.0 ** 127).all()


def test_values_of_others_read_as_they_are():
    """A cache may hold 2^128 and more all the same: infinity in fp32 and bf16."""
    kc = torch.full((1, 16, 1, 64), 448.0, device=DEV).to(F8)
    s = torch.full((1, 16, 1), 254, device=DEV, dtype=torch.uint8)
    for dtype in (F32, BF16):
        ko, vo = (torch.zeros(1, 1, 64, device=DEV, dtype=dtype) for _ in range(2))
        ops.kv_cache_read_q8(kc, kc, s, s, torch.zeros(1, device=DEV, dtype=torch.int32), ko, vo)
        torch.cuda.synchronize()
        assert torch.isinf(ko).all() and torch.isinf(vo).all()
