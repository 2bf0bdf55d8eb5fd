"""Attention over a cache in 8 bits whose scale bytes are not the least ones of their rows: any byte from 1 to 254
may stand with any values, as one scale for a whole cache or for all its positions does. Rows of zeros and of the
smallest values under large powers of two, rows of any size under one power, sinks without a value.

Tolerances as tests/test_q8_attn.py derives them: weights enter with 11 bits of themselves, whatever the bytes.
"""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests._mixers import assert_close
from tests._q8 import DEV, F8, case
from tests.test_attn_shared import Case
from tests.test_q8_attn import check

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
heads = pytest.mark.parametrize("hq,hkv,D", [(4, 1, 64), (16, 4, 128), (16, 1, 128), (12, 2, 128), (4, 2, 256)])


def row(c, table, b, j, page=16):
    """Position j of request b."""
    return int(table[b, j // page]), j % page


def powers(g, shape, low):
    """Values of +-2^x, x from `low` to low + 3: exact in e4m3 from 2^-9 to 2^8, whatever the shift."""
    x = torch.randint(0, 4, shape, generator=g, device=DEV) + low
    return (torch.exp2(x.float()) * (1 - 2 * torch.randint(0, 2, shape, generator=g, device=DEV))).to(F8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@heads
@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("byte", [125, 150, 200, 254])
def test_rows_of_zeros_under_large_powers(dtype, hq, hkv, D, n, byte):
    if hq // hkv * n > 64:
        pytest.skip("more rows than a call takes")
    c = case(1, [200, 33], hq, hkv, D, 16, n, dtype)
    for b, j in ((0, 3), (0, 40), (0, 77), (0, 199 - n), (1, 20)):
        at = row(c, c[5], b, j)
        c[2].view(torch.uint8)[at] = 0
        c[4][at] = byte
    assert check(*c, n) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@heads
def test_small_bytes_under_large_powers(dtype, hq, hkv, D):
    """Rows of one real size, as bytes from 2^-9 .. 2^-6 to 2^5 .. 2^8."""
    c = case(2, [300, 7, 64], hq, hkv, D, 16, 1, dtype)
    g = synth.generator(3, DEV)
    shift = torch.randint(0, 15, c[4].shape, generator=g, device=DEV)
    v = powers(g, c[2].shape, 5)
    v = (v.float() * torch.exp2(-shift.float())[..., None]).to(F8)
    keep = c[4] != 255                              # (rows that nobody holds are NaN)
    c[2].view(torch.uint8)[keep] = v.view(torch.uint8)[keep]
    c[4][keep] = (100 + shift).to(torch.uint8)[keep]
    assert check(*c, 1) == 0
    # and the position of the largest scores the smallest bytes of all
    at = row(c, c[5], 0, 150)
    c[1].view(torch.uint8)[at] = 0x7e
    c[2].view(torch.uint8)[at] = 0x01
    c[4][at] = 117
    q = c[0].abs()
    assert check(q, *c[1:], 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@heads
@pytest.mark.parametrize("byte", [60, 119, 127])
def test_one_scale_for_all_rows(dtype, hq, hkv, D, byte):
    """Rows from 2^-9 to 448, some of them zeros, under one power of two."""
    c = case(4, [500, 31], hq, hkv, D, 16, 1, dtype)
    g = synth.generator(5, DEV)
    low = torch.randint(-9, 6, (*c[4].shape, 1), generator=g, device=DEV).float()
    v = (powers(g, c[2].shape, 0).float() * torch.exp2(low)).to(F8)
    v.view(torch.uint8)[torch.rand(c[4].shape, generator=g, device=DEV) < 0.1] = 0
    keep = c[4] != 255
    c[2].view(torch.uint8)[keep] = v.view(torch.uint8)[keep]
    c[4][keep] = byte
    assert check(*c, 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@heads
@pytest.mark.parametrize("place", [0, 9, 170])
@pytest.mark.parametrize("byte", [1, 119, 254])
def test_a_sink_without_a_value(dtype, hq, hkv, D, place, byte):
    """A position that takes nearly all of the weight (2^30 and more of the others') and holds zeros: the result is
    the others', at their own precision."""
    c = case(6, [180], hq, hkv, D, 16, 1, dtype)
    c[3][c[3] != 255] -= 4                          # (their scores: 0 +- 2, 5 at most)
    q = c[0].abs() + 0.5                            # (all of one sign)
    at = row(c, c[5], 0, place)
    c[1].view(torch.uint8)[at] = 0x7e               # 448 in every dim, against means of zero
    c[3][at] = 127 - 9
    c[2].view(torch.uint8)[at] = 0
    c[4][at] = byte
    # the sink's score: 30 times q's mean, 1.3, times 0.875
    assert check(q.to(dtype), *c[1:], 1, scale=30.0 / D) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@heads
def test_sinks_each_above_the_one_before(dtype, hq, hkv, D):
    """Positions without a value whose scores rise by 2^14 from one to the next: none of them takes the others' weights
    away, however many there are."""
    c = case(9, [200], hq, hkv, D, 16, 1, dtype)
    c[3][c[3] != 255] -= 4                          # (the others' scores: 0 +- 2)
    q = (c[0].abs() + 0.5).to(dtype)
    for j, (k, byte) in zip((10, 40, 72, 104, 136, 168), ((0x70, 118), (0x78, 118), (0x7c, 118), (0x78, 119), (0x7a, 119),
                                                        (0x7c, 119))):
        at = row(c, c[5], 0, j)                     # 128, 256, 384, 512, 640, 768 times 2^-9
        c[1].view(torch.uint8)[at] = k
        c[3][at] = byte
        c[2].view(torch.uint8)[at] = 0
        c[4][at] = 119
    assert check(q, *c[1:], 1, scale=30.0 / D) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_behind_a_shared_prefix(D):
    c = Case(7, [(100, [140, 190, 101])], 8, 2, D, 16, 1, True)
    for b, j in ((0, 110), (1, 100), (1, 150), (2, 100)):
        at = row(c, c.full, b, j)
        c.vc.view(torch.uint8)[at] = 0
        c.vs[at] = 254
    assert c.check() == 0


def test_nan_beside_the_smallest_bytes():
    """A NaN is no size of its row, and stays one when the row is brought to another power of two."""
    q, kc, vc, ks, vs, table, lens = case(8, [90], 4, 1, 64, 16, 1, BF16)
    at = row(None, table, 0, 5)
    vc.view(torch.uint8)[at] = 0x02
    vc.view(torch.uint8)[at[0], at[1], 0, 7] = 0xff
    vs[at] = 254 - 20
    ks[at] = 100
    out = torch.zeros(q.shape, device=DEV, dtype=BF16)
    ops.attn_decode_q8(q, kc, vc, ks, vs, table, lens, 0, 0.125, out)
    torch.cuda.synchronize()
    assert torch.isnan(out[..., 7]).all() and torch.isfinite(out[..., :7]).all() and torch.isfinite(out[..., 8:]).all()
    want = torch.full((1, 4, 56), 2.0 ** -8 * 2.0 ** (234 - 127), dtype=torch.float64)     # nothing else counts
    s = (q.double().cpu() * 0.125)
    k = kc.double().cpu() * torch.exp2(ks.double().cpu() - 127)[..., None]
    rows = torch.stack([k[row(None, table, 0, j)][0] for j in range(90)])
    w = torch.softmax(torch.einsum("bhd,jd->bhj", s, rows), -1)[..., 5:6]
    assert_close(out[..., 8:].cpu(), want * w, "the others")
