"""The paged cache in 8 bits written and read back, against 64 bits: attn_norm_rope_cache_q8 (types, head sizes,
rotations, strides, padding rows, rows of zeros, tiny, huge, with infinities and NaN, device-side errors) and
kv_cache_read_q8.

A written value is off by half a step of e4m3 at most: 2^-4 of itself, or 2^-10 of the row's power of two
where it is below the least normal value (2^-6); before that the fp32 norm and rotation are off by a few 2^-24
of the row's largest value (a sum of squares of up to 256 terms, a division, a product of three, a sum of two:
16 * 2^-24 bounds them).
"""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests._mixers import assert_close, norm_rope_ref
from tests._q8 import DEV, F8, cache_pair, quantised, scale_byte, values
from tests.test_norm_rope import case

pytestmark = pytest.mark.gpu
F32, BF16, E8 = torch.float32, torch.bfloat16, torch.float8_e8m0fnu


def written(got, byte, want, what):
    """got, byte: rows of bytes and their scales; want: the rows in 64 bits (finite)."""
    got, byte = got.cpu(), byte.cpu()
    m = want.abs().amax(-1)
    near = torch.tensor([scale_byte(v) for v in m.flatten().tolist()]).view(m.shape)
    other = torch.zeros_like(near)
    for f in (1 - 2e-6, 1 + 2e-6):              # a largest value next to a border: either byte
        other = torch.where(byte == torch.tensor([scale_byte(v * f) for v in m.flatten().tolist()])
                            .view(m.shape), 1, other)
    assert ((byte == near) | (other == 1)).all(), f"{what}: scales"
    unit = torch.exp2(byte.double() - 127)[..., None]
    off = (values(got, byte) - want).abs()
    half = torch.maximum(want.abs() * 2.0 ** -4, unit * 2.0 ** -10)
    assert (off <= half * (1 + 2.0 ** -10) + 16 * 2.0 ** -24 * m[..., None]).all(), what


def check(c, pairs, weights=True, eps=1e-5, heads_first=False):
    g = synth.generator(9, DEV)
    kc, vc, ks, vs = cache_pair(g, tuple(c["kc"].shape), heads_first)
    before = [t.cpu().view(torch.uint8).clone() for t in (kc, vc, ks, vs)]
    qw, kw = (c["qw"], c["kw"]) if weights else (None, None)
    cpu = {n: t.cpu() for n, t in c.items()}
    want_q = norm_rope_ref(cpu["q"], qw.cpu() if weights else None, eps, cpu["cs"], cpu["pos"], pairs)
    want_k = norm_rope_ref(cpu["k"], kw.cpu() if weights else None, eps, cpu["cs"], cpu["pos"], pairs)
    q_out = torch.zeros(c["q"].shape, device=DEV, dtype=c["q"].dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.attn_norm_rope_cache_q8(c["q"], c["k"], c["v"], qw, kw, eps, c["cs"], c["pos"], pairs, kc, vc, ks, vs,
                                c["slots"], q_out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert_close(q_out, want_q, "q")
    slots = cpu["slots"].long()
    rows = torch.nonzero(slots >= 0)[:, 0]
    at = slots[rows]
    page = kc.shape[1]
    pick = lambda t: t.cpu().view(torch.uint8)[at // page, at % page]        # noqa: E731
    written(pick(kc).view(F8), pick(ks), want_k[rows], "k")
    written(pick(vc).view(F8), pick(vs), cpu["v"].double()[rows], "v")
    kept = torch.ones(kc.shape[0], page, dtype=torch.bool)
    kept[at // page, at % page] = False
    for t, old in zip((kc, vc, ks, vs), before):
        assert torch.equal(t.cpu().view(torch.uint8)[kept], old[kept])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (256, 256), (256, 64), (128, 0)])
@pytest.mark.parametrize("pairs", [False, True])
def test_types_sizes_rotations(dtype, D, rot, pairs):
    check(case(1, 7, 5, 3, D, rot, dtype), pairs)


@pytest.mark.parametrize("T,hq,hkv", [(1, 16, 4), (33, 1, 1), (2500, 2, 1), (130, 8, 8), (700, 3, 3)])
def test_tokens_and_heads(T, hq, hkv):
    check(case(2, T, hq, hkv, 128, 8 * 4, BF16), False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_padding_rows_without_weights_and_heads_first(dtype):
    c = case(5, 21, 4, 2, 128, 64, dtype, page=7)
    c["slots"][::4] = -1
    check(c, False, weights=False, heads_first=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_every_size(dtype):
    """Rows of zeros, of the smallest and the largest values, of a power of two, and at the border of one."""
    c = case(6, 9, 2, 2, 64, 64, dtype)
    c["cs"][:, :32], c["cs"][:, 32:] = 1, 0                      # no rotation: k is written as it is
    for i, f in enumerate((0.0, 2.0 ** -130, 2.0 ** -122, 2.0 ** 120, 1.0, 448.0, 449.0, 2.0 ** -60, 2.0 ** 60)):
        x = torch.linspace(-1, 1, 64, device=DEV) * f
        c["k"][i], c["v"][i] = x.to(dtype), x.flip(0).to(dtype)
    check(c, False, weights=False)


def test_infinities_and_nan_are_nan_and_leave_the_scale():
    c = case(7, 6, 2, 2, 64, 0, F32)
    want = c["v"].clone()
    for i, x in enumerate((float("inf"), float("-inf"), float("nan"))):
        c["v"][i, :, 5 + i] = x
        want[i, :, 5 + i] = 0
    c["v"][3] = float("inf")
    kc, vc, ks, vs = cache_pair(synth.generator(8, DEV), tuple(c["kc"].shape))
    ops.attn_norm_rope_cache_q8(c["q"], c["k"], c["v"], None, None, 1e-6, c["cs"], c["pos"], False, kc, vc, ks, vs,
                                c["slots"], torch.zeros_like(c["q"]))
    at = c["slots"].long()
    page = kc.shape[1]
    got = vc.view(torch.uint8)[at // page, at % page].view(F8).float()
    nan = torch.isnan(got)
    assert nan[3].all() and torch.equal(nan[:3], ~torch.isfinite(c["v"][:3])) and not nan[4:].any()
    fin = torch.tensor([0, 1, 2, 4, 5], device=DEV)
    byte = vs[at // page, at % page][fin].cpu()
    assert torch.equal(byte, quantised(want[fin].cpu().double())[1])


def test_positions_and_slots_out_of_range_skip_the_token():
    for name, value in (("pos", 50), ("pos", -1), ("slots", 10 ** 6)):
        c = case(7, 6, 2, 1, 64, 64, BF16)
        c[name][2] = value
        kc, vc, ks, vs = cache_pair(synth.generator(8, DEV), tuple(c["kc"].shape))
        old = kc.view(torch.uint8).clone()
        out = torch.full(c["q"].shape, 7.0, device=DEV, dtype=BF16)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ops.attn_norm_rope_cache_q8(c["q"], c["k"], c["v"], c["qw"], c["kw"], 1e-6, c["cs"], c["pos"], False,
                                    kc, vc, ks, vs, c["slots"], out, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == ops.DERR_POSITION
        assert (out[2] == 7).all() and not (out[[0, 1, 3, 4, 5]] == 7).any(-1).any()
        assert (kc.view(torch.uint8) != old).any(-1).any(-1).sum() == 5


# ---- reading back ------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hkv,D", [(1, 64), (4, 128), (3, 64), (2, 256)])
@pytest.mark.parametrize("T", [1, 77, 3000])
def test_rows_come_back(dtype, hkv, D, T):
    """In any order, some of them twice, beside padding rows and rows that are out of range; into views of
    wider rows, which keep what lies around them."""
    g = synth.generator(T, DEV)
    page, pages = 16, 40
    kc, vc, ks, vs = cache_pair(g, (pages, page, hkv, D), heads_first=T % 2 == 1, spread=20)
    slots = torch.randint(0, pages * page, (T,), generator=g, device=DEV, dtype=torch.int32)
    if T > 1:
        slots[5], slots[6], slots[T - 1] = -1, pages * page, -7
    wide = torch.full((2, T, hkv * D + 16), 7.0, device=DEV, dtype=dtype)
    ko, vo = (w[:, :hkv * D].unflatten(1, (hkv, D)) for w in wide)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.kv_cache_read_q8(kc, vc, ks, vs, slots, ko, vo, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == (ops.DERR_POSITION if T > 1 else 0)
    at = slots.long().cpu()
    ok = (at >= 0) & (at < pages * page)
    for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
        want = values(c.cpu(), s.cpu())[at[ok] // page, at[ok] % page]
        assert torch.equal(got.cpu()[ok].double(), want)            # powers of two: exact in bf16 too
        assert (got.cpu()[~ok] == 7).all()
    assert (wide[:, :, hkv * D:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hkv,D,page,T", [(20, 256, 16, 41), (9, 128, 24, 200), (33, 64, 16, 7), (17, 64, 5, 130),
                                          (1, 64, 16, 200001), (4, 128, 16, 70001)])
def test_many_heads_and_many_rows_come_back(dtype, hkv, D, page, T):
    """More units of a token than a block has threads, and more rows than a launch's blocks take at a time."""
    g = synth.generator(T, DEV)
    pages = 33
    kc, vc, ks, vs = cache_pair(g, (pages, page, hkv, D), heads_first=False, spread=20)
    slots = torch.randint(0, pages * page, (T,), generator=g, device=DEV, dtype=torch.int32)
    ko, vo = (torch.full((T, hkv, D), 7.0, device=DEV, dtype=dtype) for _ in range(2))
    ops.kv_cache_read_q8(kc, vc, ks, vs, slots, ko, vo)
    for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
        rows = values(c.cpu(), s.cpu()).to(dtype).to(DEV).flatten(0, 1)          # powers of two: exact in bf16 too
        assert torch.equal(got, rows[slots.long()])


def test_what_is_written_comes_back():
    c = case(11, 50, 4, 2, 128, 64, BF16)
    kc, vc, ks, vs = cache_pair(synth.generator(8, DEV), tuple(c["kc"].shape))
    ops.attn_norm_rope_cache_q8(c["q"], c["k"], c["v"], c["qw"], c["kw"], 1e-6, c["cs"], c["pos"], False, kc, vc,
                                ks.view(E8), vs.view(E8), c["slots"], torch.zeros_like(c["q"]))
    ko, vo = (torch.zeros(c["k"].shape, device=DEV, dtype=BF16) for _ in range(2))
    ops.kv_cache_read_q8(kc, vc, ks.view(E8), vs, c["slots"], ko, vo)
    torch.cuda.synchronize()
    want = norm_rope_ref(c["k"].cpu(), c["kw"].cpu(), 1e-6, c["cs"].cpu(), c["pos"].cpu(), False)
    for got, w in ((ko, want), (vo, c["v"].cpu().double())):
        m = w.abs().amax(-1, keepdim=True)
        # half a step, or that of values under 2^-6 of the power of two (2^-10 of at most m / 224)
        assert ((got.cpu().double() - w).abs() <= (w.abs() * 2.0 ** -4 + m * 2.0 ** -17) * 1.001 + m * 2.0 ** -20).all()


def test_offsets_beyond_32_bits():
    """Cache rows past 2^31 bytes."""
    hkv, D, page = 8, 128, 64
    pages = 2 ** 31 // (page * hkv * D) + 4
    kc, vc = (torch.zeros(pages, page, hkv, D, device=DEV, dtype=torch.uint8).view(F8) for _ in range(2))
    ks, vs = (torch.full((pages, page, hkv), 127, device=DEV, dtype=torch.uint8) for _ in range(2))
    c = case(12, 100, 8, hkv, D, 64, BF16)
    slots = torch.arange(100, device=DEV, dtype=torch.int32) + (pages * page - 100)
    ops.attn_norm_rope_cache_q8(c["q"], c["k"], c["v"], c["qw"], c["kw"], 1e-6, c["cs"], c["pos"], False, kc, vc,
                                ks, vs, slots, torch.zeros_like(c["q"]))
    ko, vo = (torch.zeros(100, hkv, D, device=DEV, dtype=F32) for _ in range(2))
    ops.kv_cache_read_q8(kc, vc, ks, vs, slots, ko, vo)
    torch.cuda.synchronize()
    last = lambda t: t[-2:].cpu().flatten(0, 1)[-100:]                  # noqa: E731
    written(last(kc.view(torch.uint8)).view(F8), last(ks),
            norm_rope_ref(c["k"].cpu(), c["kw"].cpu(), 1e-6, c["cs"].cpu(), c["pos"].cpu(), False), "k")
    written(last(vc.view(torch.uint8)).view(F8), last(vs), c["v"].cpu().double(), "v")
    assert torch.equal(ko.cpu().double(), values(last(kc.view(torch.uint8)).view(F8), last(ks)))
    assert torch.equal(vo.cpu().double(), values(last(vc.view(torch.uint8)).view(F8), last(vs)))
    assert not kc.view(torch.uint8)[:-2].any()
