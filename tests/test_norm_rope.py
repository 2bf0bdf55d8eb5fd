"""attn_norm_rope_cache against its formula in 64 bits: types, head sizes, both rotations, partial and
no rotation, no weights, padding rows, in place, both cache orders, and device-side errors."""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests._mixers import assert_close, norm_rope_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
F32, BF16 = torch.float32, torch.bfloat16


def case(seed, T, hq, hkv, D, rot, dtype, page=16, heads_first=False, max_pos=50):
    g = synth.generator(seed, DEV)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    x = rnd(T, (hq + 2 * hkv) * D + 16).to(dtype)
    q, k, v, _ = x.split([hq * D, hkv * D, hkv * D, 16], 1)
    pages = T // page + 3
    shape = (pages, hkv, page, D) if heads_first else (pages, page, hkv, D)
    kc, vc = (rnd(*shape).to(dtype) for _ in range(2))
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    c = dict(q=q.unflatten(1, (hq, D)), k=k.unflatten(1, (hkv, D)), v=v.unflatten(1, (hkv, D)),
             qw=(1 + 0.2 * rnd(D)).to(dtype), kw=(1 + 0.2 * rnd(D)).to(dtype),
             cs=rnd(max_pos, rot), pos=torch.randint(0, max_pos, (T,), generator=g, device=DEV,
                                                     dtype=torch.int32),
             kc=kc, vc=vc,
             slots=torch.randperm(pages * page, generator=g, device=DEV)[:T].to(torch.int32))
    return c


def check(c, pairs, weights=True, in_place=False, eps=1e-5):
    qw, kw = (c["qw"], c["kw"]) if weights else (None, None)
    cpu = {n: t.cpu() for n, t in c.items()}
    want_q = norm_rope_ref(cpu["q"], qw.cpu() if weights else None, eps, cpu["cs"], cpu["pos"], pairs)
    want_k = norm_rope_ref(cpu["k"], kw.cpu() if weights else None, eps, cpu["cs"], cpu["pos"], pairs)
    page = c["kc"].shape[1]
    kc, vc = cpu["kc"].double(), cpu["vc"].clone()
    for t, s in enumerate(cpu["slots"].tolist()):
        if s >= 0:
            kc[s // page, s % page] = want_k[t]
            vc[s // page, s % page] = cpu["v"][t]
    q_out = c["q"] if in_place else torch.zeros(c["q"].shape, device=DEV, dtype=c["q"].dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.attn_norm_rope_cache(c["q"], c["k"], c["v"], qw, kw, eps, c["cs"], c["pos"], pairs, c["kc"],
                             c["vc"], c["slots"], q_out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert_close(q_out, want_q, "q")
    assert_close(c["kc"], kc, "k cache")
    assert torch.equal(c["vc"].cpu(), vc)
    kept = torch.ones(kc.shape[0] * page, dtype=torch.bool)
    kept[[s for s in cpu["slots"].tolist() if s >= 0]] = False
    assert torch.equal(c["kc"].cpu().flatten(0, 1)[kept], cpu["kc"].flatten(0, 1)[kept])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 16), (128, 128), (128, 64), (256, 256), (256, 64),
                                   (128, 0)])
@pytest.mark.parametrize("pairs", [False, True])
def test_types_sizes_rotations(dtype, D, rot, pairs):
    check(case(1, 7, 5, 3, D, rot, dtype), pairs)


@pytest.mark.parametrize("T,hq,hkv", [(1, 16, 4), (33, 1, 1), (2500, 2, 1), (130, 8, 8)])
def test_tokens_and_heads(T, hq, hkv):
    check(case(2, T, hq, hkv, 128, 8 * 4, BF16), False)


def test_pairs_rotate_any_even_part():
    check(case(3, 5, 2, 1, 64, 6, BF16), True)


def test_without_weights_there_is_no_norm():
    check(case(4, 9, 4, 2, 128, 128, BF16), False, weights=False)


def test_padding_rows_in_place_and_heads_first_cache():
    c = case(5, 21, 4, 2, 128, 64, BF16, page=7, heads_first=True)
    c["slots"][::4] = -1
    check(c, False, in_place=True)


def test_zero_heads_stay_zero():
    c = case(6, 3, 2, 1, 64, 64, F32)
    c["q"].zero_()
    check(c, True, eps=1e-6)


def test_positions_and_slots_out_of_range_skip_the_token():
    for name, value in (("pos", 50), ("pos", -1), ("slots", 10 ** 6)):
        c = case(7, 6, 2, 1, 64, 64, BF16)
        c[name][2] = value
        out = torch.full(c["q"].shape, 7.0, device=DEV, dtype=BF16)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        before = c["kc"].clone()
        ops.attn_norm_rope_cache(c["q"], c["k"], c["v"], c["qw"], c["kw"], 1e-6, c["cs"], c["pos"],
                                 False, c["kc"], c["vc"], c["slots"], out, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == ops.DERR_POSITION
        assert (out[2] == 7).all() and not (out[[0, 1, 3, 4, 5]] == 7).any(-1).any()
        assert (c["kc"] != before).any(-1).any(-1).sum() == 5
