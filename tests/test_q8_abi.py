"""What the operators over a cache in 8 bits refuse: argument checks of the C entry points with fake pointers
(nothing is launched; only where there is no GPU), and the binding's own checks."""
import pytest
import torch

from state_cached_causal_gb300 import build as cbuild
from state_cached_causal_gb300 import ops
from tests.test_mixer_abi import FAKE, _Placed, _two, no_gpu

F8, U8 = torch.float8_e4m3fn, torch.uint8


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return ops.load()


def cache(k=FAKE, v=FAKE, page=16 * 2 * 128, tok=2 * 128, head=128, ks=FAKE + 1, vs=FAKE + 3, cp=32, ct=2, ch=1,
          pages=4, size=16, heads=2, dim=128):
    return ops.KvCacheQ8(k, v, page, tok, head, ks, vs, cp, ct, ch, pages, size, heads, dim)


BAD_CACHE = [(dict(c=cache(k=None)), -1), (dict(c=cache(v=FAKE + 8)), -1), (dict(c=cache(ks=None)), -1),
             (dict(c=cache(vs=None)), -1), (dict(c=cache(page=0)), -1), (dict(c=cache(tok=8)), -1),
             (dict(c=cache(head=-128)), -1), (dict(c=cache(cp=0)), -1), (dict(c=cache(ct=-2)), -1),
             (dict(c=cache(ch=0)), -1), (dict(c=cache(pages=0)), -1), (dict(c=cache(size=0)), -1),
             (dict(c=cache(heads=0)), -1), (dict(c=cache(dim=96)), -2)]


@pytest.mark.parametrize("kw,want", BAD_CACHE + [
    (dict(q=None), -1), (dict(qs=500), -1), (dict(k=FAKE + 2), -1), (dict(vs=128), -1), (dict(o=None), -1),
    (dict(os=516), -1), (dict(qw=FAKE + 1), -1), (dict(eps=-1.0), -1), (dict(cs=None), -1), (dict(mp=0), -1),
    (dict(rot=130), -1), (dict(rot=24), -1), (dict(pos=None), -1), (dict(sl=None), -1), (dict(T=-1), -1),
    (dict(hq=0), -1), (dict(dt=9), -1), (dict(T=0), 0), (dict(), -3)])
@no_gpu
def test_norm_arguments(lib, kw, want):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, qw=FAKE, kw=FAKE, eps=1e-6, cs=FAKE, mp=10, rot=128,
             il=0, pos=FAKE, c=cache(), sl=FAKE, T=3, hq=4, dt=1, o=FAKE, os=512)
    a.update(kw)
    assert lib.attn_norm_rope_cache_q8(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"], a["eps"], a["cs"], a["mp"], a["rot"],
        a["il"], a["pos"], a["c"], a["sl"], a["T"], a["hq"], a["dt"], a["o"], a["os"], None, None) == want


@pytest.mark.parametrize("kw,want", BAD_CACHE + [
    (dict(sl=None), -1), (dict(T=-1), -1), (dict(T=0), 0), (dict(dt=2), -1), (dict(ko=None), -1),
    (dict(vo=FAKE + 4), -1), (dict(kos=252), -1), (dict(vos=128), -1), (dict(), -3)])
@no_gpu
def test_read_arguments(lib, kw, want):
    a = dict(c=cache(), sl=FAKE, T=3, dt=1, ko=FAKE, kos=256, vo=FAKE, vos=256)
    a.update(kw)
    assert lib.kv_cache_read_q8(a["c"], a["sl"], a["T"], a["dt"], a["ko"], a["kos"], a["vo"], a["vos"], None,
                                None) == want


@pytest.mark.parametrize("kw,want", BAD_CACHE + [
    (dict(q=None), -1), (dict(qs=128), -1), (dict(o=FAKE + 2), -1), (dict(os=513), -1), (dict(bt=None), -1),
    (dict(bts=4), -1), (dict(w=-1), -1), (dict(w=2 ** 28, bts=2 ** 28), -1), (dict(sl=None), -1), (dict(B=-1), -1),
    (dict(B=2 ** 30), -1), (dict(ns=-1), -1), (dict(ns=8), -2), (dict(hq=5), -1), (dict(hq=0), -1),
    (dict(hq=34, ns=3), -2), (dict(dt=4), -1), (dict(B=0), 0), (dict(), -3)])
@no_gpu
def test_attn_arguments(lib, kw, want):
    a = dict(q=FAKE, qs=512, c=cache(), bt=FAKE, bts=5, w=5, sl=FAKE, B=3, ns=0, hq=4, dt=1, o=FAKE, os=512,
             lse=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    assert lib.attn_decode_q8(a["q"], a["qs"], a["c"], a["bt"], a["bts"], a["w"], a["sl"], a["B"], a["ns"], a["hq"],
                              0.1, a["dt"], a["o"], a["os"], a["lse"], a["ws"], a["wsb"], None, None) == want


def _calls():
    _, norm, attn, i = _two()
    c, s = torch.zeros(5, 16, 2, 64, dtype=U8).view(F8), torch.zeros(5, 16, 2, dtype=U8)
    q8 = dict(k_cache=c, v_cache=c, k_scale=s, v_scale=s)
    rows = torch.zeros(4, 2, 64)
    return ({**norm, **q8}, dict(q8, slot_mapping=i(4), k_out=rows, v_out=rows), {**attn, **q8}, q8, i)


def test_binding_checks():
    norm, read, attn, q8, i = _calls()
    c, s = q8["k_cache"], q8["k_scale"]
    bad_cache = [(dict(k_cache=c.view(U8)), TypeError), (dict(v_cache=c.float()), TypeError),
                 (dict(k_scale=s.to(torch.int32)), TypeError), (dict(v_scale=s.float()), TypeError),
                 (dict(v_cache=c[:, :, :1]), ValueError), (dict(k_cache=c[:4], v_cache=c[:4]), ValueError),
                 (dict(k_scale=s[:, :8]), ValueError), (dict(v_scale=s.transpose(0, 1)), ValueError),
                 (dict(v_scale=s.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                 (dict(v_cache=torch.zeros(5, 2, 16, 64, dtype=U8).view(F8).transpose(1, 2)), ValueError)]
    for fn, call, more in (
            (ops.attn_norm_rope_cache_q8, norm, [
                (dict(positions=i(4).long()), TypeError), (dict(k=norm["q"]), ValueError),
                (dict(q_weight=torch.zeros(32)), ValueError), (dict(slot_mapping=i(3)), ValueError),
                (dict(slot_mapping=i(8)[::2]), ValueError), (dict(q=norm["q"].half()), TypeError)]),
            (ops.kv_cache_read_q8, read, [
                (dict(slot_mapping=i(4).long()), TypeError), (dict(slot_mapping=i(8)[::2]), ValueError),
                (dict(slot_mapping=i(5)), ValueError), (dict(k_out=read["k_out"][:3]), ValueError),
                (dict(v_out=read["v_out"].bfloat16()), TypeError), (dict(v_out=read["v_out"][:, :1]), ValueError),
                (dict(k_out=read["k_out"].half(), v_out=read["v_out"].half()), TypeError)]),
            (ops.attn_decode_q8, attn, [
                (dict(seq_lens=i(4).long()), TypeError), (dict(out=read["k_out"]), ValueError),
                (dict(n_spec=1), ValueError), (dict(block_table=i(3, 3)), ValueError),
                (dict(seq_lens=i(4, 2)[:, 0]), ValueError),
                (dict(workspace=torch.zeros(64, 64, dtype=U8).t()), ValueError)])):
        for bad, err in bad_cache + more + [(dict(dev_err=torch.zeros(4, dtype=U8)), TypeError),
                                            (dict(dev_err=i(0)), ValueError)]:
            with pytest.raises(err):
                fn(**{**call, **bad})
        with pytest.raises(ValueError, match="must live on the GPU"):
            fn(**call)


@no_gpu
@pytest.mark.parametrize("in_c", [True, False])
def test_both_marshallings_reach_the_library(in_c, monkeypatch):
    """With tensors that say they are on the current device both get as far as the launch, which fails here; one
    on another device is refused."""
    lib = ops.load()
    if in_c and ops._fast is None:
        pytest.skip("the C module is not built")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda stream: None)
    seen = []
    if in_c:
        ops._fast.init(lib._handle, (torch.float32, torch.bfloat16, torch.int32, U8, torch.bool, F8,
                                     torch.float8_e8m0fnu), lambda d: seen.append(d) or 0, None, lambda: 0)
    else:
        monkeypatch.setattr(ops, "_fast", None)
    norm, read, attn, q8, i = _calls()
    attn = dict(attn, workspace=torch.zeros(1 << 26, dtype=U8), lse=torch.zeros(4, 4))
    try:
        for fn, call in (("attn_norm_rope_cache_q8", norm), ("kv_cache_read_q8", read), ("attn_decode_q8", attn)):
            for scales in (q8["k_scale"], q8["k_scale"].view(torch.float8_e8m0fnu)):
                call = dict(call, k_scale=scales, dev_err=i(1))
                tensors = [n for n, t in call.items() if torch.is_tensor(t)]
                here = {n: _Placed(t) if n in tensors else t for n, t in call.items()}
                with pytest.raises(ops.CConvError, match=fn):
                    getattr(ops, fn)(**here)
                assert not in_c or seen.pop() == 0
                for n in tensors:
                    with pytest.raises(ValueError, match="current device"):
                        getattr(ops, fn)(**{**here, n: _Placed(call[n], 1)})
                assert not seen
    finally:
        ops._load_fast(lib)
