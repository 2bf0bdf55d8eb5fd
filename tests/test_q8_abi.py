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
    groups = dict(cu_groups=i(3), prefix_lens=i(2))
    shared = dict(attn, q=attn["q"].bfloat16(), out=attn["out"].bfloat16(), **groups)
    plain = {k: v for k, v in shared.items() if not k.endswith("_scale")}
    plain.update(k_cache=torch.zeros(5, 16, 2, 64).bfloat16(), v_cache=torch.zeros(5, 16, 2, 64).bfloat16())
    try:
        for fn, call in (("attn_norm_rope_cache_q8", norm), ("kv_cache_read_q8", read), ("attn_decode_q8", attn),
                         ("attn_decode_shared_q8", shared), ("attn_decode_shared", plain)):
            for scales in (q8["k_scale"], q8["k_scale"].view(torch.float8_e8m0fnu)):
                call = dict(call, dev_err=i(1), **(dict(k_scale=scales) if "k_scale" in call else {}))
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


# ---- attention of groups that share a prefix ----------------------------------------

def _kv(c):
    return ops.KvCache(c.k, c.v, c.s_page, c.s_token, c.s_head, c.num_pages, c.page_size, c.num_kv_heads,
                       c.head_dim, 1)


SHARED = [(dict(q=None), -1), (dict(qs=128), -1), (dict(o=FAKE + 2), -1), (dict(os=513), -1), (dict(bt=None), -1),
          (dict(bts=4), -1), (dict(w=-1), -1), (dict(w=2 ** 28, bts=2 ** 28), -1), (dict(sl=None), -1),
          (dict(cu=None), -1), (dict(pl=None), -1), (dict(G=-1), -1), (dict(G=4), -1), (dict(B=-1, G=0), -1),
          (dict(B=2 ** 30), -1), (dict(ns=-1), -1), (dict(ns=8), -2), (dict(hq=5), -1), (dict(hq=0), -1),
          (dict(hq=34, ns=3), -2), (dict(dt=0), -2), (dict(dt=4), -1), (dict(B=0, G=0), 0), (dict(), -3),
          (dict(G=0, cu=None, pl=None), -3)]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,want", SHARED)
@no_gpu
def test_shared_arguments(lib, kw, want, q8):
    a = dict(q=FAKE, qs=512, c=cache(), bt=FAKE, bts=5, w=5, sl=FAKE, B=3, cu=FAKE, pl=FAKE, G=2, ns=0, hq=4, dt=1,
             o=FAKE, os=512, lse=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    c = a["c"] if q8 else _kv(a["c"])
    if not q8 and a["dt"] == 0:
        c.dtype = 0
    fn = lib.attn_decode_shared_q8 if q8 else lib.attn_decode_shared
    assert fn(a["q"], a["qs"], c, a["bt"], a["bts"], a["w"], a["sl"], a["B"], a["cu"], a["pl"], a["G"], a["ns"],
              a["hq"], 0.1, a["dt"], a["o"], a["os"], a["lse"], a["ws"], a["wsb"], None, None) == want


@pytest.mark.parametrize("kw,want", BAD_CACHE)
@no_gpu
def test_shared_caches(lib, kw, want):
    for q8 in (True, False):
        if not q8 and kw["c"].k == FAKE and kw["c"].v == FAKE and want == -1 and (
                not kw["c"].k_scale or not kw["c"].v_scale or min(kw["c"].c_page, kw["c"].c_token,
                                                                   kw["c"].c_head) <= 0):
            continue                                    # (only scales are wrong)
        c = kw["c"] if q8 else _kv(kw["c"])
        if not q8 and c.s_token == 8:
            continue                                    # (16 bytes of bf16)
        fn = lib.attn_decode_shared_q8 if q8 else lib.attn_decode_shared
        assert fn(FAKE, 512, c, FAKE, 5, 5, FAKE, 3, FAKE, FAKE, 2, 0, 4, 0.1, 1, FAKE, 512, None, FAKE, 1 << 40,
                  None, None) == want


@no_gpu
def test_shared_workspace_sizes_are_checked(lib):
    f = lib.attn_decode_shared_workspace_bytes
    assert f(-1, 0, 0, 4, 2, 128) == -1 and f(1, 0, 0, 5, 2, 128) == -1 and f(2, 3, 0, 4, 2, 128) == -1
    assert f(2, -1, 0, 4, 2, 128) == -1 and f(1, 0, 9, 4, 2, 128) == -2 and f(1, 1, 0, 4, 2, 80) == -2


def test_shared_binding_checks(monkeypatch):
    _, _, attn, q8, i = _calls()
    plain = {k: v for k, v in _two()[2].items()}
    bf = lambda t: t.bfloat16() if t.dtype == torch.float32 else t      # noqa: E731
    plain = {k: bf(v) if torch.is_tensor(v) else v for k, v in plain.items()}
    attn = {k: bf(v) if torch.is_tensor(v) and k in ("q", "out") else v for k, v in attn.items()}
    groups = dict(cu_groups=i(3), prefix_lens=i(2))
    for fn, call in ((ops.attn_decode_shared, {**plain, **groups}), (ops.attn_decode_shared_q8, {**attn, **groups})):
        for bad, err in ((dict(cu_groups=i(3).long()), TypeError), (dict(prefix_lens=i(2).float()), TypeError),
                         (dict(cu_groups=i(2)), ValueError), (dict(cu_groups=i(4)), ValueError),
                         (dict(cu_groups=i(6)[::2]), ValueError), (dict(prefix_lens=i(2, 2)[:, 0]), ValueError),
                         (dict(seq_lens=i(4).long()), TypeError), (dict(block_table=i(3, 3)), ValueError),
                         (dict(dev_err=i(0)), ValueError), (dict(workspace=torch.zeros(64, 64, dtype=U8).t()),
                                                            ValueError)):
            with pytest.raises(err):
                fn(**{**call, **bad})
        with pytest.raises(ValueError, match="must live on the GPU"):
            fn(**call)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["norm", "read", "attn", "attn32", "shared", "shared8"])
def test_both_marshallings_agree(what, monkeypatch):
    """The C module serves these calls, and Python's marshalling gives the same results."""
    from tests import _q8
    from tests.test_attn_shared import Case
    ops.load()
    if ops._fast is None:
        pytest.skip("the C module is not built")
    dev, dt = torch.device("cuda"), torch.float32 if what == "attn32" else torch.bfloat16
    c = _q8.case(3, [40, 7, 100], 4, 2, 64, 16, 1, dt)
    q, kc, vc, ks, vs, table, lens = c
    sh = Case(4, [(40, [50, 60, 41])], 4, 2, 64, 16, 1, what == "shared8")
    cos = torch.randn(32, 64, device=dev)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)       # noqa: E731
    rows = torch.randn(3, 2, 64, device=dev).to(dt)

    def call():
        caches = [t.view(U8).clone() for t in (kc, vc, ks, vs)]
        k, v = (t.view(F8) for t in caches[:2])
        out, lse = torch.zeros_like(q, memory_format=torch.contiguous_format), torch.zeros(3, 4, device=dev)
        back = [torch.zeros(3, 2, 64, device=dev, dtype=dt) for _ in range(2)]
        if what == "norm":
            ops.attn_norm_rope_cache_q8(q, rows, rows, None, rows[0, 0] * 0 + 1, 1e-6, cos, i(1, 2, 3), True, k, v,
                                        *caches[2:], i(5, -1, 30), out)
        elif what == "read":
            ops.kv_cache_read_q8(k, v, *caches[2:], i(3, -1, 17), *back)
        elif what.startswith("shared"):
            out = torch.zeros_like(sh.q, memory_format=torch.contiguous_format)
            sh.call(out, lse)
        else:
            ops.attn_decode_q8(q, k, v, *caches[2:], table, lens, 0, 0.125, out, lse)
        torch.cuda.synchronize()
        return [*caches, out, lse, *back]

    served, real = [], ops._fast

    class Spy:
        def __getattr__(self, n):
            return lambda *x: served.append(getattr(real, n)(*x)) or served[-1]

    monkeypatch.setattr(ops, "_fast", Spy())
    one = call()
    assert served == [0]
    monkeypatch.setattr(ops, "_fast", None)
    for a, b in zip(one, call()):
        assert torch.equal(a, b)
