"""What the operators behind the convolutions refuse: argument checks of the C entry points with fake
pointers (nothing is launched; only where there is no GPU), and the binding's own checks."""
import ctypes

import pytest
import torch

from state_cached_causal_gb300 import build as cbuild
from state_cached_causal_gb300 import ops

FAKE = 0x10000
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: CPU-only")


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return ops.load()


def state(p=FAKE, slot=4 * 128 * 128, head=128 * 128, slots=4, dt=0):
    return ops.GdnState(p, slot, head, slots, dt)


def gdn(lib, which, **kw):
    a = dict(q=FAKE, qs=256, k=FAKE, ks=256, v=FAKE, vs=512, a=FAKE, as_=4, b=FAKE, bs=4, A=FAKE, dtb=FAKE,
             st=state(), idx=FAKE, cu=FAKE, hi=None, B=2, T=8, ns=3, na=FAKE, hk=2, hv=4, dk=128, dv=128,
             dt=1, out=FAKE, os=512)
    a.update(kw)
    head = (a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["a"], a["as_"], a["b"], a["bs"], a["A"],
            a["dtb"], a["st"], a["idx"])
    tail = (a["hk"], a["hv"], a["dk"], a["dv"], 0.1, 1, a["dt"], a["out"], a["os"], None, None)
    if which == "fwd":
        return lib.gdn_fwd_varlen(*head, a["cu"], a["hi"], a["B"], a["T"], *tail)
    return lib.gdn_update(*head, a["B"], a["ns"], a["na"], a["hi"], *tail)


BAD_GDN = [(dict(q=None), -1), (dict(k=FAKE + 2), -1), (dict(v=None), -1), (dict(out=None), -1),
           (dict(qs=255), -1), (dict(ks=128), -1), (dict(vs=508), -1), (dict(os=516), -1), (dict(a=None), -1),
           (dict(b=FAKE + 1), -1), (dict(as_=3), -1), (dict(A=None), -1), (dict(dtb=None), -1),
           (dict(st=state(p=None)), -1), (dict(st=state(p=FAKE + 4)), -1), (dict(st=state(slots=0)), -1),
           (dict(st=state(head=128)), -1), (dict(st=state(dt=3)), -1), (dict(st=state(slot=0)), -1),
           (dict(st=state(head=128 * 128 + 2)), -1), (dict(idx=None), -1), (dict(B=-1), -1), (dict(hk=0), -1),
           (dict(hv=3), -1), (dict(dk=0), -1), (dict(dk=96), -2), (dict(dv=256), -2), (dict(dt=2), -1),
           (dict(B=2 ** 30), -1), (dict(B=0), 0)]


@pytest.mark.parametrize("which", ["fwd", "update"])
@pytest.mark.parametrize("kw,want", BAD_GDN)
@no_gpu
def test_gdn_arguments(lib, which, kw, want):
    assert gdn(lib, which, **kw) == want


@no_gpu
def test_gdn_own_arguments(lib):
    assert gdn(lib, "fwd", cu=None) == -1 and gdn(lib, "fwd", T=-1) == -1
    assert gdn(lib, "update", ns=-1) == -1 and gdn(lib, "update", ns=8) == -2
    assert gdn(lib, "update", na=None) == -1
    assert gdn(lib, "fwd") == -3 and gdn(lib, "update") == -3     # a valid call without a GPU fails loudly


def cache(k=FAKE, v=FAKE, page=16 * 2 * 128, tok=2 * 128, head=128, pages=4, size=16, heads=2, dim=128, dt=1):
    return ops.KvCache(k, v, page, tok, head, pages, size, heads, dim, dt)


def norm(lib, **kw):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, qw=FAKE, kw=FAKE, eps=1e-6, cs=FAKE, mp=10, rot=128,
             il=0, pos=FAKE, c=cache(), sl=FAKE, T=3, hq=4, dt=1, o=FAKE, os=512)
    a.update(kw)
    return lib.attn_norm_rope_cache(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"], a["eps"],
                                    a["cs"], a["mp"], a["rot"], a["il"], a["pos"], a["c"], a["sl"], a["T"],
                                    a["hq"], a["dt"], a["o"], a["os"], None, None)


BAD_CACHE = [(dict(c=cache(k=None)), -1), (dict(c=cache(v=FAKE + 8)), -1), (dict(c=cache(page=0)), -1),
             (dict(c=cache(tok=4)), -1), (dict(c=cache(head=-128)), -1), (dict(c=cache(pages=0)), -1),
             (dict(c=cache(size=0)), -1), (dict(c=cache(heads=0)), -1), (dict(c=cache(dim=96)), -2),
             (dict(c=cache(dt=0)), -2), (dict(c=cache(dt=7)), -1)]


@pytest.mark.parametrize("kw,want", BAD_CACHE + [
    (dict(q=None), -1), (dict(qs=500), -1), (dict(k=FAKE + 2), -1), (dict(vs=128), -1), (dict(o=None), -1),
    (dict(os=516), -1), (dict(qw=FAKE + 1), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(cs=None), -1), (dict(mp=0), -1), (dict(rot=130), -1), (dict(rot=-2), -1), (dict(rot=7), -1),
    (dict(rot=24), -1), (dict(rot=7, il=1), -1), (dict(pos=None), -1), (dict(sl=None), -1), (dict(T=-1), -1),
    (dict(hq=0), -1), (dict(dt=9), -1), (dict(T=0), 0)])
@no_gpu
def test_norm_arguments(lib, kw, want):
    assert norm(lib, **kw) == want


def attn(lib, **kw):
    a = dict(q=FAKE, qs=512, c=cache(), bt=FAKE, bts=5, w=5, sl=FAKE, B=3, ns=0, hq=4, dt=1, o=FAKE, os=512,
             lse=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.attn_decode(a["q"], a["qs"], a["c"], a["bt"], a["bts"], a["w"], a["sl"], a["B"], a["ns"], a["hq"],
                           0.1, a["dt"], a["o"], a["os"], a["lse"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,want", BAD_CACHE + [
    (dict(q=None), -1), (dict(qs=128), -1), (dict(o=FAKE + 2), -1), (dict(os=513), -1), (dict(bt=None), -1),
    (dict(bts=4), -1), (dict(w=-1), -1), (dict(w=2 ** 28, bts=2 ** 28), -1), (dict(sl=None), -1), (dict(B=-1), -1),
    (dict(B=2 ** 30), -1), (dict(ns=-1), -1), (dict(ns=8), -2), (dict(hq=5), -1), (dict(hq=0), -1),
    (dict(hq=34, ns=3), -2), (dict(dt=4), -1), (dict(B=0), 0)])
@no_gpu
def test_attn_arguments(lib, kw, want):
    assert attn(lib, **kw) == want


@no_gpu
def test_workspace_sizes_are_checked(lib):
    f = lib.attn_decode_workspace_bytes
    assert f(-1, 0, 4, 2, 128) == -1 and f(1, 0, 5, 2, 128) == -1
    assert f(1, 9, 4, 2, 128) == -2 and f(1, 0, 4, 2, 80) == -2 and f(1, 0, 66, 1, 128) == -2


def test_binding_checks():
    z = torch.zeros
    q, v, ab = z(4, 2, 64), z(4, 4, 64), z(4, 4)
    vec, st, i32 = z(4), z(3, 4, 64, 64), z(4, dtype=torch.int32)
    call = dict(q=q, k=q, v=v, a=ab, b=ab, A_log=vec, dt_bias=vec, states=st, state_idx=i32, n_spec=0,
                num_accepted=None, has_init=None, scale=1.0, out=v)
    for bad, err in ((dict(state_idx=i32.long()), TypeError), (dict(k=q.bfloat16()), TypeError),
                     (dict(A_log=vec.double()), TypeError), (dict(A_log=z(3)), ValueError),
                     (dict(states=st.transpose(2, 3)), ValueError), (dict(states=st[:, :2]), ValueError),
                     (dict(q=q[:, :1]), ValueError), (dict(a=z(4, 3)), ValueError), (dict(out=v[:3]), ValueError),
                     (dict(n_spec=1), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                     (dict(), ValueError)):                       # the last: host tensors
        with pytest.raises(err):
            ops.gdn_update(**{**call, **bad})
    with pytest.raises(ValueError):
        ops.gdn_fwd_varlen(q, q, v, ab, ab, vec, vec, st, i32, i32, None, 1.0, v)
    c, p = z(5, 16, 2, 64), z(4, dtype=torch.int32)
    norm = dict(q=v, k=q, v=q, q_weight=None, k_weight=None, eps=1e-6, cos_sin=z(9, 64), positions=p,
                interleaved=False, k_cache=c, v_cache=c, slot_mapping=p, q_out=v)
    for bad, err in ((dict(positions=p.long()), TypeError), (dict(k=v), ValueError), (dict(q_out=q), ValueError),
                     (dict(v_cache=c[:, :, :1]), ValueError), (dict(v_cache=c.bfloat16()), TypeError),
                     (dict(q_weight=z(32)), ValueError), (dict(cos_sin=z(9, 64).double()), TypeError),
                     (dict(slot_mapping=p[:3]), ValueError), (dict(), ValueError)):
        with pytest.raises(err):
            ops.attn_norm_rope_cache(**{**norm, **bad})
    dec = dict(q=v, k_cache=c, v_cache=c, block_table=z(4, 3, dtype=torch.int32), seq_lens=p, n_spec=0, scale=1.0,
               out=v)
    for bad, err in ((dict(seq_lens=p.long()), TypeError), (dict(out=q), ValueError), (dict(n_spec=1), ValueError),
                     (dict(block_table=z(3, 3, dtype=torch.int32)), ValueError),
                     (dict(lse=z(4, 4).double()), ValueError), (dict(out=v.bfloat16()), TypeError),
                     (dict(k_cache=z(5, 16, 2, 32)), ValueError), (dict(), ValueError)):
        with pytest.raises(err):
            ops.attn_decode(**{**dec, **bad})


# ---- the marshalling in C takes the same calls as the one in Python ---------------

@pytest.mark.gpu
@pytest.mark.parametrize("what", ["fwd", "update", "norm", "attn"])
def test_both_marshallings_agree(what, monkeypatch):
    dev, bf = torch.device("cuda"), torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(3)

    def rnd(*shape, dtype=bf):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    rows = rnd(6, (2 + 2 + 4) * 64)
    q, k, v = (t.unflatten(1, (-1, 64)) for t in rows.split([128, 128, 256], 1))
    gates, A, dt = rnd(6, 8), rnd(4, dtype=torch.float32), rnd(4, dtype=torch.float32)
    states, cache = rnd(8, 4, 64, 64, dtype=torch.float32), rnd(4, 2, 16, 2, 64)
    cos = rnd(32, 64, dtype=torch.float32)

    def call():
        st, c = states.clone(), cache.clone()
        out = torch.zeros(6, 4, 64, device=dev, dtype=bf)
        lse = torch.zeros(6, 4, device=dev)
        if what == "fwd":
            ops.gdn_fwd_varlen(q, k, v, gates[:, :4], gates[:, 4:], A, dt, st, ints(2, 5),
                               ints(0, 1, 6), None, 0.125, out)
        elif what == "update":
            ops.gdn_update(q, k, v, gates[:, :4], gates[:, 4:], A, dt, st, ints(1, 2, 3, 4, 5, 6)
                           .view(3, 2), 1, ints(1, 2, 1), None, 0.125, out)
        elif what == "norm":
            ops.attn_norm_rope_cache(v, k, q, rnd(64) * 0 + 1, None, 1e-6, cos,
                                     ints(0, 1, 2, 3, 4, 5), True, c[:, 0], c[:, 1],
                                     ints(9, 30, -1, 0, 17, 63), out)
        else:
            ops.attn_decode(v, c[:, 0], c[:, 1], ints(1, 0, 3, 2).view(2, 2), ints(19, 3), 2, 0.125,
                            out, lse)
        torch.cuda.synchronize()
        return st, c, out, lse

    ops.load()
    served = []
    if ops._fast is not None:
        name = {"fwd": "gdn_fwd_varlen", "update": "gdn_update", "norm": "attn_norm_rope_cache",
                "attn": "attn_decode"}[what]
        real, plain = ops._fast, getattr(ops._fast, name)

        class Spy:
            def __getattr__(self, n):
                return (lambda *x: served.append(plain(*x)) or served[-1]) if n == name else \
                    getattr(real, n)

        monkeypatch.setattr(ops, "_fast", Spy())
    one = call()
    assert ops._fast is None or served == [0]
    monkeypatch.setattr(ops, "_fast", None)
    for a, b in zip(one, call()):
        assert torch.equal(a, b)


def _two():
    """Two valid sets of arguments (host tensors): of the delta rule and of attention."""
    z = torch.zeros
    q, v, ab, c = z(4, 2, 64), z(4, 4, 64), z(4, 4), z(5, 16, 2, 64)
    i = lambda *s: z(*s, dtype=torch.int32)                     # noqa: E731
    gdn = dict(q=q, k=q, v=v, a=ab, b=ab, A_log=z(4), dt_bias=z(4), states=z(8, 4, 64, 64), scale=1.0, out=v)
    norm = dict(q=v, k=q, v=q, q_weight=None, k_weight=None, eps=1e-6, cos_sin=z(9, 64), positions=i(4),
                interleaved=False, k_cache=c, v_cache=c, slot_mapping=i(4), q_out=v)
    attn = dict(q=v, k_cache=c, v_cache=c, block_table=i(4, 3), seq_lens=i(4), n_spec=0, scale=1.0, out=v)
    return gdn, norm, attn, i


def test_binding_refuses_short_and_strided_indices():
    """Index and flag vectors are read as so many entries side by side: others are refused, by name."""
    gdn, norm, attn, i = _two()
    flags = torch.zeros(8, dtype=torch.uint8)
    fwd = dict(gdn, state_idx=i(2), cu_seqlens=i(3), has_init=None)
    upd = dict(gdn, state_idx=i(4), n_spec=0, num_accepted=None, has_init=None)
    spec = dict(gdn, state_idx=i(2, 2), n_spec=1, num_accepted=i(2), has_init=None)
    cases = [(ops.gdn_fwd_varlen, fwd, "state_idx", i(2, 4)[:, 0]), (ops.gdn_fwd_varlen, fwd, "state_idx", i(2, 4)),
             (ops.gdn_fwd_varlen, fwd, "cu_seqlens", i(6)[::2]), (ops.gdn_fwd_varlen, fwd, "cu_seqlens", i(2)),
             (ops.gdn_fwd_varlen, fwd, "has_init", flags[:1]), (ops.gdn_fwd_varlen, fwd, "has_init", flags[:4:2]),
             (ops.gdn_update, upd, "state_idx", i(4, 2)[:, 0]), (ops.gdn_update, upd, "has_init", flags[:3]),
             (ops.gdn_update, upd, "has_init", flags[::2]), (ops.gdn_update, spec, "num_accepted", i(1)),
             (ops.gdn_update, spec, "num_accepted", i(4)[::2]),
             (ops.attn_norm_rope_cache, norm, "positions", i(8)[::2]),
             (ops.attn_norm_rope_cache, norm, "positions", i(3)),
             (ops.attn_norm_rope_cache, norm, "slot_mapping", i(8)[::2]),
             (ops.attn_norm_rope_cache, norm, "slot_mapping", i(3)),
             (ops.attn_decode, attn, "seq_lens", i(4, 2)[:, 0]), (ops.attn_decode, attn, "seq_lens", i(4, 2)),
             (ops.attn_decode, attn, "workspace", torch.zeros(64, 64, dtype=torch.uint8).t())]
    for fn, call, name, bad in cases:
        with pytest.raises(ValueError, match=name):
            fn(**{**call, name: bad})
    for fn, call in ((ops.gdn_fwd_varlen, fwd), (ops.gdn_update, upd), (ops.attn_norm_rope_cache, norm),
                     (ops.attn_decode, attn)):
        with pytest.raises(TypeError, match="dev_err"):
            fn(**call, dev_err=torch.zeros(4, dtype=torch.uint8))
        with pytest.raises(ValueError, match="dev_err"):
            fn(**call, dev_err=i(0))


def test_binding_takes_what_it_does_not_read():
    """A short num_accepted without draft tokens, and vectors longer than needed, get as far as the check
    of where the tensors live."""
    gdn, norm, attn, i = _two()
    flags = torch.zeros(8, dtype=torch.uint8)
    for fn, call in ((ops.gdn_update, dict(gdn, state_idx=i(4), n_spec=0, num_accepted=i(1), has_init=flags)),
                     (ops.gdn_update, dict(gdn, state_idx=i(4, 1), n_spec=0, num_accepted=None, has_init=None)),
                     (ops.gdn_fwd_varlen, dict(gdn, state_idx=i(2, 1), cu_seqlens=i(3), has_init=flags)),
                     (ops.attn_norm_rope_cache, {**norm, "positions": i(9), "slot_mapping": i(9)}),
                     (ops.attn_decode, dict(attn, workspace=torch.zeros(9, dtype=torch.uint8)))):
        with pytest.raises(ValueError, match="must live on the GPU"):
            fn(**call)


class _Placed:
    """A host tensor that says it lives on a GPU: its address goes to the library, which has none."""

    def __init__(self, t, dev=0):
        self.t, self.dev, self.is_cuda = t, dev, True

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def _placed_calls():
    gdn, norm, attn, i = _two()
    flags, err = torch.zeros(8, dtype=torch.uint8), i(1)
    return [("gdn_fwd_varlen", dict(gdn, state_idx=i(2), cu_seqlens=i(3), has_init=flags, dev_err=err)),
            ("gdn_update", dict(gdn, state_idx=i(2, 2), n_spec=1, num_accepted=i(2), has_init=flags, dev_err=err)),
            ("attn_norm_rope_cache", dict(norm, q_weight=torch.zeros(64), k_weight=torch.zeros(64), dev_err=err)),
            ("attn_decode", dict(attn, lse=torch.zeros(4, 4), workspace=torch.zeros(1 << 26, dtype=torch.uint8),
                                 dev_err=err))]


@no_gpu
@pytest.mark.parametrize("in_c", [True, False])
def test_tensors_of_a_call_share_the_current_device(in_c, monkeypatch):
    """A call whose tensors lie on another device than the current one, whose stream and SMs it would take,
    or on two, is refused; C leaves it to Python, which raises. (Without a GPU a call that is not refused
    ends with the launch's status.)"""
    lib = ops.load()
    if in_c and ops._fast is None:
        pytest.skip("the C module is not built")
    current = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(ops, "_raw_stream", lambda stream: None)
    seen = []
    if in_c:
        ops._fast.init(lib._handle, (torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.bool),
                       lambda d: seen.append(d) or 0, None, lambda: current[0])
    else:
        monkeypatch.setattr(ops, "_fast", None)
    try:
        for fn, call in _placed_calls():
            tensors = [n for n, t in call.items() if torch.is_tensor(t)]
            here = {n: _Placed(t) if n in tensors else t for n, t in call.items()}
            with pytest.raises(ops.CConvError, match=fn):
                getattr(ops, fn)(**here)
            assert not in_c or seen.pop() == 0
            for n in tensors:
                with pytest.raises(ValueError, match="current device"):
                    getattr(ops, fn)(**{**here, n: _Placed(call[n], 1)})
            current[0] = 1
            with pytest.raises(ValueError, match="current device"):
                getattr(ops, fn)(**here)
            current[0] = 0
            assert not seen
    finally:
        ops._load_fast(lib)


@no_gpu
def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        ops._raw_stream(Stream())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert ops._raw_stream(Stream()) == 0
