"""The gated delta rule (gdn_fwd_varlen, gdn_update) against its recurrence in 64 bits: lengths
around the chunk and the recurrent kernel's limits, types, head layouts, strides, gates at their
ends, equal keys, empty sequences, padding rows, foreign rows of NaN, and device-side errors."""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests._mixers import assert_close, gdn_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
F32, BF16 = torch.float32, torch.bfloat16


def inputs(seed, T, hk, hv, dk, dv, dtype, *, lead=0, keys="silu", gates="normal", spare=1):
    """Rows [lead, lead + T) hold the inputs; what surrounds them is NaN. q, k and v are views of
    one row of channels."""
    g = synth.generator(seed, DEV)
    rows = lead + T + spare
    x = torch.randn(rows, (2 * hk * dk + hv * dv), generator=g, device=DEV)
    x = x * torch.sigmoid(x)
    a = torch.randn(rows, hv, generator=g, device=DEV)
    b = torch.randn(rows, hv, generator=g, device=DEV)
    if keys == "equal":
        x[:, hk * dk:2 * hk * dk] = x[lead, hk * dk:2 * hk * dk].clone()
        b += 8
        a -= 12
    if keys == "zero":
        x[lead::3, hk * dk:2 * hk * dk] = 0
    if gates == "ends":
        a = torch.where(a > 0.5, 60.0, torch.where(a < -0.5, -60.0, a))
        b = torch.where(b > 0.5, 60.0, torch.where(b < -0.5, -60.0, b))
    for t in (x, a, b):
        t[:lead] = float("nan")
        t[lead + T:] = float("nan")
    x, a, b = x.to(dtype), a.to(dtype), b.to(dtype)
    q, k, v = x.split([hk * dk, hk * dk, hv * dv], 1)
    A_log = torch.log(1 + 15 * torch.rand(hv, generator=g, device=DEV))
    dt_bias = torch.randn(hv, generator=g, device=DEV) - 4
    return (q.unflatten(1, (hk, dk)), k.unflatten(1, (hk, dk)), v.unflatten(1, (hv, dv)), a, b,
            A_log, dt_bias)


def pool(seed, slots, hv, dk, dv, dtype, gap=False):
    g = synth.generator(seed + 77, DEV)
    st = (0.3 * torch.randn(slots, hv + (1 if gap else 0), dk, dv, generator=g, device=DEV)).to(dtype)
    return st[:, :hv]


def check_fwd(seed, lens, hk, hv, dk, dv, dtype, st_dtype, *, lead=0, slots=None, idx=None,
              init=None, scale=0.1, l2norm=True, gap=False, stream=None, **kw):
    T = sum(lens)
    q, k, v, a, b, A_log, dt_bias = inp = inputs(seed, T, hk, hv, dk, dv, dtype, lead=lead, **kw)
    slots = slots or len(lens) + 2
    st = pool(seed, slots, hv, dk, dv, st_dtype, gap)
    before = st.clone()
    g = torch.Generator().manual_seed(seed)
    idx = torch.randperm(slots, generator=g)[:len(lens)].tolist() if idx is None else idx
    init = [int(i % 2 == 0) for i in range(len(lens))] if init is None else init
    cu = (synth.cu_from_lens(lens, "cpu") + lead).to(DEV)
    out = torch.full((v.shape[0], hv, dv), 7.0, device=DEV, dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.gdn_fwd_varlen(*inp, st, torch.tensor(idx, dtype=torch.int32, device=DEV), cu,
                       torch.tensor(init, dtype=torch.uint8, device=DEV), scale, out,
                       qk_l2norm=l2norm, dev_err=err, num_tokens=lead + T, stream=stream)
    torch.cuda.synchronize()
    assert err.item() == 0
    want_st = before.double().cpu()
    at = lead
    cpu = [t.double().cpu() for t in inp]
    for n, slot, h in zip(lens, idx, init):
        S0 = want_st[slot].clone() if slot >= 0 and h else torch.zeros(hv, dk, dv).double()
        rows = [t[at:at + n] for t in cpu[:5]]
        o, states = gdn_ref(*rows, cpu[5], cpu[6], S0, scale, l2norm)
        assert_close(out[at:at + n], o, f"outputs of a sequence of {n}")
        if slot >= 0:
            assert_close(st[slot], states[-1], f"state of a sequence of {n}")
        at += n
    for s in set(range(slots)) - {i for i in idx if i >= 0}:
        assert torch.equal(st[s], before[s]), "a slot of no sequence was written"
    assert (out[:lead] == 7).all() and (out[lead + T:] == 7).all()


@pytest.mark.parametrize("lens", [[1], [2, 1], [0, 1, 0, 5], [15, 16, 17], [63, 64, 65], [127, 128, 129],
                                  [1, 1, 1, 200, 33], [777]])
def test_lengths(lens):
    check_fwd(len(lens) + lens[0], lens, 2, 4, 128, 128, BF16, F32, lead=3)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("st", [F32, BF16])
def test_types_and_head_sizes(dk, dv, dtype, st):
    check_fwd(11, [70, 1, 9], 1, 2, dk, dv, dtype, st)


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 3), (4, 4), (2, 8)])
def test_head_layouts(hk, hv):
    check_fwd(12, [90, 20], hk, hv, 128, 128, BF16, BF16)


def test_more_chains_than_blocks():
    """9 sequences of 32 heads: 256 or more chains, several for each block of the persistent kernel,
    of whole and partial chunks in turn."""
    check_fwd(21, [70, 9, 128, 1, 64, 33, 130, 12, 65], 16, 32, 128, 128, BF16, F32)


@pytest.mark.parametrize("keys,gates", [("equal", "normal"), ("zero", "normal"), ("silu", "ends")])
@pytest.mark.parametrize("lens", [[130], [5]])
def test_hard_values(keys, gates, lens):
    check_fwd(13, lens, 1, 2, 128, 128, BF16, F32, keys=keys, gates=gates)


def test_without_normalisation():
    """Raw q and k (keys small enough for the rule to be stable without it)."""
    q, k, v, a, b, A_log, dt_bias = inputs(14, 100, 1, 1, 128, 128, BF16)
    k.mul_(0.05)
    st = pool(14, 1, 1, 128, 128, F32)
    S0 = st[0].double().cpu()
    out = torch.zeros(v.shape, device=DEV, dtype=BF16)
    ops.gdn_fwd_varlen(q, k, v, a, b, A_log, dt_bias, st,
                       torch.zeros(1, dtype=torch.int32, device=DEV),
                       torch.tensor([0, 100], dtype=torch.int32, device=DEV), None, 0.1, out,
                       qk_l2norm=False, num_tokens=100)
    torch.cuda.synchronize()
    cpu = [t.double().cpu() for t in (q, k, v, a, b)]
    o, states = gdn_ref(*[t[:100] for t in cpu], A_log.double().cpu(), dt_bias.double().cpu(), S0,
                        0.1, False)
    assert_close(out[:100], o, "outputs")
    assert_close(st[0], states[-1], "state")


def test_padding_rows_and_strided_pool():
    check_fwd(15, [40, 66, 1, 0, 2], 1, 2, 128, 128, BF16, F32, idx=[3, -1, -1, 0, 6], slots=8,
              init=[1, 1, 0, 0, 1], gap=True)


def test_empty_sequences_keep_or_clear_their_slot():
    check_fwd(16, [0, 0, 3], 1, 1, 128, 128, BF16, F32, init=[1, 0, 1])


def test_other_stream():
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    check_fwd(17, [65, 1], 1, 2, 128, 128, BF16, F32, stream=s)


def test_split_sequences_carry_their_state():
    """One pass over 150 tokens equals 70, 1, 1 and 78 tokens in turn through the pool."""
    inp = inputs(18, 150, 1, 2, 128, 128, BF16, spare=0)
    whole, parts = pool(18, 2, 2, 128, 128, F32), pool(18, 2, 2, 128, 128, F32)
    o1, o2 = (torch.zeros(150, 2, 128, device=DEV, dtype=BF16) for _ in range(2))
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    ops.gdn_fwd_varlen(*inp, whole, one, torch.tensor([0, 150], dtype=torch.int32, device=DEV),
                       None, 0.1, o1)
    for s, e in ((0, 70), (70, 71), (71, 72), (72, 150)):
        if e - s == 1:
            ops.gdn_update(*[t[s:e] for t in inp[:5]], *inp[5:], parts, one, 0, None, None, 0.1,
                           o2[s:e])
        else:
            ops.gdn_fwd_varlen(*inp, parts, one, torch.tensor([s, e], dtype=torch.int32, device=DEV),
                               None, 0.1, o2)
    torch.cuda.synchronize()
    assert_close(parts[1], whole[1].double().cpu(), "state")
    assert_close(o2, o1.double().cpu(), "outputs")


def test_fwd_is_the_same_every_time():
    inp = inputs(19, 400, 2, 4, 128, 128, BF16, spare=0)
    got = []
    for _ in range(3):
        st = pool(19, 3, 4, 128, 128, F32)
        out = torch.zeros(400, 4, 128, device=DEV, dtype=BF16)
        ops.gdn_fwd_varlen(*inp, st, torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                           torch.tensor([0, 300, 400], dtype=torch.int32, device=DEV), None, 0.1, out)
        torch.cuda.synchronize()
        got.append((out, st))
    assert all(torch.equal(o, got[0][0]) and torch.equal(s, got[0][1]) for o, s in got[1:])


def _fwd(inp, lens, st):
    out = torch.zeros(sum(lens), inp[2].shape[1], 128, device=DEV, dtype=BF16)
    ops.gdn_fwd_varlen(*inp, st, torch.arange(len(lens), dtype=torch.int32, device=DEV),
                       synth.cu_from_lens(lens, DEV), None, 0.1, out)
    return out


@pytest.mark.parametrize("where", ["q", "k", "v", "a", "state"])
def test_what_is_not_finite_stays_in_its_sequence(where):
    """Several chains a block, every other sequence with an infinity or NaN: the others keep their
    bits, and so do the chunks of 64 tokens before it."""
    lens = [130 + 7 * (i % 5) for i in range(58)] + [1, 3, 1, 2]
    inp = inputs(23, sum(lens), 2, 8, 128, 128, BF16, spare=0)
    st = pool(23, len(lens), 8, 128, 128, F32)
    good_st = st.clone()
    good = _fwd(inp, lens, good_st)
    at = 0
    for i, n in enumerate(lens):
        if i % 2:
            bad = (float("nan"), float("inf"), -float("inf"))[i // 2 % 3]
            if where == "state":
                st[i, :, 5, 17] = bad
            else:
                inp[dict(q=0, k=1, v=2, a=3)[where]][at + (100 if n > 100 else 0)] = bad
        at += n
    out = _fwd(inp, lens, st)
    torch.cuda.synchronize()
    at = 0
    for i, n in enumerate(lens):
        keep = n if i % 2 == 0 else 64 if n > 100 and where != "state" else 0
        assert torch.equal(out[at:at + keep], good[at:at + keep]), i
        if i % 2 == 0:
            assert torch.equal(st[i], good_st[i]), i
        at += n


def test_captured_in_a_graph():
    """Both kernels of a call, replayed: what follows in the graph sees both results."""
    lens = [200, 1, 2000, 5, 64]
    inp = inputs(24, sum(lens), 2, 4, 128, 128, BF16, spare=0)
    start = pool(24, len(lens), 4, 128, 128, F32)
    want_st = start.clone()
    want = _fwd(inp, lens, want_st)
    st, idx, cu = start.clone(), torch.arange(5, dtype=torch.int32, device=DEV), synth.cu_from_lens(lens, DEV)
    out, copies = torch.zeros_like(want), (torch.zeros_like(want), torch.zeros_like(start))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.copy_(start)
        ops.gdn_fwd_varlen(*inp, st, idx, cu, None, 0.1, out)
        copies[0].copy_(out)
        copies[1].copy_(st)
    for _ in range(3):
        for c in copies:
            c.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(copies[0], want) and torch.equal(copies[1], want_st)


def test_fwd_device_errors_skip_the_sequence():
    inp = inputs(20, 80, 1, 1, 128, 128, BF16, spare=0)
    for idx, cu, bit in (([0, 5], [0, 70, 80], ops.DERR_SLOT_RANGE),
                         ([0, 1], [0, 70, 60], ops.DERR_CU_SEQLENS),
                         ([0, 1], [0, 70, 99], ops.DERR_CU_SEQLENS)):
        st = pool(20, 2, 1, 128, 128, F32)
        before = st.clone()
        out = torch.full((80, 1, 128), 7.0, device=DEV, dtype=BF16)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ops.gdn_fwd_varlen(*inp, st, torch.tensor(idx, dtype=torch.int32, device=DEV),
                           torch.tensor(cu, dtype=torch.int32, device=DEV), None, 0.1, out,
                           dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == bit
        assert (out[70:] == 7).all() and not (out[:70] == 7).all()
        assert torch.equal(st[1], before[1]) and not torch.equal(st[0], before[0])


# ---- update ----------------------------------------------------------------

@pytest.mark.parametrize("n_spec", [0, 1, 3, 7])
@pytest.mark.parametrize("d,dtype,st_dtype", [(128, BF16, F32), (128, BF16, BF16), (64, BF16, F32),
                                              (64, F32, F32), (128, F32, BF16)])
def test_update(n_spec, d, dtype, st_dtype):
    B, n, hk, hv = 5, 1 + n_spec, 2, 4
    inp = inputs(30 + n_spec, B * n, hk, hv, d, d, dtype, spare=0)
    slots = B * n + 3
    st = pool(30, slots, hv, d, d, st_dtype, gap=True)
    before = st.double().cpu()
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(n)).to(torch.int32)[:B * n]
    idx = idx.reshape(B, n).clone()
    idx[3, n - 1] = -1                                   # a token whose state is not kept
    acc = torch.tensor([1 + i % n for i in range(B)], dtype=torch.int32)
    init = torch.tensor([1, 0, 1, 1, 1], dtype=torch.uint8)
    out = torch.zeros(B * n, hv, d, device=DEV, dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.gdn_update(*inp, st, idx.to(DEV), n_spec, acc.to(DEV), init.to(DEV), 0.2, out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    cpu = [t.double().cpu() for t in inp]
    written = set()
    for s in range(B):
        src = int(idx[s, acc[s] - 1])
        S0 = before[src] if src >= 0 and init[s] else torch.zeros(hv, d, d).double()
        o, states = gdn_ref(*[t[s * n:(s + 1) * n] for t in cpu[:5]], cpu[5], cpu[6], S0, 0.2)
        assert_close(out[s * n:(s + 1) * n], o, f"outputs of request {s}")
        for t in range(n):
            if idx[s, t] >= 0:
                written.add(int(idx[s, t]))
                assert_close(st[int(idx[s, t])], states[t + 1], f"state {t} of request {s}")
    for slot in set(range(slots)) - written:
        assert torch.equal(st[slot].double().cpu(), before[slot])


def test_update_device_errors_skip_the_request():
    inp = inputs(40, 8, 1, 1, 64, 64, BF16, spare=0)
    for idx, acc, bit in (([[0, 1, 2, 3], [4, 5, 9, 6]], [1, 1], ops.DERR_SLOT_RANGE),
                          ([[0, 1, 2, 3], [4, 5, 6, 7]], [1, 5], ops.DERR_NUM_ACCEPTED),
                          ([[0, 1, 2, 3], [4, 5, 6, 7]], [1, 0], ops.DERR_NUM_ACCEPTED)):
        st = pool(40, 8, 1, 64, 64, F32)
        before = st.clone()
        out = torch.full((8, 1, 64), 7.0, device=DEV, dtype=BF16)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ops.gdn_update(*inp, st, torch.tensor(idx, dtype=torch.int32, device=DEV), 3,
                       torch.tensor(acc, dtype=torch.int32, device=DEV), None, 0.2, out, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == bit
        assert (out[4:] == 7).all() and not (out[:4] == 7).all()
        assert torch.equal(st[4:], before[4:]) and not torch.equal(st[:4], before[:4])


def test_update_offsets_beyond_32_bits():
    """A state slot past 2^31 elements."""
    hv, d = 32, 128
    slots = 2 ** 31 // (hv * d * d) + 3
    st = torch.zeros(slots, hv, d, d, device=DEV, dtype=BF16)
    g = synth.generator(41, DEV)
    st[slots - 1] = (0.3 * torch.randn(hv, d, d, generator=g, device=DEV)).to(BF16)
    S0 = st[slots - 1].double().cpu()
    inp = inputs(41, 1, 16, hv, d, d, BF16, spare=0)
    out = torch.zeros(1, hv, d, device=DEV, dtype=BF16)
    ops.gdn_update(*inp, st, torch.tensor([slots - 1], dtype=torch.int32, device=DEV), 0, None, None,
                   0.2, out)
    torch.cuda.synchronize()
    o, states = gdn_ref(*[t.double().cpu() for t in inp], S0, 0.2)
    assert_close(out, o, "outputs")
    assert_close(st[slots - 1], states[1], "state")
    assert not st[:slots - 1].any()
