"""Ways through the mixers that only larger or other calls take: blocks that work on several items or chains,
more sequences than one launch orders, blocks of query rows, and caches whose heads lie apart."""
import pytest
import torch

from state_cached_causal_gb300 import ops
from tests._mixers import assert_close, gdn_ref
from tests.test_attn_decode import case, check
from tests.test_gdn import BF16, DEV, F32, check_fwd, inputs, pool

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("st_dtype", [F32, BF16])
@pytest.mark.parametrize("dtype,d,n_spec", [(BF16, 128, 0), (BF16, 128, 3), (BF16, 64, 1), (F32, 128, 0)])
def test_update_with_several_items_a_block(dtype, d, n_spec, st_dtype):
    """8 heads of 4 (2) column blocks: 3520 (2816) items, three (two) or more for each of the grid's blocks, which
    request the next one's state, tokens, gates and indices ahead. Some requests start from zeros, some
    are skipped rows of padding, some keep no state."""
    B, n, hk, hv = 110 if d == 128 else 176, 1 + n_spec, 4, 8
    inp = inputs(61 + n_spec, B * n, hk, hv, d, d, dtype, spare=0)
    slots = B * n + 5
    st = pool(61, slots, hv, d, d, st_dtype)
    before = st.double().cpu()
    g = torch.Generator().manual_seed(n)
    idx = torch.randperm(slots, generator=g)[:B * n].to(torch.int32).reshape(B, n).clone()
    idx[::7, n - 1] = -1
    idx[5] = -1                                            # a row of padding
    acc = torch.randint(1, n + 1, (B,), generator=g, dtype=torch.int32)
    init = (torch.rand(B, generator=g) < 0.8).to(torch.uint8)
    out = torch.zeros(B * n, hv, d, device=DEV, dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.gdn_update(*inp, st, idx.to(DEV), n_spec, acc.to(DEV), init.to(DEV), 0.2, out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    cpu = [t.double().cpu() for t in inp]
    want_out, want_st = torch.zeros(out.shape, dtype=torch.float64), before.clone()
    for s in range(B):
        src = int(idx[s, acc[s] - 1])
        S0 = before[src] if src >= 0 and init[s] else torch.zeros(hv, d, d).double()
        o, states = gdn_ref(*[t[s * n:(s + 1) * n] for t in cpu[:5]], cpu[5], cpu[6], S0, 0.2)
        want_out[s * n:(s + 1) * n] = o
        for t in range(n):
            if idx[s, t] >= 0:
                want_st[int(idx[s, t])] = states[t + 1]
    for s in range(B):
        assert_close(out[s * n:(s + 1) * n], want_out[s * n:(s + 1) * n], f"outputs of request {s}")
    for slot in range(slots):
        assert_close(st[slot], want_st[slot], f"slot {slot}")


@gpu
@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 128), (F32, 64, 64)])
def test_fwd_of_short_sequences_with_several_items_a_block(dtype, dk, dv):
    """1 to 8 tokens, empty ones among them: token batches that go on within an item and from one to the next."""
    lens = [(5 * i) % 9 for i in range(150)]
    check_fwd(62, lens, 4, 8, dk, dv, dtype, F32, init=[int(i % 3 > 0) for i in range(150)])


@gpu
@pytest.mark.parametrize("with_init", [True, False])
def test_more_sequences_than_a_launch_orders(with_init):
    """700 sequences, long and short ones on both sides of the 640th."""
    lens = [65 if i % 40 == 7 else 9 + i % 5 if i % 9 == 0 else i % 3 for i in range(700)]
    lens[637:644] = [70, 1, 130, 12, 64, 0, 9]
    lens[-1] = 100
    if with_init:
        check_fwd(63, lens, 1, 2, 128, 128, BF16, F32, init=[int(i % 2 == 0) for i in range(700)])
        return
    T = sum(lens)
    inp = inputs(64, T, 1, 2, 128, 128, BF16, spare=0)
    st = pool(64, 700, 2, 128, 128, F32)
    cpu = [t.double().cpu() for t in inp]
    before = st.double().cpu()
    cu = torch.tensor([sum(lens[:i]) for i in range(701)], dtype=torch.int32)
    out = torch.zeros(T, 2, 128, device=DEV, dtype=BF16)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.gdn_fwd_varlen(*inp, st, torch.arange(700, dtype=torch.int32, device=DEV), cu.to(DEV), None, 0.1, out,
                       dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for i, n in enumerate(lens):
        a = int(cu[i])
        o, states = gdn_ref(*[t[a:a + n] for t in cpu[:5]], *cpu[5:], before[i], 0.1)
        assert_close(out[a:a + n], o, f"outputs of sequence {i}")
        assert_close(st[i], states[-1], f"state of sequence {i}")


@gpu
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("hq,hkv,n", [(8, 4, 1), (8, 8, 3), (4, 1, 1), (16, 2, 2)])
@pytest.mark.parametrize("page", [16, 7])
def test_heads_that_lie_apart(D, hq, hkv, n, page):
    """[pages, heads, page, dim] caches in bf16: a copy a head and position; one head: several positions."""
    assert check(*case(71, [1, 95, 260, 0], hq, hkv, D, page, n, BF16, heads_first=True), n) == 0


@gpu
@pytest.mark.parametrize("D,dtype", [(256, BF16), (128, BF16), (128, F32)])
@pytest.mark.parametrize("hq,hkv,n", [(8, 1, 4), (8, 1, 8), (16, 2, 5), (32, 4, 6), (17, 1, 3)])
def test_blocks_of_query_rows(D, dtype, hq, hkv, n):
    """24 to 64 rows a kv head, two to eight blocks of them, the last one not full."""
    assert check(*case(72, [700, n, 33, 2], hq, hkv, D, 16, n, dtype), n) == 0
