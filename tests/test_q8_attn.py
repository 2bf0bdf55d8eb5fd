"""attn_decode_q8 against softmax attention in 64 bits over the values that the cache's bytes and scales stand
for: as tests/test_attn_decode.py and tests/test_attn_rounding.py are for attn_decode, with rows of several
sizes and NaN where no request holds a row.

A bf16 result is rounded once: the softmax weights enter as fp16 (2^-11 of each at most, independent of one
another, so 2^-12 of the result's norm and thereabouts), q and the cache exactly. An error of d (of the value)
turns the rounding of a value over for a share d / u of them, u the distance of neighbours (2^-7 of the value at
most), which makes sqrt(d u) <= 2^-9 of the norm against the rounded result of 64 bits.
"""
import pytest
import torch

from state_cached_causal_gb300 import ops
from tests._mixers import assert_close, attn_ref
from tests._q8 import DEV, F8, cache_pair, case, in_64_bits, values
from state_cached_causal_gb300 import synth

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def run(q, kc, vc, ks, vs, table, lens, n, scale=None, stream=None, lse=None, workspace=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out = torch.full(q.shape, 7.0, device=DEV, dtype=q.dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.attn_decode_q8(q, kc, vc, ks, vs, table, lens, n - 1, scale, out, lse=lse, dev_err=err, stream=stream,
                       workspace=workspace)
    torch.cuda.synchronize()
    k, v = in_64_bits(kc, vc, ks, vs)
    want, want_lse = attn_ref(q.cpu(), k, v, table.cpu(), lens.tolist(), n, scale)
    return out, want, want_lse, err.item()


def check(q, kc, vc, ks, vs, table, lens, n, **kw):
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out, want, want_lse, err = run(q, kc, vc, ks, vs, table, lens, n, lse=lse, **kw)
    assert_close(out, want, "out")
    if q.dtype is BF16 and want.norm() > 0:
        off = (out.cpu().double() - want.to(BF16).double()).norm() / want.norm()
        assert off <= 2.0 ** -9, f"{off:.3g}"
    fin = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse.cpu()), fin)
    # fp32 sums of exact products, magnitudes of a few tens at most
    assert torch.allclose(lse.cpu().double()[fin], want_lse[fin], rtol=1e-5, atol=1e-4)
    return err


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[1], [0, 1, 2], [31, 32, 33], [63, 64, 65, 0, 7], [127, 129, 1000], [5000]])
def test_lengths(dtype, lens):
    assert check(*case(1, lens, 4, 2, 128, 16, 1, dtype), 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 4), (6, 2), (16, 1), (8, 8)])
def test_heads(dtype, D, hq, hkv):
    assert check(*case(2, [70, 3, 300], hq, hkv, D, 16, 1, dtype), 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [2, 4, 8])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (16, 4), (8, 1)])
def test_draft_tokens(dtype, n, hq, hkv):
    # lengths below n leave the first rows with nothing to see
    assert check(*case(3, [n, 1, 64 + n, 200, 0], hq, hkv, 128, 16, n, dtype), n) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [1, 7, 16, 48, 128])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 64), (4, 4, 128), (3, 1, 64)])
def test_pages(dtype, page, heads_first, hq, hkv, D):
    assert check(*case(4, [1, 95, 260], hq, hkv, D, page, 1, dtype, heads_first), 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores_and_rows_of_many_sizes(dtype):
    assert check(*case(5, [300, 40], 4, 1, 128, 16, 1, dtype, big=4.0, spread=5), 1) == 0


def test_many_requests():
    lens = [(37 * i) % 190 for i in range(700)]
    assert check(*case(6, lens, 2, 1, 64, 16, 1, BF16), 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hq,hkv,n,D", [(16, 2, 8, 64), (8, 1, 8, 256), (17, 1, 3, 128), (32, 4, 6, 128)])
def test_blocks_of_rows_and_many_parts(dtype, hq, hkv, n, D):
    assert check(*case(12, [6000, 8, 9, 33, 10], hq, hkv, D, 16, n, dtype), n) == 0


def test_values_far_apart():
    """Values 2^40 times as large as others, under weights that make up for it, and scales at both ends."""
    q, kc, vc, ks, vs, table, lens = case(14, [200], 4, 1, 64, 16, 1, BF16)
    vs[int(table[0, 3])] = 127 + 40
    ks[int(table[0, 3])] = 127 - 20               # (scores near zero there)
    vs[int(table[0, 5])] = 1
    vs[int(table[0, 6])] = 20
    assert check(q * 3, kc, vc, ks, vs, table, lens, 1) == 0
    vs[:] = 1 + 30
    out, want, _, _ = run(q, kc, vc, ks, vs, table, lens, 1)
    assert ((out.cpu().double() - want).norm() / want.norm()) < 2.0 ** -8


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_queries_of_any_size(size):
    """q and the scale that makes up for it: bf16 values that fp16 does not hold."""
    c = case(15, [150, 9], 4, 2, 128, 16, 1, BF16)
    q = (c[0].float() * size).to(BF16)
    assert check(q, *c[1:], 1, scale=128 ** -0.5 / size) == 0


def test_other_stream_and_callers_workspace():
    c = case(7, [500, 20], 16, 4, 128, 16, 1, BF16)
    ws = torch.full((ops.attn_decode_workspace_bytes(2, 0, 16, 4, 128),), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert check(*c, 1, stream=torch.cuda.Stream(), workspace=ws) == 0


def test_the_same_every_time_and_replayed():
    q, kc, vc, ks, vs, table, lens = case(8, [3000, 20, 777], 16, 4, 128, 16, 4, BF16)
    ws = torch.empty(ops.attn_decode_workspace_bytes(3, 3, 16, 4, 128), dtype=torch.uint8, device=DEV)
    out = torch.zeros(q.shape, device=DEV, dtype=BF16)
    got = []
    for _ in range(2):
        out.zero_()
        ops.attn_decode_q8(q, kc, vc, ks, vs, table, lens, 3, 0.1, out, workspace=ws)
        torch.cuda.synchronize()
        got.append(out.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.attn_decode_q8(q, kc, vc, ks, vs, table, lens, 3, 0.1, out, workspace=ws)
    out.zero_()
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], out)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 64), (16, 4, 128), (12, 1, 128), (4, 2, 256)])
def test_draft_values_that_are_nan(dtype, hq, hkv, D):
    """NaN in a draft token's key and values reach its own row and those after it only."""
    n = 4
    q, kc, vc, ks, vs, table, lens = case(13, [18, 4, 100, 65], hq, hkv, D, 16, n, dtype)
    for b, length in enumerate(lens.tolist()):
        last = length - 1 - (b % 2)                       # the last draft token, or the one before
        page = int(table[b, last // 16])
        vc.view(torch.uint8)[page, last % 16, :, 3 + 2 * b] = 0x7f
        vc.view(torch.uint8)[page, last % 16, 0, D - 1 - b] = 0xff
    kc.view(torch.uint8)[int(table[2, 99 // 16]), 99 % 16] = 0x7f
    out, want, _, _ = run(q, kc, vc, ks, vs, table, lens, n)
    nan = torch.isnan(want)
    assert nan.any() and torch.equal(torch.isnan(out.cpu()), nan)
    assert_close(out.nan_to_num(0), want.masked_fill(nan, 0), "out")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_bad_page_is_left_out(dtype):
    q, kc, vc, ks, vs, table, lens = case(9, [100, 40], 4, 2, 128, 16, 1, dtype)
    table[0, 2], table[1, 0] = -1, kc.shape[0]
    assert check(q, kc, vc, ks, vs, table, lens, 1) == ops.DERR_PAGE


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_a_bad_length_skips_the_request(dtype, bad):
    q, kc, vc, ks, vs, table, lens = case(10, [100, 40, 30], 4, 2, 128, 16, 1, dtype)
    good = lens.clone()
    lens[1] = bad
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.attn_decode_q8(q, kc, vc, ks, vs, table, lens, 0, 0.1, out, dev_err=err)
    torch.cuda.synchronize()
    want = attn_ref(q.cpu(), *in_64_bits(kc, vc, ks, vs), table.cpu(), good.tolist(), 1, 0.1)[0]
    assert err.item() == ops.DERR_SEQ_LEN
    assert (out[1] == 7).all()
    assert_close(out[[0, 2]], want[[0, 2]], "the others")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_beyond_32_bits(dtype):
    """Cache rows past 2^31 bytes."""
    hkv, D, page = 8, 128, 64
    pages = 2 ** 31 // (page * hkv * D) + 4
    kc, vc = (torch.zeros(pages, page, hkv, D, device=DEV, dtype=torch.uint8).view(F8) for _ in range(2))
    ks, vs = (torch.full((pages, page, hkv), 127, device=DEV, dtype=torch.uint8) for _ in range(2))
    g = synth.generator(11, DEV)
    for to, new in zip((kc, vc, ks, vs), cache_pair(g, (3, page, hkv, D))):
        to.view(torch.uint8)[-3:] = new.view(torch.uint8)
    q = torch.randn(1, 16, D, generator=g, device=DEV).to(dtype)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device=DEV)
    out = torch.zeros(q.shape, device=DEV, dtype=dtype)
    ops.attn_decode_q8(q, kc, vc, ks, vs, table, torch.tensor([150], dtype=torch.int32, device=DEV), 0, 0.1, out)
    torch.cuda.synchronize()
    tail = lambda t: t.view(torch.uint8)[-3:].cpu()                    # noqa: E731
    want, _ = attn_ref(q.cpu(), values(tail(kc).view(F8), tail(ks)), values(tail(vc).view(F8), tail(vs)),
                       torch.tensor([[2, 0, 1]]), [150], 1, 0.1)
    assert_close(out, want, "out")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_padded_batch_and_scales_of_any_stride(dtype):
    """Rows behind the last request are left as they were; scales that are views of wider tensors."""
    q, kc, vc, ks, vs, table, lens = case(16, [40, 0, 90], 8, 4, 64, 16, 1, dtype)
    wide = [torch.zeros(*s.shape[:2], 2 * s.shape[2] + 1, dtype=torch.uint8, device=DEV) for s in (ks, vs)]
    views = [w[:, :, 1::2] for w in wide]
    for w, s in zip(views, (ks, vs)):
        w.copy_(s)
    more = torch.cat([q, q], 0)
    out = torch.full(more.shape, 7.0, device=DEV, dtype=dtype)
    ops.attn_decode_q8(more, kc, vc, *views, table, lens, 0, 0.1, out)
    torch.cuda.synchronize()
    want = attn_ref(q.cpu(), *in_64_bits(kc, vc, ks, vs), table.cpu(), lens.tolist(), 1, 0.1)[0]
    assert_close(out[:3], want, "out")
    assert (out[3:] == 7).all()
