"""attn_decode against softmax attention in 64 bits: lengths from nothing to many tiles, pages that end
inside a tile, head groups, draft tokens, types, both cache orders, large scores, tables with rubbish
behind a request's length, NaN in cache rows that nobody sees, and device-side errors."""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests._mixers import assert_close, attn_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
F32, BF16 = torch.float32, torch.bfloat16


def case(seed, lens, hq, hkv, D, page, n, dtype, heads_first=False, big=1.0):
    g = synth.generator(seed, DEV)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    used = [(x + page - 1) // page for x in lens]
    pages = sum(used) + 2
    shape = (pages, hkv, page, D) if heads_first else (pages, page, hkv, D)
    kc, vc = (rnd(*shape).to(dtype) for _ in range(2))
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    width = max(used + [1]) + 2
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
        tail = used[b] * page - lens[b]
        if tail:                                  # the rest of the last page was never written
            kc[int(table[b, u - 1]), page - tail:] = float("nan")
            vc[int(table[b, u - 1]), page - tail:] = float("nan")
    q = (big * rnd(len(lens) * n, hq * D + 16)).to(dtype)[:, :hq * D].unflatten(1, (hq, D))
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def check(q, kc, vc, table, lens, n, scale=None, stream=None, lse=True, workspace=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out = torch.full(q.shape, 7.0, device=DEV, dtype=q.dtype)
    lse = torch.full(q.shape[:2], 7.0, device=DEV) if lse else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.attn_decode(q, kc, vc, table, lens, n - 1, scale, out, lse=lse, dev_err=err, stream=stream,
                    workspace=workspace)
    torch.cuda.synchronize()
    want, want_lse = attn_ref(q.cpu(), kc.cpu(), vc.cpu(), table.cpu(), lens.tolist(), n, scale)
    assert_close(out, want, "out")
    if lse is not None:
        fin = torch.isfinite(want_lse)
        assert torch.equal(torch.isfinite(lse.cpu()), fin)
        # fp32 sums of exact products, magnitudes of a few tens at most
        assert torch.allclose(lse.cpu().double()[fin], want_lse[fin], rtol=1e-5, atol=1e-4)
    return err.item()


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
def test_pages(dtype, page, heads_first):
    assert check(*case(4, [1, 95, 260], 8, 2, 64, page, 1, dtype, heads_first), 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(dtype):
    assert check(*case(5, [300, 40], 4, 1, 128, 16, 1, dtype, big=30.0), 1) == 0


def test_many_requests():
    lens = [(37 * i) % 190 for i in range(700)]
    assert check(*case(6, lens, 2, 1, 64, 16, 1, BF16), 1) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_of_many_parts(dtype):
    """A join of hundreds of rows, those of one request cut into more parts than a warp has lanes."""
    assert check(*case(12, [6000, 8, 9, 33, 10], 16, 2, 64, 16, 8, dtype), 8) == 0


def test_other_stream_and_callers_workspace():
    c = case(7, [500, 20], 16, 4, 128, 16, 1, BF16)
    ws = torch.full((ops.attn_decode_workspace_bytes(2, 0, 16, 4, 128),), 255, dtype=torch.uint8,
                    device=DEV)
    torch.cuda.synchronize()
    assert check(*c, 1, stream=torch.cuda.Stream(), lse=False, workspace=ws) == 0


def test_the_same_every_time():
    q, kc, vc, table, lens = case(8, [3000, 20, 777], 16, 4, 128, 16, 4, BF16)
    got = []
    for _ in range(3):
        out = torch.zeros(q.shape, device=DEV, dtype=BF16)
        ops.attn_decode(q, kc, vc, table, lens, 3, 0.1, out)
        torch.cuda.synchronize()
        got.append(out)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 64), (16, 4, 128), (12, 1, 128), (4, 2, 256)])
def test_draft_values_that_are_not_finite(dtype, hq, hkv, D):
    """Infinities and NaN in a draft token's key and values reach its own row and those after it only."""
    n = 4
    q, kc, vc, table, lens = case(13, [18, 4, 100, 65], hq, hkv, D, 16, n, dtype)
    bad = [float("inf"), float("-inf"), float("nan"), float("inf")]
    for b, length in enumerate(lens.tolist()):
        last = length - 1 - (b % 2)                       # the last draft token, or the one before
        page = int(table[b, last // 16])
        vc[page, last % 16, :, 3 + 2 * b] = bad[b]
        vc[page, last % 16, 0, D - 1 - b] = bad[(b + 1) % 4]
    kc[int(table[2, 99 // 16]), 99 % 16] = float("nan")
    out = torch.zeros(q.shape, device=DEV, dtype=dtype)
    ops.attn_decode(q, kc, vc, table, lens, n - 1, D ** -0.5, out)
    torch.cuda.synchronize()
    want, _ = attn_ref(q.cpu(), kc.cpu(), vc.cpu(), table.cpu(), lens.tolist(), n, D ** -0.5)
    nan = torch.isnan(want)
    assert nan.any() and torch.isinf(want).any() and torch.equal(torch.isnan(out.cpu()), nan)
    assert_close(out.nan_to_num(0, float("inf"), -float("inf")), want.masked_fill(nan, 0), "out")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_bad_page_is_left_out(dtype):
    q, kc, vc, table, lens = case(9, [100, 40], 4, 2, 128, 16, 1, dtype)
    table[0, 2], table[1, 0] = -1, kc.shape[0]
    assert check(q, kc, vc, table, lens, 1) == ops.DERR_PAGE


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_a_bad_length_skips_the_request(dtype, bad):
    q, kc, vc, table, lens = case(10, [100, 40, 30], 4, 2, 128, 16, 1, dtype)
    want, _ = attn_ref(q.cpu(), kc.cpu(), vc.cpu(), table.cpu(), lens.tolist(), 1, 0.1)
    lens[1] = bad
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ops.attn_decode(q, kc, vc, table, lens, 0, 0.1, out, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == ops.DERR_SEQ_LEN
    assert (out[1] == 7).all()
    assert_close(out[[0, 2]], want[[0, 2]], "the others")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_beyond_32_bits(dtype):
    """Cache rows past 2^31 elements."""
    hkv, D, page = 8, 128, 64
    pages = 2 ** 31 // (page * hkv * D) + 4
    kc, vc = (torch.zeros(pages, page, hkv, D, device=DEV, dtype=dtype) for _ in range(2))
    g = synth.generator(11, DEV)
    for c in (kc, vc):
        c[-3:] = torch.randn(3, page, hkv, D, generator=g, device=DEV).to(dtype)
    q = torch.randn(1, 16, D, generator=g, device=DEV).to(dtype)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device=DEV)
    out = torch.zeros(q.shape, device=DEV, dtype=dtype)
    ops.attn_decode(q, kc, vc, table, torch.tensor([150], dtype=torch.int32, device=DEV), 0, 0.1, out)
    torch.cuda.synchronize()
    want, _ = attn_ref(q.cpu(), kc[-3:].cpu(), vc[-3:].cpu(), torch.tensor([[2, 0, 1]]), [150], 1, 0.1)
    assert_close(out, want, "out")
