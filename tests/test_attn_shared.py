"""attn_decode_shared and attn_decode_shared_q8 against softmax attention in 64 bits, each request over all its
positions: prefixes from one position to many tiles, units of few and of many rows, groups of every kind,
requests that do not see their prefix whole, pages that end inside a tile, head sizes, draft tokens, both cache
orders and types, large scores, values that are not finite, device-side errors.

Rounding: over a cache in bf16 a result is rounded once, as tests/test_attn_rounding.py derives it for
attn_decode (weights as two bf16 terms: 2^-11 of the norm against the rounded result of 64 bits); over one in 8
bits the request's own positions have weights of 11 bits (tests/test_q8_attn.py: 2^-9). That is the root of the
mean square over many values; a call of few has whole turned roundings: of N values N d / u are (d = 2^-15,
u = 2^-7 to 2^-8), 0.5 to 1 of 128, and one alone is off by a step, 2^-7 of its value at most. So one step of the
largest value is allowed besides.
"""
import pytest
import torch

from state_cached_causal_gb300 import ops, synth
from tests import _q8
from tests._mixers import assert_close, attn_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16
BAD = 2 ** 30


class Case:
    """`groups`: (prefix, lengths of its requests); `loose`: lengths of requests before and behind the groups. The
    block tables of a group's later requests name no page of the prefix (they are not read), unless `own_copy`
    (a request that does not see the prefix whole reads its own, so it has copies)."""

    def __init__(self, seed, groups, hq, hkv, D, page, n=1, q8=False, heads_first=False, big=1.0, loose=([], [])):
        g = synth.generator(seed, DEV)
        lens = list(loose[0]) + [x for _, ls in groups for x in ls] + list(loose[1])
        cu, first = [len(loose[0])], {}
        for _, ls in groups:
            cu.append(cu[-1] + len(ls))
        for (p, ls), a in zip(groups, cu):
            for b in range(a, a + len(ls)):
                first[b] = (a, p)
        width = max([(x + page - 1) // page for x in lens] + [(p + page - 1) // page for p, _ in groups] + [1]) + 2
        pages = len(lens) * width + 2
        if q8:
            self.kc, self.vc, self.ks, self.vs = _q8.cache_pair(g, (pages, page, hkv, D), heads_first)
        else:
            shape = (pages, hkv, page, D) if heads_first else (pages, page, hkv, D)
            self.kc, self.vc = (torch.randn(*shape, generator=g, device=DEV).to(BF16) for _ in range(2))
            if heads_first:
                self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = perm[:len(lens) * width].view(len(lens), width).clone().cpu()
        bytes_ = lambda t: t if t.dtype is not _q8.F8 else t.view(torch.uint8)      # noqa: E731
        parts = [bytes_(self.kc), bytes_(self.vc)] + ([self.ks, self.vs] if q8 else [])
        self.first, self.parts, self.page = first, parts, page
        self.full = table.clone()                         # what the reference reads
        self.copy_prefix()
        for b, x in enumerate(lens):
            used = (x + page - 1) // page
            whole = first.get(b, (b, 0))
            keep = used if b != whole[0] else max(used, (whole[1] + page - 1) // page)
            table[b, keep:] = BAD
            if b != whole[0] and x - (n - 1) >= whole[1]:
                table[b, :whole[1] // page] = BAD
            # rows that nobody holds
            held = max(x, whole[1]) if b == whole[0] else x
            for t, bad in zip(parts, (float("nan"), float("nan")) if not q8 else (0x7f, 0x7f, 255, 255)):
                rest = torch.arange(held, (held + page - 1) // page * page, device=DEV)
                t[self.full[b].to(DEV)[rest // page].long(), rest % page] = bad
        self.table, self.n, self.q8 = table.to(DEV), n, q8
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        self.prefix = torch.tensor([p for p, _ in groups], dtype=torch.int32, device=DEV)
        q = big * torch.randn(len(lens) * n, hq * D + 16, generator=g, device=DEV)
        self.q = q.to(BF16)[:, :hq * D].unflatten(1, (hq, D))
        self.scale = D ** -0.5

    def copy_prefix(self):
        """Every request's copy of the prefix as its group's first request has it."""
        for b, (a, p) in self.first.items():
            if b != a:
                for t in self.parts:
                    at = torch.arange(p, device=DEV)
                    src, dst = (self.full[i].to(DEV)[at // self.page].long() for i in (a, b))
                    t[dst, at % self.page] = t[src, at % self.page]

    def call(self, out, lse=None, stream=None, workspace=None, err=None):
        s = [self.ks, self.vs] if self.q8 else []
        fn = ops.attn_decode_shared_q8 if self.q8 else ops.attn_decode_shared
        fn(self.q, self.kc, self.vc, *s, self.table, self.lens, self.cu, self.prefix, self.n - 1, self.scale, out,
           lse=lse, dev_err=err, stream=stream, workspace=workspace)

    def want(self):
        k, v = _q8.in_64_bits(self.kc, self.vc, self.ks, self.vs) if self.q8 else (self.kc.cpu(), self.vc.cpu())
        return attn_ref(self.q.cpu(), k, v, self.full, self.lens.tolist(), self.n, self.scale)

    def run(self, **kw):
        out = torch.full(self.q.shape, 7.0, device=DEV, dtype=BF16)
        lse = torch.full(self.q.shape[:2], 7.0, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.call(out, lse, err=err, **kw)
        torch.cuda.synchronize()
        return out, lse, err.item()

    def check(self, **kw):
        out, lse, err = self.run(**kw)
        want, want_lse = self.want()
        assert_close(out, want, "out")
        if want.norm() > 0:
            off = (out.cpu().double() - want.to(BF16).double()).norm() / want.norm()
            step = 2.0 ** -7 * (want.abs().max() / want.norm()).item()
            assert off <= (2.0 ** -9 if self.q8 else 2.0 ** -11) + step, f"{off:.3g}"
        fin = torch.isfinite(want_lse)
        assert torch.equal(torch.isfinite(lse.cpu()), fin)
        # fp32 sums of exact products, magnitudes of a few tens at most
        assert torch.allclose(lse.cpu().double()[fin], want_lse[fin], rtol=1e-5, atol=1e-4)
        return err


both = pytest.mark.parametrize("q8", [False, True])


@both
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [1, 16, 63, 64, 127, 128, 129, 300, 1000])
def test_prefix_lengths(prefix, D, q8):
    lens = [prefix + 1, prefix + 40, prefix + 3]
    assert Case(1, [(prefix, lens)], 4, 2, D, 16, q8=q8).check() == 0


@both
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 4), (6, 2), (16, 1), (8, 8), (9, 3)])
def test_heads(D, hq, hkv, q8):
    assert Case(2, [(400, [401, 470])], hq, hkv, D, 16, q8=q8).check() == 0


@both
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("requests,group,n", [(30, 4, 1), (32, 4, 1), (33, 4, 1), (64, 4, 1), (65, 4, 1), (70, 8, 1),
                                              (20, 4, 4), (40, 2, 8)])
def test_row_units(requests, group, n, D, q8):
    """120 to 640 rows a kv head: one row tile, two, several units, the last one not full."""
    lens = [200 + n - 1 + (7 * i) % 30 for i in range(requests)]
    assert Case(3, [(200, lens)], group, 1, D, 16, n, q8=q8).check() == 0


@both
@pytest.mark.parametrize("n", [1, 2, 4, 8])
def test_requests_that_do_not_see_the_prefix_whole(n, q8):
    """Some shorter than the prefix, some whose first draft tokens lie in it, empty ones; the first of the group
    among them."""
    lens = [150, 150 + n - 1, 150 + n - 2, 1, 0, 149, 200, 40, 153]
    assert Case(4, [(150, lens)], 8, 2, 128, 16, n, q8=q8).check() == 0
    assert Case(5, [(150, [2, 170, 300])], 8, 2, 64, 16, n, q8=q8).check() == 0


@both
def test_groups(q8):
    """Groups of one, empty ones, ones without a prefix, of many sizes; requests in no group."""
    groups = [(70, [90]), (33, []), (0, [5, 100]), (500, [501, 640, 500, 777]), (1, [2, 30]), (128, [129] * 9),
              (0, []), (64, [80, 90, 100])]
    assert Case(6, groups, 8, 4, 64, 16, 1, q8, loose=([17, 0], [60, 1, 2])).check() == 0
    many = [((13 * i) % 90, [(13 * i) % 90 + 1 + (i + j) % 40 for j in range(i % 4)]) for i in range(60)]
    assert Case(7, many, 4, 2, 64, 16, 1, q8).check() == 0
    assert Case(8, [], 4, 2, 64, 16, 1, q8, loose=([30, 5], [])).check() == 0


@both
@pytest.mark.parametrize("page", [1, 7, 16, 48, 128])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 64), (4, 4, 128), (3, 1, 64), (2, 2, 256)])
def test_pages(page, heads_first, hq, hkv, D, q8):
    assert Case(9, [(190, [191, 260, 203]), (6, [9, 30])], hq, hkv, D, page, 1, q8, heads_first).check() == 0


@both
def test_long_prefixes_cut_between_many_blocks(q8):
    assert Case(10, [(20000, [20001, 20050]), (3000, [3001, 3002])], 8, 4, 128, 64, 2, q8).check() == 0
    assert Case(11, [(9000, [9100 + i for i in range(40)])], 16, 2, 64, 64, 1, q8).check() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [1.0, -0.7, 0.0])
def test_large_scores_and_signs(scale, D):
    """Maxima that rise by far more than the slack from tile to tile; weights of the smallest score; all alike."""
    c = Case(12, [(700, [701, 720, 1000])], 4, 1, D, 16, big=3.0)
    c.kc *= torch.linspace(0.1, 2, c.kc.shape[0], device=DEV)[:, None, None, None].to(BF16)
    c.kc.nan_to_num_(0)
    c.vc.nan_to_num_(0)
    c.copy_prefix()
    c.scale = scale
    out, lse, err = c.run()
    want, want_lse = c.want()
    assert err == 0
    # scores of up to several hundred: an fp32 score is off by 2^-24 of that, and its weight by as much
    assert_close(out, want, "out")
    assert torch.allclose(lse.cpu().double(), want_lse, rtol=1e-5, atol=1e-3)


@both
def test_values_that_are_not_finite(q8):
    """An infinity or NaN among the prefix's values makes its column so for all rows that see it."""
    c = Case(13, [(300, [301, 350, 20])], 4, 2, 64, 16, 1, q8)
    at = int(c.table[0, 5])
    if q8:
        c.vc.view(torch.uint8)[at, 3, :, 7] = 0x7f
    else:
        c.vc[at, 3, :, 7], c.vc[at, 4, 0, 9] = float("inf"), float("nan")
    other = [int(c.full[b, 5]) for b in (1, 2)]
    for b in other:
        c.vc.view(torch.uint8 if q8 else BF16)[b] = c.vc.view(torch.uint8 if q8 else BF16)[at]
    out, _, _ = c.run()
    want, _ = c.want()
    out = out.cpu()
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.isnan(want).any()
    assert torch.equal(out.double()[torch.isinf(want)], want[torch.isinf(want)])
    fin = torch.isfinite(want)
    assert_close(out[fin], want[fin], "the others")


def test_keys_that_are_nan():
    c = Case(14, [(300, [301, 350])], 4, 2, 64, 16)
    c.kc[int(c.table[0, 9]), 3, 1] = float("nan")
    out, lse, _ = c.run()
    assert torch.isnan(out[:, 2:]).all() and torch.isnan(lse[:, 2:]).all()
    assert not torch.isnan(out[:, :2]).any()


@both
def test_other_stream_and_callers_workspace(q8):
    c = Case(15, [(500, [520, 600, 501])], 16, 4, 128, 16, 1, q8)
    ws = torch.full((ops.attn_decode_shared_workspace_bytes(3, 1, 0, 16, 4, 128),), 255, dtype=torch.uint8,
                    device=DEV)
    torch.cuda.synchronize()
    assert c.check(stream=torch.cuda.Stream(), workspace=ws) == 0


@both
def test_the_same_every_time_and_replayed(q8):
    """A graph whose lengths and groups change between replays, too."""
    c = Case(16, [(3000, [3100, 3001, 3500]), (100, [130, 200])], 16, 4, 128, 16, 1, q8)
    ws = torch.empty(ops.attn_decode_shared_workspace_bytes(5, 2, 0, 16, 4, 128), dtype=torch.uint8, device=DEV)
    out = torch.zeros(c.q.shape, device=DEV, dtype=BF16)
    got = []
    for _ in range(2):
        out.zero_()
        c.call(out, workspace=ws)
        torch.cuda.synchronize()
        got.append(out.clone())
    assert torch.equal(got[0], got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(out, workspace=ws)
    out.zero_()
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out)
    c.lens.copy_(torch.tensor([3050, 2000, 3400, 120, 101], dtype=torch.int32))
    c.prefix.copy_(torch.tensor([2999, 97], dtype=torch.int32))
    c.table[1] = c.full[1].to(DEV)
    for b, a, p in ((2, 0, 2999), (4, 3, 97)):          # the page that the prefix now ends in
        c.table[b, p // 16] = c.full[b, p // 16]
    graph.replay()
    torch.cuda.synchronize()
    want, _ = c.want()
    assert_close(out, want, "replayed with other lengths")


@both
def test_against_attn_decode(q8):
    """The same call without the groups."""
    c = Case(17, [(1000, [1001 + 9 * i for i in range(20)])], 8, 2, 128, 16, 1, q8)
    out, lse, err = c.run()
    plain, plain_lse = torch.zeros_like(out), torch.zeros_like(lse)
    s = [c.ks, c.vs] if q8 else []
    (ops.attn_decode_q8 if q8 else ops.attn_decode)(c.q, c.kc, c.vc, *s, c.full.to(DEV), c.lens, 0, c.scale, plain,
                                                    plain_lse)
    torch.cuda.synchronize()
    assert ((out.double() - plain.double()).norm() / plain.double().norm()).item() < 2.0 ** -8
    assert torch.allclose(lse, plain_lse, rtol=1e-5, atol=1e-4)


# ---- what only the device sees -----------------------------------------------

@both
def test_a_bad_page_of_the_prefix_is_left_out(q8):
    c = Case(18, [(200, [201, 260])], 4, 2, 64, 16, 1, q8)
    c.table[0, 3] = -1
    c.full[:, 3] = -1
    out, _, err = c.run()
    assert err == ops.DERR_PAGE
    assert_close(out, c.want()[0], "out")


@both
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_a_bad_length_skips_the_request(bad, q8):
    c = Case(19, [(200, [201, 260, 300])], 4, 2, 64, 16, 1, q8)
    want, _ = c.want()
    c.lens[1] = bad
    out, lse, err = c.run()
    assert err == ops.DERR_SEQ_LEN
    assert (out[1] == 7).all() and (lse[1] == 7).all()
    assert_close(out[[0, 2]], want[[0, 2]], "the others")


@both
@pytest.mark.parametrize("prefix,cu", [([-5, 64], None), ([10 ** 7, 64], None), (None, [0, 9, 5]), (None, [-2, 3, 5]),
                                       (None, [0, 3, 70])])
def test_bad_groups_count_as_ones_without_a_prefix(prefix, cu, q8):
    c = Case(20, [(100, [101, 120, 130]), (64, [70, 90])], 4, 2, 64, 16, 1, q8)
    c.table = c.full.to(DEV)                       # every request has its pages
    if prefix is not None:
        c.prefix.copy_(torch.tensor(prefix, dtype=torch.int32))
    if cu is not None:
        c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    out, _, err = c.run()
    assert err & ops.DERR_GROUP and not err & ops.DERR_TIMEOUT
    assert_close(out, c.want()[0], "out")


def test_groups_that_overlap_are_reported():
    c = Case(21, [(64, [70] * 40)] * 3, 16, 1, 64, 16)
    c.cu.copy_(torch.tensor([0, 120, 120, 120], dtype=torch.int32))
    c.table = c.full.to(DEV)
    c.prefix.fill_(64)
    assert c.run()[2] == 0                         # (the others are empty)
    c.cu.copy_(torch.tensor([0, 120, 0, 120], dtype=torch.int32))
    out, _, err = c.run()
    assert err & ops.DERR_GROUP and not err & ops.DERR_TIMEOUT


def test_padded_batch():
    """Rows behind the last request stay as they were; requests of length 0 write zeros."""
    c = Case(22, [(100, [101, 0, 130])], 4, 2, 64, 16)
    more = torch.cat([c.q, c.q], 0)
    out = torch.full(more.shape, 7.0, device=DEV, dtype=BF16)
    ops.attn_decode_shared(more, c.kc, c.vc, c.table, c.lens, c.cu, c.prefix, 0, c.scale, out)
    torch.cuda.synchronize()
    assert_close(out[:3], c.want()[0], "out")
    assert (out[1] == 0).all() and (out[3:] == 7).all()


def test_offsets_beyond_32_bits():
    """Cache rows past 2^31 elements."""
    hkv, D, page = 8, 128, 64
    pages = 2 ** 31 // (page * hkv * D) + 8
    kc, vc = (torch.zeros(pages, page, hkv, D, device=DEV, dtype=BF16) for _ in range(2))
    g = synth.generator(11, DEV)
    for c in (kc, vc):
        c[-6:] = torch.randn(6, page, hkv, D, generator=g, device=DEV).to(BF16)
    q = torch.randn(2, 16, D, generator=g, device=DEV).to(BF16)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2, pages - 5], [BAD, BAD, pages - 4, pages - 6]],
                         dtype=torch.int32, device=DEV)
    full = torch.tensor([[5, 3, 4, 1], [5, 3, 2, 0]])
    out = torch.zeros(q.shape, device=DEV, dtype=BF16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)         # noqa: E731
    ops.attn_decode_shared(q, kc, vc, table, i32(150, 200), i32(0, 2), i32(128), 0, 0.1, out)
    torch.cuda.synchronize()
    want, _ = attn_ref(q.cpu(), kc[-6:].cpu(), vc[-6:].cpu(), full, [150, 200], 1, 0.1)
    assert_close(out, want, "out")
