"""attn_decode_shared where a group's first request does not see the prefix whole: an empty or finished one, a short
one, one of a refused length. The prefix is read through the block table of the first request that does see it, and
not at all where none does: entries of a table beyond a request's length are anything, as for attn_decode. And the
SMs are divided by the positions that requests have left when each counts what it sees.
"""
import os
import shutil
import subprocess

import pytest
import torch

from state_cached_causal_gb300 import build as cbuild
from state_cached_causal_gb300 import ops
from tests._mixers import assert_close
from tests.test_attn_shared import BAD, DEV, Case

both = pytest.mark.parametrize("q8", [False, True])


def own_tables(c, stale):
    """Every request's table names what it holds itself; behind that its entries are `stale`."""
    c.table = c.full.clone()
    for b, x in enumerate(c.lens.tolist()):
        c.table[b, (max(x, 0) + c.page - 1) // c.page:] = stale
    c.table = c.table.to(DEV)


@pytest.mark.gpu
@both
@pytest.mark.parametrize("stale", [-1, BAD, 0, 3])
@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("first", [0, 1, 150, 202])
def test_a_first_request_that_is_too_short(first, n, stale, q8):
    for D in (64, 128, 256):
        c = Case(1, [(203, [first, 230, 5, 204 + n]), (300, [0, 0, 301 + n, 500]), (64, [63, 30])], 8, 2, D, 16, n, q8)
        own_tables(c, stale)
        assert c.check() == 0


@pytest.mark.gpu
@both
@pytest.mark.parametrize("stale", [-1, 2])
def test_a_first_request_of_a_refused_length(stale, q8):
    c = Case(2, [(203, [250, 230, 240])], 8, 2, 128, 16, 1, q8)
    want, _ = c.want()
    c.lens[0] = -3
    own_tables(c, stale)
    out, _, err = c.run()
    assert err == ops.DERR_SEQ_LEN
    assert (out[0] == 7).all()
    assert_close(out[1:], want[1:], "the others")


@pytest.mark.gpu
@both
def test_no_request_sees_the_prefix(q8):
    """Not even a page of it is looked at."""
    c = Case(3, [(4096, [100 + 37 * i for i in range(70)])], 16, 4, 128, 16, 1, q8)
    own_tables(c, BAD)
    assert c.check() == 0


@pytest.mark.gpu
@both
def test_pages_that_only_the_first_request_names(q8):
    """As where later tables begin behind the prefix: the first request's table is read."""
    c = Case(4, [(203, [20, 230, 250])], 8, 2, 128, 16, 1, q8)      # (tables of 1 and 2 name no page of the prefix)
    assert c.check() == 0
    c.table[0, 4] = c.table[1, 4] = -1                              # nobody does
    c.full[1:, 4] = -1
    out, _, err = c.run()
    assert err == ops.DERR_PAGE
    assert_close(out, c.want()[0], "out")


def test_sms_by_what_requests_see(tmp_path):
    """The counts that the SMs are divided by, from the kernels' own functions compiled for the host: a request that
    does not see its prefix whole counts in full, and a prefix that nobody sees is no work."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "sms.cu"
    src.write_text(r'''
#include "attn_decode.cuh"
#include <stdio.h>
int main() {
  using namespace cconv;
  const int cu[] = {2, 66, 66, 76}, prefix[] = {4096, 100, 512};
  for (int seen = 0; seen <= 64; seen += 32) {
    int32_t lens[80];
    for (int b = 0; b < 80; ++b) lens[b] = b < 2 || b >= 66 ? 600 : b - 2 < 64 - seen ? 4000 : 4100;
    lens[70] = -1;
    AttnArgs a = {};
    a.seq_lens = lens, a.cu_groups = cu, a.prefix_lens = prefix, a.groups = 3;
    a.B = 80, a.q_len = 2, a.G = 4, a.Hkv = 4, a.hw = 4, a.units = 1, a.table_width = 400, a.page_size = 16;
    a.unit_rows = 256, a.prefix_tile = 128, a.own_tile = 16, a.start_places = 8, a.pair_places = 2;
    a.sms = 152, a.place_cost = 22, a.tile_cost = 15;
    int64_t places = 0, positions = 0;
    for (int g = 0; g < 3; ++g) places += attn_group_of(a, g).places();
    for (int b = 0; b < 80; ++b) positions += attn_behind(a, b);
    printf("%d %lld %lld %d %d\n", seen, (long long)places, (long long)positions, attn_group_of(a, 0).lead,
           attn_prefix_sms(a, places, positions));
  }
}
''')
    exe = tmp_path / "sms"
    subprocess.run([nvcc, *cbuild.CFLAGS, str(src), "-o", str(exe)], check=True, capture_output=True)
    rows = [[int(x) for x in line.split()] for line in
            subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    third = 4 * (8 + 1 * 4)                             # 10 requests x 8 rows: a unit a kv head, one row tile
    first = 4 * (8 + 2 * 32) * 2                        # 64 x 8 rows: two units of two row tiles
    for seen, places, positions, lead, sms in rows:
        assert places == third + (first if seen else 0)
        assert positions == 6 * 600 + 9 * (600 - 512) + (64 - seen) * 4000 + seen * (4100 - 4096)
        assert lead == (2 + 64 - seen if seen else -1)
    few, some, all_ = (r[4] for r in rows)
    assert few < 16 and some < 40 and all_ > 60
