"""The line of prefixes of attn_decode_shared, walked on the host by the kernel's own functions (csrc/attn_line.cuh and
attn_decode.cuh, compiled for it): every tile of a prefix that some request sees is taken once, by the block where the
join looks for it; parts have places of their own, side by side; rows, heads and readers are the group's."""
import os
import shutil
import subprocess

import pytest

from state_cached_causal_gb300 import build as cbuild

SOURCE = r'''
#include "attn_line.cuh"
#include <map>
#include <set>
#include <stdio.h>
#include <stdlib.h>
#include <tuple>
#include <vector>
using namespace cconv;
static uint32_t state = 1;
static int pick(int n) { return (state = state * 1664525u + 1013904223u) / 65536u % n; }
#define CHECK(x) do { if (!(x)) { printf("call %d, line %d: %s\n", call, __LINE__, #x); return 1; } } while (0)

template <int ROWS>
static int walk(int call) {
  const int sizes[] = {0, 1, 2, 3, 16, 33, 64, 65, 130, 250}, pre[] = {0, 1, 64, 128, 129, 300, 1000, 9000};
  const int sms[] = {3, 10, 152};
  AttnArgs a = {};
  a.q_len = 1 + pick(4), a.G = 1 + pick(4), a.Hkv = 1 << pick(3), a.hw = a.Hkv, a.units = 1;
  a.table_width = 1024, a.page_size = 16, a.unit_rows = ROWS, a.prefix_tile = ROWS / 2, a.own_tile = 16;
  a.sms = sms[pick(3)], a.place_cost = 22, a.tile_cost = 15;
  a.start_places = pick(2) ? 8 : 3, a.pair_places = 1 + pick(2);
  std::vector<int> cu = {pick(3)}, prefix, lens(cu[0], 5);
  a.groups = 1 + pick(9);
  for (int g = 0; g < a.groups; ++g) {
    const int n = sizes[pick(10)], p = pick(20) ? pre[pick(8)] : -1 - pick(2), short_ = pick(4);
    for (int b = 0; b < n; ++b)
      lens.push_back(p > 0 && (short_ == 0 || (short_ == 1 && b < n / 2)) ? pick(p + a.q_len - 1) - (pick(9) == 0)
                                                                          : (p > 0 ? p : 0) + a.q_len - 1 + pick(50));
    cu.push_back(cu.back() + n);
    prefix.push_back(p);
  }
  lens.push_back(7);
  a.B = (int)lens.size(), a.seq_lens = lens.data(), a.cu_groups = cu.data(), a.prefix_lens = prefix.data();
  int64_t total = 0, units = 0, positions = 0;
  std::vector<int64_t> line, first;
  for (int g = 0; g < a.groups; ++g) {
    const AttnGroup s = attn_group_of(a, g);
    line.push_back(total), first.push_back(units);
    total += s.places(), units += s.units;
    int lead = -1;
    for (int b = cu[g]; b < cu[g + 1]; ++b)
      if (lead < 0 && lens[b] - (a.q_len - 1) >= prefix[g]) lead = b;
    CHECK((s.units > 0) == (prefix[g] > 0 && lead >= 0) && (prefix[g] <= 0 || s.lead == lead));
  }
  for (int b = 0; b < a.B; ++b) positions += attn_behind(a, b);
  const int64_t grid = line_runs(attn_prefix_sms(a, total, positions), total);
  CHECK(total == 0 || grid > 0);
  std::map<std::tuple<int, int64_t, int>, int> taken;
  std::set<int64_t> slots;
  for (int block = 0; block < grid; ++block) {
    LineRun r;
    r.p = block * total / grid, r.end = (block + 1) * total / grid, r.total = total, r.grid = grid;
    CHECK(r.end - r.p >= 2);
    int g = 0;
    while (r.p >= line[g] + attn_group_of(a, g).places()) ++g;
    r.g = g, r.line = line[g], r.unit = first[g], r.lead = attn_group_of(a, g).lead;
    LineSeg s;
    while (line_segment<ROWS>(a, block, r, s)) {
      const AttnGroup of = attn_group_of(a, r.g);
      const int64_t u = s.slot - block - first[r.g];
      CHECK(u >= 0 && u < of.units && s.h == u % a.Hkv && s.row0 == u / a.Hkv * ROWS);
      CHECK(s.first == cu[r.g] && s.prefix == prefix[r.g] && s.lead == of.lead);
      CHECK(s.rows > 0 && s.rows <= ROWS && s.row0 + s.rows <= of.rows && (s.rows == ROWS || s.row0 + s.rows == of.rows));
      CHECK(s.pair == (ROWS == 256 && s.rows > 128));
      CHECK(slots.insert(s.slot).second && s.slot < units + grid);
      CHECK(s.j0 >= 0 && s.j1 <= of.tiles);
      for (int j = s.j0; j < s.j1; ++j) {
        CHECK(taken.emplace(std::make_tuple(r.g, u, j), block).second);
        CHECK(attn_block_of(line[r.g] + of.place_of(u) + (int64_t)j * of.tile_places(u), total, grid) == block);
      }
    }
    CHECK(r.p == r.end);
  }
  size_t all = 0;
  for (int g = 0; g < a.groups; ++g) {
    const AttnGroup s = attn_group_of(a, g);
    all += s.units * (s.units > 0 ? s.tiles : 0);
    for (int64_t u = 0; u < s.units; ++u)          // a unit's parts: neighbouring blocks, each with tiles of it
      for (int j = 1; j < s.tiles; ++j) {
        const int d = taken[std::make_tuple(g, u, j)] - taken[std::make_tuple(g, u, j - 1)];
        CHECK(d == 0 || d == 1);
      }
  }
  CHECK(taken.size() == all);
  return 0;
}

int main() {
  for (int call = 0; call < 400; ++call)
    if (walk<256>(call) || walk<128>(call)) return 1;
  puts("ok");
}
'''


def test_every_tile_is_taken_once_where_the_join_looks(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    (tmp_path / "line.cu").write_text(SOURCE)
    exe = tmp_path / "line"
    r = subprocess.run([nvcc, *cbuild.CFLAGS, str(tmp_path / "line.cu"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.stdout.strip() == "ok", r.stdout
