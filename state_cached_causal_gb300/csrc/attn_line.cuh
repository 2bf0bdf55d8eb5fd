// The prefixes' line (attn_shared.cu, attn_decode.cuh) as a block walks it: what its run
// holds of which unit, and where the parts of that go. Also compiled for the host, where
// every run of a call can be walked.
#pragma once

#include "attn_decode.cuh"

namespace cconv {

// Blocks that have a run: no run is shorter than two places.
__host__ __device__ __forceinline__ int64_t line_runs(int64_t sms, int64_t total) {
  return sms < total / 2 ? sms : total / 2;
}

struct LineRun {
  int64_t p, end, total, grid;
  int64_t line, unit;         // of group g: its first place and unit
  int g, lead;                // (its first request that sees the prefix)
};

// One segment: tiles [j0, j1) of a unit: rows [row0, row0 + rows) of group g and kv head h.
struct LineSeg {
  int first, prefix;          // the group's first request, and its prefix
  int lead;                   // the request whose table names the prefix
  int h, j0, j1, rows, row0;
  int64_t slot;
  bool pair;                  // two row tiles on the same positions
};

// The next segment of block `block`'s run; false behind the last. ROWS: of a unit.
template <int ROWS>
__host__ __device__ __forceinline__ bool line_segment(const AttnArgs& a, int block, LineRun& r,
                                                      LineSeg& s) {
  while (r.p < r.end) {
    AttnGroup g = attn_group_of<true>(a, r.g);
    while (r.p >= r.line + g.places()) {      // (groups without units, too)
      r.line += g.places();
      r.unit += g.units;
      g = attn_group_of(a, ++r.g);
      r.lead = g.lead;
    }
    int64_t rel = r.p - r.line;
    const bool whole = rel < g.full * g.per_full;
    if (!whole) rel -= g.full * g.per_full;
    const int per = whole ? g.per_full : g.per, wide = whole ? g.pair : g.wide;
    // (a 64-bit division takes a hundred instructions)
    int u = rel <= INT32_MAX ? (int)((uint32_t)rel / (uint32_t)per) : (int)(rel / per);
    const int off = (int)(rel - (int64_t)u * per);
    const int64_t left = r.end - r.p;
    const int take = per - off < left ? per - off : (int)left;
    r.p += take;
    // (wide is 1 or 2)
    const int from = off - g.start + wide - 1, to = from + take;
    s.j0 = (from > 0 ? from : 0) >> (wide - 1);
    s.j1 = (to > 0 ? to : 0) >> (wide - 1);
    if (s.j1 <= s.j0) continue;
    if (!whole) u += (int)g.full;
    const int mt = u / a.Hkv;
    s.first = g.first, s.prefix = g.prefix, s.lead = r.lead;
    s.h = u - mt * a.Hkv;
    s.row0 = mt * ROWS;
    const int behind = (int)g.rows - s.row0;
    s.rows = behind < ROWS ? behind : ROWS;
    s.pair = ROWS == 256 && s.rows > 128;
    // from one segment to the next the unit's number or the block's rises
    s.slot = r.unit + u + block;
    return true;
  }
  return false;
}

}  // namespace cconv
