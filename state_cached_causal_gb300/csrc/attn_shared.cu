// Entry points attn_decode_shared and attn_decode_shared_q8: attention of new tokens
// where groups of requests share their first positions.
//
// Three launches. attn_prefix_kernel multiplies a group's prefix once, for the rows of
// all its requests; the kernels of attn_decode take each request's positions behind
// it (from attn_start on); attn_shared_join_kernel joins both. The second runs beside the
// first, whose results it does not need: the SMs are divided between the two by their
// work (attn_prefix_sms).
//
// attn_prefix_kernel. The rows of a group and kv head (requests x new tokens x query
// heads of the kv head) are cut into units of 256 (128 for heads of 256), a unit's
// prefix into tiles of 128 positions (64). All tiles of the call form a line, which
// the grid's blocks, one an SM, cut into equal runs, as in attn_decode.cuh; with
// several row units the blocks that hold the same tiles of each walk them at the same
// time, so that K and V come from memory once and from the L2 for the others. A
// block's warps:
// - four copy K and V of a tile, row by row wherever its page lies, into a ring in the
//   128-byte swizzle (from 8 bits: by way of a place of bytes, converted to bf16, exactly);
// - one issues the products on tcgen05: scores S = Q K^T into tensor memory, then
//   O += P V with P from tensor memory, O in tensor memory;
// - two times four are a softmax each, a row a thread: maximum and weights of a tile of
//   scores, weights as two bf16 terms (16 bits, so that a result is rounded once) in
//   place of the scores. A maximum that has risen by less than 2^8 leaves the sums
//   as they are; otherwise the thread multiplies its row of O first.
// Two streams of tiles alternate, so that one's softmax runs behind the other's
// products: the two row tiles of 128 on the same K and V, or, where the unit has no
// more than 128 rows, the even and the odd tiles of positions on the same rows. (Heads
// of 256 leave tensor memory for one stream.)
//
// With many rows it is bound by the products (scores, and twice the weights'), with few
// by the bytes of K and V, from 8 bits by their conversion to bf16 in the copying warps.
// 16 query heads on 4 kv heads of 128: 256 requests behind 32768 positions, with up to
// 1024 of their own (338 MB, 70 GFLOP and a half more for the weights' second terms)
// 146 us; a tile for two row tiles takes a block 2.5 us, 10 TFLOP/s, 0.9 of what cuBLAS
// keeps up an SM. 8 requests behind 131072 positions 74 us for 270 MB, of which 10 to 13
// are before the first products (code, page table, copies) and 9 the join; seven groups of
// 96 requests with 4 tokens, from 8 bits, 95 us. Attended one by one (attn_decode) the
// first would read 17.5 GB.
#include "attn_line.cuh"
#include "q8.cuh"
#include "tc.cuh"

#include <math.h>

namespace cconv {
namespace {

constexpr int kSoftWarps = 4;                     // of a stream
constexpr int kCopyWarp0 = 2 * kSoftWarps, kCopyWarps = 4;
constexpr int kMmaWarp = kCopyWarp0 + kCopyWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kMasks = 16;                        // tiles whose masks are kept
constexpr long long kWaitClocks = 4000000000LL;   // seconds; a tile takes microseconds
constexpr float kSlack = 8.0f;                    // log2 of how far a weight may pass 1

struct Rec {          // a group's place on the line and among the units (-1: not taken)
  int64_t line;
  int32_t unit, tiles;
};

struct PrefixArgs {
  AttnArgs a;
  Rec* rec;           // [groups + 1]: of each group; the line's length and its runs
  float* po;          // [units + grid][NT * 128][D]: weighted values
  float2* ps;         // [units + grid][NT * 128]: maximum (natural), sum
  int64_t max_units;
  int32_t grid;
};

template <int D, bool Q8 = false>
struct Shape {
  static constexpr int NT = D == 256 ? 1 : 2;            // streams
  static constexpr int kRowsU = 128 * NT;                // rows of a unit
  static constexpr int kN = D == 256 ? 64 : 128;         // positions of a tile
  static constexpr int kPanelQ = 128 * 128;              // 64 dims of 128 rows
  static constexpr int kPanel = kN * 128;                // 64 dims of a tile
  static constexpr int kQ = D / 64 * kPanelQ;
  static constexpr int kStage = D / 64 * kPanel;
  static constexpr int kRaw = Q8 ? 4 : 0;                // items of bytes on their way
  static constexpr int kStages = (D == 64 ? 8 : 5) - kRaw / 2;
};

struct Ctl {
  uint64_t full[8], empty[8];
  uint64_t q_full[2], s_full[2], p_full[2][4], o_full[2], fin;
  int64_t scan[3 * (kThreads / 32)];
  uint32_t mask[kMasks][kCopyWarps];
  uint32_t tmem;
  int dead;
};

// Bounded wait of a whole warp; once one of a block's waits has been given up, all are.
struct Wait {
  volatile int* dead;
  int32_t* err;
  __device__ __forceinline__ bool operator()(uint64_t* bar, int phase) const {
    long long t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1; !__any_sync(0xffffffffu, mbar_try(bar, (uint32_t)phase & 1u)); ++it) {
      if ((it & 63u) == 0) {
        const long long now = clock64();
        if (t0 == 0) t0 = now;
        const bool late = now - t0 > kWaitClocks;
        if (__any_sync(0xffffffffu, late || *dead != 0)) {
          if (late) flag_error(err, CCONV_DERR_TIMEOUT);
          *dead = 1;
          return false;
        }
      }
    }
    __syncwarp();
    return true;
  }
};

// ---- the line -------------------------------------------------------------------

// As attn_split, over the groups. The first block notes every group for the join.
template <int D>
__device__ __forceinline__ bool split(const PrefixArgs& x, int64_t* sm, LineRun& r) {
  const AttnArgs& a = x.a;
  const int tid = threadIdx.x, per = (a.groups + kThreads - 1) / kThreads;
  const int g0 = min(a.groups, tid * per), g1 = min(a.groups, g0 + per);
  int64_t lines = 0, units = 0, own = 0;      // own: positions behind the prefixes
#pragma unroll 1
  for (int b = tid; b < a.B; b += kThreads) own += attn_behind(a, b);
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    const AttnGroup s = attn_group_of(a, g);
    lines += s.places();
    units += s.units;
    if (blockIdx.x == 0 &&
        !attn_group_ok(a, a.cu_groups[g], a.cu_groups[g + 1], a.prefix_lens[g]))
      flag_error(a.dev_err, CCONV_DERR_GROUP);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) own += __shfl_xor_sync(0xffffffffu, own, d);
  int64_t li = lines, ui = units;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t l = __shfl_up_sync(0xffffffffu, li, d), u = __shfl_up_sync(0xffffffffu, ui, d);
    if ((tid & 31) >= d) li += l, ui += u;
  }
  constexpr int kWarps = kThreads / 32;
  if ((tid & 31) == 31)
    sm[tid >> 5] = li, sm[kWarps + (tid >> 5)] = ui, sm[2 * kWarps + (tid >> 5)] = own;
  __syncthreads();
  own = 0;
  int64_t lb = 0, ub = 0, ls = 0, us = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < (tid >> 5)) lb += sm[w], ub += sm[kWarps + w];
    ls += sm[w], us += sm[kWarps + w], own += sm[2 * kWarps + w];
  }
  li += lb - lines, ui += ub - units;         // before this thread's groups
  // (groups that overlap may have more rows than the call: none is taken then)
  const bool fits = us <= x.max_units;
  r.total = fits ? ls : 0;
  r.grid = line_runs(attn_prefix_sms(a, ls, own), r.total);
  if (blockIdx.x == 0) {
    if (!fits && tid == 0) flag_error(a.dev_err, CCONV_DERR_GROUP);
    if (tid == 0) x.rec[a.groups] = Rec{r.total, (int32_t)r.grid, 0};
    int64_t l = li, u = ui;
    for (int g = g0; g < g1; ++g) {
      const AttnGroup s = attn_group_of(a, g);
      x.rec[g] = Rec{l, fits && s.units > 0 ? (int32_t)u : -1, s.tiles};
      l += s.places(), u += s.units;
    }
  }
  r.p = blockIdx.x < r.grid ? blockIdx.x * r.total / r.grid : r.total;
  r.end = blockIdx.x < r.grid ? (blockIdx.x + 1) * r.total / r.grid : r.total;
  __syncthreads();
  if (lines > 0 && r.p >= li && r.p < li + lines) {
    int g = g0;
    for (;; ++g) {
      const AttnGroup s = attn_group_of(a, g);
      sm[3] = s.lead;
      if (r.p < li + s.places()) break;
      li += s.places(), ui += s.units;
    }
    sm[0] = g, sm[1] = li, sm[2] = ui;
  }
  __syncthreads();
  r.g = (int)sm[0], r.line = sm[1], r.unit = sm[2], r.lead = (int)sm[3];
  return r.p < r.end;
}

// ---- copies ---------------------------------------------------------------------

// Item i of a segment of n tiles: which tile, K or V, in the order the products take them.
struct Item {
  int tile;
  bool isv;
};
__device__ __forceinline__ Item item_of(int i, int n, bool split) {
  if (!split) return {i >> 1, (i & 1) != 0};
  if (i < min(n, 2)) return {i, false};                 // K0, K1
  if (n == 1) return {0, true};
  const int k = i - 2;
  if ((k & 1) && (k >> 1) + 2 < n) return {(k >> 1) + 2, false};
  return {i == 2 * n - 1 ? n - 1 : k >> 1, true};
}

// Place of 16-byte unit u of row r in a tile.
template <int PANEL>
__device__ __forceinline__ uint32_t place(int r, int u) {
  return (u >> 3) * PANEL + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}

// What the copies know of an item, from the lane that has its row on.
struct Piece {
  int page;             // as the table has it
  int tok, h;           // token of the page, kv head
  int seq;              // the tile's number, as masks are kept by
  bool isv, there;      // V; false: behind the last item
  bool row;             // the lane has a row of the prefix
};
struct Row {
  int64_t at;           // where its values begin (-1: none, zeros)
  float f;              // their scale
};

template <int D, bool Q8>
__device__ __forceinline__ bool copy_role(const PrefixArgs& x, LineRun run, Ctl& c,
                                          unsigned char* ring, unsigned char* raw,
                                          const Wait& wait) {
  using S = Shape<D, Q8>;
  const AttnArgs& a = x.a;
  constexpr int kRowsW = S::kN / kCopyWarps;            // rows of a warp: lane r has row r's
  constexpr int kRowBytes = D * (Q8 ? 1 : 2), kLanes = kRowBytes / 16;   // of a row
  constexpr int kPer = 32 / kLanes, kPasses = kRowsW / kPer;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kCopyWarp0;
  const int sub = lane / kLanes, u = lane % kLanes;
  // The items one after the other, over the run's segments: pages are looked up, and
  // scales and (in 8 bits) values requested, some items before they are needed.
  LineSeg s;
  int i = 0, n = 0, seq = 0;
  bool more = true;
  auto next = [&]() {
    Piece p = {-1, 0, 0, 0, false, false, false};
    if (more && i == 2 * n) {
      seq += n;
      i = 0;
      more = line_segment<Shape<D>::kRowsU>(x.a, blockIdx.x, run, s);
      n = more ? s.j1 - s.j0 : 0;
      if (more && s.lead != s.first &&
          (uint32_t)a.table[(int64_t)s.lead * a.table_rs] >= (uint32_t)a.num_pages)
        s.lead = s.first;
    }
    if (!more) return p;
    const Item m = item_of(i++, n, S::NT == 2 && !s.pair);
    const int pos = (s.j0 + m.tile) * S::kN + w * kRowsW + lane;
    p.h = s.h;
    p.seq = seq + m.tile;
    p.isv = m.isv;
    p.there = true;
    if (lane < kRowsW && pos < s.prefix) {
      const int at = a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
      p.tok = a.page_shift >= 0 ? pos & (a.page_size - 1) : pos - at * a.page_size;
      p.row = true;
      p.page = a.table[(int64_t)s.lead * a.table_rs + at];
    }
    return p;
  };
  auto row_of = [&](const Piece& p) {
    Row r = {-1, 0.0f};
    if (p.row && (uint32_t)p.page >= (uint32_t)a.num_pages) {
      if (!p.isv) flag_error(a.dev_err, CCONV_DERR_PAGE);
    } else if (p.row) {
      r.at = p.page * a.s_page + p.tok * a.s_tok + (int64_t)p.h * a.s_head;
      if constexpr (Q8)
        r.f = q8_scale((p.isv ? a.vsc : a.ksc)[p.page * a.c_page + p.tok * a.c_tok +
                                               (int64_t)p.h * a.c_head]);
    }
    return r;
  };
  auto note = [&](const Piece& p, const Row& row) {
    if (p.isv) return;
    const uint32_t mask = __ballot_sync(0xffffffffu, row.at >= 0);
    if (lane == 0) c.mask[p.seq % kMasks][w] = mask;
  };
  if constexpr (!Q8) {
    Piece now = next(), then = next();
#pragma unroll 1
    for (int it = 0; now.there; ++it) {
      const int st = it % S::kStages;
      const Row row = row_of(now);
      const Piece after = next();
      const char* const base = now.isv ? a.vc : a.kc;
      if (!wait(&c.empty[st], (it / S::kStages & 1) ^ 1)) return false;
      note(now, row);
      const uint32_t dst = smem_addr(ring) + st * S::kStage;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int r = p * kPer + sub;
        const int64_t at = __shfl_sync(0xffffffffu, row.at, r);
        cp_async16(dst + place<S::kPanel>(w * kRowsW + r, u),
                   base + (at >= 0 ? at * 2 + u * 16 : 0), at >= 0);
      }
      // (arrives when the thread's copies have; the products' warp orders them before
      // its own reads)
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                       smem_addr(&c.full[st]))
                   : "memory");
      now = then, then = after;
    }
  } else {
    // An item's bytes come by copies of the thread that converts them, to a place of its
    // own, three items ahead; pages are looked up an item before that. (With the bytes
    // of one item on their way, in registers, the copies' latency was what a tile took.)
    const uint32_t mine = smem_addr(raw) + (threadIdx.x - kCopyWarp0 * 32) * 16;
    auto issue = [&](const Piece& p, int it) {
      const Row row = row_of(p);
      const char* const base = p.isv ? a.vc : a.kc;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int64_t at = __shfl_sync(0xffffffffu, row.at, k * kPer + sub);
        cp_async16(mine + (it % S::kRaw * kPasses + k) * (kCopyWarps * 512),
                   base + (at >= 0 ? at + u * 16 : 0), at >= 0);
      }
      cp_async_commit();
      return row;
    };
    Piece p0 = next(), p1 = next(), p2 = next(), p3 = next();
    Row r0 = issue(p0, 0), r1 = issue(p1, 1), r2 = issue(p2, 2);
#pragma unroll 1
    for (int it = 0; p0.there; ++it) {
      const int st = it % S::kStages;
      const Row r3 = issue(p3, it + 3);
      const Piece p4 = next();
      cp_async_wait<3>();
      if (!wait(&c.empty[st], (it / S::kStages & 1) ^ 1)) return false;
      note(p0, r0);
      unsigned char* const dst = ring + st * S::kStage;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int r = p * kPer + sub;
        const float k = __shfl_sync(0xffffffffu, r0.f, r);
        uint32_t v[4], o[8];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(mine + (it % S::kRaw * kPasses + p) * (kCopyWarps * 512))
                     : "memory");
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[4];
          unpack_e4m3x4(v[e], y);
          o[2 * e] = pack_bf16x2(y[0] * k, y[1] * k);
          o[2 * e + 1] = pack_bf16x2(y[2] * k, y[3] * k);
        }
        *reinterpret_cast<uint4*>(dst + place<S::kPanel>(w * kRowsW + r, 2 * u)) =
            make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + place<S::kPanel>(w * kRowsW + r, 2 * u + 1)) =
            make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async();
      mbar_arrive(&c.full[st]);
      p0 = p1, p1 = p2, p2 = p3, p3 = p4;
      r0 = r1, r1 = r2, r2 = r3;
    }
  }
  return true;
}

// ---- products -------------------------------------------------------------------

constexpr int kColS = 0, kColO = 256;      // of tensor memory: scores of both streams, sums

// The order in which a softmax turns 32 scores after the other into weights: those first
// that its first pass read last.
template <int N>
__host__ __device__ constexpr int chunk_at(int j) {
  return N / 32 - 1 - j;
}

template <int D, bool Q8>
__device__ __forceinline__ bool mma_role(const PrefixArgs& x, LineRun run, Ctl& c, uint32_t q_addr,
                                         uint32_t ring, const Wait& wait, uint32_t tmem) {
  using S = Shape<D, Q8>;
  constexpr uint32_t kIdS = tc::idesc(128, S::kN), kIdO = tc::idesc(128, D, false, true);
  const uint64_t q0 = tc::desc_sw128(q_addr, 16);
  const uint64_t k0 = tc::desc_sw128(ring, 16), v0 = tc::desc_sw128(ring, S::kPanel);
  int it = 0, segs[2] = {0, 0}, ps[2] = {0, 0};
  auto filled = [&](int i) {
    if (!wait(&c.full[i % S::kStages], i / S::kStages)) return false;
    fence_proxy_async();          // (per-thread copies come by the generic proxy)
    return true;
  };
  // scores of stream s from item i, its Q being tile qt
  auto scores = [&](int s, int qt, int i) {
    const uint64_t q = q0 + ((qt * S::kQ) >> 4), k = k0 + ((i % S::kStages * S::kStage) >> 4);
    if (tc::elect()) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        tc::mma_ss(tmem + kColS + s * 128, q + (((ks >> 2) * S::kPanelQ + (ks & 3) * 32) >> 4),
                   k + (((ks >> 2) * S::kPanel + (ks & 3) * 32) >> 4), kIdS, ks > 0);
      tc::commit(&c.s_full[s]);
    }
    __syncwarp();
  };
  // sums of stream s: both terms of its weights times item i, 32 positions after the
  // other as the weights come
  auto values = [&](int s, int i, bool first, bool last) {
    const uint64_t v = v0 + ((i % S::kStages * S::kStage) >> 4);
    const int phase = ps[s]++;
#pragma unroll
    for (int j = 0; j < S::kN / 32; ++j) {
      const int k = chunk_at<S::kN>(j);
      if (!wait(&c.p_full[s][k], phase)) return false;
      tc::fence_after();
      if (tc::elect()) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            tc::mma_ts(tmem + kColO + s * D, tmem + kColS + s * 128 + k * 32 + t * 16 + h * 8,
                       v + (((2 * k + h) * 2048) >> 4), kIdO, !first || j > 0 || h > 0 || t > 0);
        if (last && j + 1 == S::kN / 32) tc::commit(&c.o_full[s]);
      }
      __syncwarp();
    }
    return true;
  };
  auto release = [&](int i) {
    if (tc::elect()) tc::commit(&c.empty[i % S::kStages]);
    __syncwarp();
  };
  // (read from one lane, as below: the products take their operands from uniform
  // registers, where the compiler keeps what it knows to be the same in the warp)
  auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  LineSeg s;
  while (same(line_segment<Shape<D>::kRowsU>(x.a, blockIdx.x, run, s))) {
    const int n = same(s.j1 - s.j0);
    const bool pair = same(s.pair);
    if (!wait(&c.q_full[0], segs[0]++)) return false;
    if (pair && !wait(&c.q_full[1], segs[1]++)) return false;
    if (!filled(it)) return false;
    tc::fence_after();
    if (pair || S::NT == 1) {
      scores(0, 0, it);
      if (pair) scores(1, 1, it);
      release(it++);
#pragma unroll 1
      for (int t = 0; t < n; ++t) {             // items: V of tile t, K of the next
        const bool more = t + 1 < n;
        if (!filled(it) || !values(0, it, t == 0, !more)) return false;
        if (more) {
          if (!filled(it + 1)) return false;
          scores(0, 0, it + 1);
        }
        if (pair && !values(1, it, t == 0, !more)) return false;
        release(it++);
        if (more) {
          if (pair) scores(1, 1, it);
          release(it++);
        }
      }
    } else {
      scores(0, 0, it);
      release(it++);
      if (n > 1) {
        if (!filled(it)) return false;
        scores(1, 0, it);
        release(it++);
      }
#pragma unroll 1
      for (int t = 0; t < n; t += 2) {          // a tile of each stream
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (t + k >= n) break;
          if (!filled(it) || !values(k, it, t == 0, t + k + 2 >= n)) return false;
          release(it++);
          if (t + k + 2 < n) {
            if (!filled(it)) return false;
            scores(k, 0, it);
            release(it++);
          }
        }
      }
    }
  }
  return true;
}

// ---- softmax --------------------------------------------------------------------

// Writes the statistics of a part without positions.
template <int D>
__device__ __forceinline__ void empty_part(const PrefixArgs& x, const LineSeg& s, int stream) {
  using S = Shape<D>;
  const int r = threadIdx.x & 127;
  x.ps[s.slot * S::kRowsU + stream * 128 + r] = make_float2(-INFINITY, 0.0f);
}

// Scores of positions without a row (behind the prefix, on a bad page) become -inf.
template <int N>
__device__ __noinline__ void hide(uint32_t sc, const uint32_t (&keep)[N / 32]) {
#pragma unroll 1
  for (int k = 0; k < N / 32; ++k) {
    const uint32_t bits = k == 0 ? keep[0] : k == 1 ? keep[N > 32 ? 1 : 0]
                                 : k == 2 ? keep[N > 64 ? 2 : 0] : keep[N > 96 ? 3 : 0];
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t v[16], t[8];
      tc::ld16(sc + k * 32 + h * 16, v);
      tc::wait_ld(v);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (!(bits >> (h * 16 + e) & 1u)) v[e] = 0xff800000u;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = v[e];
      tc::st8(sc + k * 32 + h * 16, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = v[8 + e];
      tc::st8(sc + k * 32 + h * 16 + 8, t);
    }
  }
  tc::wait_st();
}

template <int D>
__device__ __forceinline__ bool soft_role(const PrefixArgs& x, LineRun run, Ctl& c,
                                          unsigned char* q_all, const Wait& wait, uint32_t tmem,
                                          int stream) {
  using S = Shape<D>;
  const AttnArgs& a = x.a;
  const int r = threadIdx.x & 127, rows_all = a.G * a.q_len;
  const uint32_t lanes = tmem + ((uint32_t)(r >> 5) << 21);
  const uint32_t sc = lanes + kColS + stream * 128, oc = lanes + kColO + stream * D;
  // Q carries the scale's sign, so that the largest score has the largest weight (and a
  // scale of zero is the least normal number, which leaves hidden scores at -inf)
  const float sl2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 0x1p-126f);
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
  int tiles_done = 0, segs = 0, seq = 0;
  bool ok = true;
  auto valid_of = [&](const LineSeg& s) { return s.rows - (s.pair ? stream * 128 : 0); };
  // Where row r of a segment's Q begins (-1: no row; the even and the odd tiles of one
  // row tile share the first stream's).
  auto q_row = [&](const LineSeg& s) {
    int64_t mine = -1;
    if (r < valid_of(s) && (stream == 0 || s.pair)) {
      const uint32_t R = (uint32_t)(s.row0 + stream * 128 + r), b = R / (uint32_t)rows_all;
      const uint32_t k = R - b * (uint32_t)rows_all, tok = k / (uint32_t)a.G;
      mine = ((int64_t)(s.first + (int)b) * a.q_len + tok) * a.q_rs +
             (int64_t)(s.h * a.G + (int)(k - tok * a.G)) * D;
    }
    return mine;
  };
  // Q of the warp's 32 rows, of which lane i knows where row i begins.
  unsigned char* const q_mine = q_all + stream * S::kQ;
  const int lane = r & 31, w = r >> 5;
  auto load_q = [&](int64_t mine) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes, kBatch = D == 64 ? 8 : 16;
#pragma unroll 1
    for (int p0 = 0; p0 < 32 / kPer; p0 += kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int p = 0; p < kBatch; ++p) {
        const int64_t at = __shfl_sync(0xffffffffu, mine, (p0 + p) * kPer + lane / kLanes);
        v[p] = at >= 0 ? ldg16(a.q + at * 2 + lane % kLanes * 16) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int p = 0; p < kBatch; ++p) {
        v[p].x ^= flip, v[p].y ^= flip, v[p].z ^= flip, v[p].w ^= flip;
        const int row = w * 32 + (p0 + p) * kPer + lane / kLanes;
        *reinterpret_cast<uint4*>(q_mine + place<S::kPanelQ>(row, lane % kLanes)) = v[p];
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.q_full[stream]);
  };
  LineSeg s, next;
  bool more = line_segment<Shape<D>::kRowsU>(x.a, blockIdx.x, run, next);
  int64_t q_at = more ? q_row(next) : -1;
  while (more) {
    s = next;
    const int n = s.j1 - s.j0;
    const bool two = S::NT == 2 && !s.pair;
    const int step = two ? 2 : 1, t_first = two ? stream : 0, valid = valid_of(s);
    if (ok && (stream == 0 || s.pair)) load_q(q_at);
    // the next segment's rows of Q come to the L2 meanwhile
    more = line_segment<Shape<D>::kRowsU>(x.a, blockIdx.x, run, next);
    q_at = more ? q_row(next) : -1;
    if (q_at >= 0)
      for (int k = 0; k < D * 2; k += 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + q_at * 2 + k));
    if (!ok || t_first >= n) {              // (given up, or no tile for this stream)
      empty_part<D>(x, s, stream);
      seq += n;
      continue;
    }
    const bool idle = (r & ~31) >= valid;    // no row of this warp's: nobody reads its sums
    float m = -INFINITY, l = 0.0f;          // (m: what the weights are relative to)
#pragma unroll 1
    for (int t = t_first; t < n; t += step) {
      if (!wait(&c.s_full[stream], tiles_done++)) {
        ok = false;
        break;
      }
      tc::fence_after();
      if (idle) {
        if ((r & 31) == 0)
          for (int k = 0; k < S::kN / 32; ++k) mbar_arrive(&c.p_full[stream][k]);
        continue;
      }
      uint32_t keep[S::kN / 32];
      bool all = true;
#pragma unroll
      for (int k = 0; k < S::kN / 32; ++k) {
        const uint32_t* w = c.mask[(seq + t) % kMasks];
        keep[k] = S::kN == 128 ? w[k] : w[2 * k] | w[2 * k + 1] << 16;
        all = all && keep[k] == 0xffffffffu;
      }
      if (!all) hide<S::kN>(sc, keep);
      // ---- the largest score
      uint32_t v[2][32];                  // scores; of the last two chunks behind this pass
      float mx = -INFINITY;
#pragma unroll 1
      for (int k = 0; k < S::kN / 32; k += 2) {
        tc::ld32(sc + k * 32, v[0]);
        tc::ld32(sc + k * 32 + 32, v[1]);
        tc::wait_ld(v[0]);
        tc::wait_ld(v[1]);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          mx = fmaxf(mx, fmaxf(__uint_as_float(v[0][e]), __uint_as_float(v[1][e])));
      }
      const float top = mx * sl2;
      const bool rises = top > m + kSlack || (m == -INFINITY && top > m);
      if (__any_sync(0xffffffffu, rises)) {
        const float mn = rises ? top : m;
        const float corr = rises ? tc::ex2(m - mn) : 1.0f;
        m = mn;
        l *= corr;
        if (t != t_first) {
          // (the product before this tile's scores has ended with them)
#pragma unroll 1
          for (int k = 0; k < D; k += 16) {
            uint32_t v[16], h[8];
            tc::ld16(oc + k, v);
            tc::wait_ld(v);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * corr);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = v[e];
            tc::st8(oc + k, h);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = v[8 + e];
            tc::st8(oc + k + 8, h);
          }
        }
      }
      const float base = m == -INFINITY ? 0.0f : -m;
      // ---- weights, in place of the scores: of 32 positions first terms, then second
      float sum = 0.0f, sum1 = 0.0f;
#pragma unroll 1
      for (int k0 = S::kN / 32 - 2; k0 >= 0; k0 -= 2) {
        // (rolled: with all of a tile unrolled the roles' code was fetched more slowly
        // than it ran)
        if (k0 + 2 < S::kN / 32) {
          tc::ld32(sc + k0 * 32 + 32, v[1]);
          tc::ld32(sc + k0 * 32, v[0]);
          tc::wait_ld(v[1]);
          tc::wait_ld(v[0]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int k = k0 + 1 - j;
          uint32_t(&now)[32] = v[1 - j];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const uint32_t* w = now + h * 16 + e;
              float p0, p1;
              fma_x2(p0, p1, __uint_as_float(w[0]), __uint_as_float(w[1]), sl2, sl2, base, base);
              p0 = tc::ex2(p0);
              p1 = tc::ex2(p1);
              fma_x2(sum, sum1, p0, p1, 1.0f, 1.0f, sum, sum1);
              // The first term is cut a little below the weight, so that the second is above
              // zero: terms of zero times an infinite value would make NaN.
              float c0, c1;
              mul_x2(c0, c1, p0, p1, 0.99609375f, 0.99609375f);
              const uint32_t first = __byte_perm(__float_as_uint(c0), __float_as_uint(c1), 0x7632);
              float l0, l1;
              fma_x2(l0, l1, __uint_as_float(first << 16), __uint_as_float(first & 0xffff0000u),
                     -1.0f, -1.0f, p0, p1);
              hi[e / 2] = first;
              lo[e / 2] = pack_bf16x2(l0, l1);
            }
            tc::st8(sc + k * 32 + h * 8, hi);
            tc::st8(sc + k * 32 + 16 + h * 8, lo);
          }
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if ((r & 31) == 0) mbar_arrive(&c.p_full[stream][k]);
        }
      }
      l += sum + sum1;
    }
    if (ok && !wait(&c.o_full[stream], segs++)) ok = false;
    seq += n;
    if (!ok) {
      empty_part<D>(x, s, stream);
      continue;
    }
    tc::fence_after();
    // Sums go out by whole lines, 32 columns at a time, through the place of the warp's
    // rows of Q (every product with this Q has ended with the sums): a row a thread
    // writes 32 lines an instruction, which took 4 us.
    const int64_t row0 = s.slot * S::kRowsU + stream * 128 + w * 32;
    const int rows = min(max(valid - w * 32, 0), 32);
#pragma unroll 1
    for (int k = 0; k < (idle ? 0 : D); k += 32) {
      uint32_t v[32];
      tc::ld32(oc + k, v);
      tc::wait_ld(v);
      unsigned char* const at = q_mine + (k / 32 % (D / 64)) * S::kPanelQ + w * 32 * 128;
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *reinterpret_cast<uint4*>(at + lane * 128 + ((e ^ (lane & 7)) << 4)) =
            make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int rr = e * 4 + (lane >> 3), u = lane & 7;
        const uint4 o = *reinterpret_cast<const uint4*>(at + rr * 128 + ((u ^ (rr & 7)) << 4));
        if (rr < rows)
          *reinterpret_cast<uint4*>(x.po + (row0 + rr) * D + k + u * 4) = o;
      }
    }
    __syncwarp();
    tc::fence_before();           // (before this stream's next sums begin)
    x.ps[row0 + lane] = make_float2(m * 0.6931471805599453f, l);
  }
  return ok;
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 1) attn_prefix_kernel(const PrefixArgs x) {
  using S = Shape<D, Q8>;
  extern __shared__ __align__(1024) unsigned char shared_dyn[];
  unsigned char* const base = shared_dyn + ((1024u - (smem_addr(shared_dyn) & 1023u)) & 1023u);
  unsigned char* const ring = base + S::NT * S::kQ;
  unsigned char* const raw = ring + S::kStages * S::kStage;
  Ctl& c = *reinterpret_cast<Ctl*>(raw + S::kRaw * S::kStage / 2);
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  LineRun run;
  if (!split<D>(x, c.scan, run)) return;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&c.full[i], kCopyWarps * 32);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.q_full[i], kSoftWarps);
      mbar_init(&c.s_full[i], 1);
      for (int k = 0; k < 4; ++k) mbar_init(&c.p_full[i][k], kSoftWarps);
      mbar_init(&c.o_full[i], 1);
    }
    mbar_init(&c.fin, 1);
    c.dead = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&c.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
  const Wait wait{&c.dead, x.a.dev_err};
  if (warp < kCopyWarp0) {
    const int stream = warp / kSoftWarps;
    if (stream < S::NT) soft_role<D>(x, run, c, base, wait, tmem, stream);
  } else if (warp < kMmaWarp) {
    copy_role<D, Q8>(x, run, c, ring, raw, wait);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    mma_role<D, Q8>(x, run, c, smem_addr(base), smem_addr(ring), wait, tmem);
    // every product that was issued ends before tensor memory is given back
    if (tc::elect()) tc::commit(&c.fin);
    __syncwarp();
    long long t0 = clock64();
    while (!__any_sync(0xffffffffu, mbar_try(&c.fin, 0)))
      if (__any_sync(0xffffffffu, clock64() - t0 > kWaitClocks)) break;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ---- join -----------------------------------------------------------------------

// A row's parts: of its group's prefix, then of its own positions. W warps take a row, each
// every W-th part.
template <int D, int W>
__global__ void __launch_bounds__(256) attn_shared_join_kernel(const PrefixArgs x, const int n) {
  using S = Shape<D>;
  constexpr int kPairs = D / 64, kBatch = D == 256 ? 4 : 8, kRowsB = 8 / W;
  const AttnArgs& a = x.a;
  __shared__ float sums[W > 1 ? 8 : 1][W > 1 ? D + 2 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % W;
  const int64_t at = (int64_t)blockIdx.x * kRowsB + warp / W;   // request, kv head, row of it
  const int rows_all = a.G * a.q_len;
  // (the warps of a row all go on or all leave)
  if (at >= n) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int b = (int)(at / (a.Hkv * rows_all)), k = (int)(at % (a.Hkv * rows_all));
  const int h = k / rows_all, rr = k % rows_all;
  // what the call's arguments tell, before the kernels whose results are joined are done
  const int unit = h / a.hw * a.rblocks + rr / a.rows;
  const int64_t bu = (int64_t)b * a.units + unit;
  const int g = attn_start(a, b) > 0 ? attn_group(a, b) : -1;
  AttnGroup s = {};
  if (g >= 0) s = attn_group_of<true>(a, g);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 c = *reinterpret_cast<const int2*>(a.meta + bu * 2);
  Rec rec = {}, all = {};
  if (g >= 0) rec = x.rec[g], all = x.rec[a.groups];
  // own positions
  if (!attn_joins(c.x, c.y, a.grid)) return;
  const int64_t one = (int64_t)a.hw * a.rows * (D + 2);
  const float* const own =
      a.part + (bu + c.x) * one + (int64_t)(h % a.hw * a.rows + rr % a.rows) * (D + 2);
  const int owns = c.y - c.x + 1;
  // the prefix
  int shared = 0;
  int64_t slot = 0;
  bool two = false;
  if (g >= 0) {
    if (rec.unit < 0) return;                     // (groups that overlap: reported)
    const int64_t R = (int64_t)(b - s.first) * rows_all + rr, mt = R / S::kRowsU;
    const int64_t u = mt * a.Hkv + h, line = rec.line + s.place_of(u);
    const int p0 = attn_block_of(line, all.line, all.unit);
    const int p1 =
        attn_block_of(line + (int64_t)(s.tiles - 1) * s.tile_places(u), all.line, all.unit);
    two = S::NT == 2 && s.rows - mt * S::kRowsU <= 128;
    shared = (p1 - p0 + 1) * (two ? 2 : 1);
    slot = (rec.unit + u + p0) * S::kRowsU + R % S::kRowsU;
  }
  const int parts = shared + owns;
  auto row_of = [&](int i) {          // of the prefix: part i's row
    return two ? slot + (int64_t)(i >> 1) * S::kRowsU + (i & 1) * 128
               : slot + (int64_t)i * S::kRowsU;
  };
  auto stats = [&](int i) {
    if (i >= parts) return make_float2(-INFINITY, 0.0f);
    return i < shared ? x.ps[row_of(i)]
                      : *reinterpret_cast<const float2*>(own + (i - shared) * one + D);
  };
  auto values = [&](int i) { return i < shared ? x.po + row_of(i) * D : own + (i - shared) * one; };
  // the warp's parts: w0, w0 + W, ..
  const int mine = (parts - w0 + W - 1) / W;
  float m = -INFINITY;
  for (int i = lane; i < parts; i += 32) m = fmaxf(m, stats(i).x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float l = 0.0f, acc[kPairs][2] = {};
  for (int i0 = 0; i0 < mine; i0 += 32) {
    const float2 ml = stats(i0 + lane < mine ? (i0 + lane) * W + w0 : parts);
    const float f = ml.x == -INFINITY ? 0.0f : expf(ml.x - m);
    // (a row of NaN scores has a sum without a maximum)
    l += ml.x == -INFINITY ? (ml.y != ml.y ? ml.y : 0.0f) : f * ml.y;
    const int end = min(32, mine - i0);
    for (int k0 = 0; k0 < end; k0 += kBatch) {
      float2 v[kBatch][kPairs];
      float wk[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        wk[q] = __shfl_sync(0xffffffffu, f, (k0 + q) & 31);
        const bool in = k0 + q < end && wk[q] != 0.0f;      // (empty parts are not written)
        const float* p = in ? values((i0 + k0 + q) * W + w0) : nullptr;
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
          v[q][j] = in ? *reinterpret_cast<const float2*>(p + j * 64 + lane * 2)
                       : make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          acc[j][0] = fmaf(wk[q], v[q][j].x, acc[j][0]);
          acc[j][1] = fmaf(wk[q], v[q][j].y, acc[j][1]);
        }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if constexpr (W > 1) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      *reinterpret_cast<float2*>(&sums[warp][j * 64 + lane * 2]) =
          make_float2(acc[j][0], acc[j][1]);
    if (lane == 0) sums[warp][D] = l;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "n"(W * 32) : "memory");   // the row's
    if (w0 != 0) return;
#pragma unroll
    for (int k = 1; k < W; ++k) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        acc[j][0] += sums[warp + k][j * 64 + lane * 2];
        acc[j][1] += sums[warp + k][j * 64 + lane * 2 + 1];
      }
      l += sums[warp + k][D];
    }
  }
  const int64_t orow = (int64_t)b * a.q_len + rr / a.G;
  const int hq = h * a.G + rr % a.G;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  char* const o = a.out + (orow * a.out_rs + (int64_t)hq * D + lane * 2) * 2;
#pragma unroll
  for (int j = 0; j < kPairs; ++j)
    *reinterpret_cast<uint32_t*>(o + j * 128) = pack_bf16x2(acc[j][0] * inv, acc[j][1] * inv);
  if (a.lse && lane == 0) a.lse[orow * a.Hq + hq] = l != 0.0f ? m + logf(l) : -INFINITY;
}

// ---- host side ------------------------------------------------------------------

// Places in the workspace.
struct SharedPlan {
  AttnPlan own;
  int64_t max_units, part, rec, po, ps, bytes;    // offsets in bytes
};
SharedPlan shared_plan(bool q8, int sms, int64_t B, int64_t groups, int q_len, int G, int Hkv,
                       int D) {
  SharedPlan p;
  p.own = attn_plan(CCONV_DTYPE_BF16, q8, sms, B, q_len, G, Hkv, D);
  auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  const int rows = D == 256 ? 128 : 256;
  p.max_units = groups > 0 ? (B * G * q_len / rows + groups) * Hkv : 0;
  const int64_t slots = groups > 0 ? p.max_units + sms : 0;
  p.part = up(p.own.meta_bytes);
  p.rec = up(p.part + (B * p.own.units + p.own.grid) * p.own.hw * p.own.rows * (D + 2) * 4);
  p.po = up(p.rec + (groups + 1) * (int64_t)sizeof(Rec));
  p.ps = up(p.po + slots * rows * D * 4);
  p.bytes = p.ps + slots * rows * (int64_t)sizeof(float2);
  return p;
}

int check_shared(int32_t num_seqs, int32_t num_groups, int32_t n_spec, int32_t Hq, int32_t Hkv,
                 int32_t D) {
  const int rc = attn_check_sizes(num_seqs, n_spec, Hq, Hkv, D);
  if (rc != CCONV_OK) return rc;
  // (slots of the prefixes' parts, and rows, are counted in 32 bits)
  if (num_groups < 0 || num_groups > num_seqs || (int64_t)num_groups * Hkv > INT32_MAX / 2 ||
      (int64_t)num_seqs * Hq * (1 + n_spec) > INT32_MAX - 1024)
    return CCONV_ERR_INVALID;
  return CCONV_OK;
}

template <int D, bool Q8>
cudaError_t launch_prefix(const PrefixArgs& x, cudaStream_t st) {
  using S = Shape<D, Q8>;
  constexpr int smem = 1024 + S::NT * S::kQ + S::kStages * S::kStage + S::kRaw * S::kStage / 2 +
                       (int)sizeof(Ctl);
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  static std::atomic<uint64_t> full;
  const cudaError_t e =
      mix_full_smem(reinterpret_cast<const void*>(attn_prefix_kernel<D, Q8>), full);
  if (e != cudaSuccess) return e;
  attn_prefix_kernel<D, Q8><<<x.grid, kThreads, smem, st>>>(x);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_shared_join(const PrefixArgs& x, cudaStream_t st) {
  const int n = x.a.B * x.a.Hq * x.a.q_len;
  // a warp a row where that fills the GPU, else a block's eight
  return n >= 2048
             ? attn_launch_beside(true, attn_shared_join_kernel<D, 1>, x, n, (n + 7) / 8, 256, 0, st)
             : attn_launch_beside(true, attn_shared_join_kernel<D, 8>, x, n, n, 256, 0, st);
}

// What both entry points check and do; a's cache is set.
int decode_shared(AttnArgs& a, int D, bool q8, const void* q, int64_t q_row_stride,
                  const int32_t* block_table, int64_t block_table_row_stride, int32_t table_width,
                  const int32_t* seq_lens, int32_t num_seqs, const int32_t* cu_groups,
                  const int32_t* prefix_lens, int32_t num_groups, int32_t n_spec,
                  int32_t num_q_heads, float scale, int32_t dtype, void* out,
                  int64_t out_row_stride, float* lse, void* workspace, int64_t workspace_bytes,
                  int32_t* dev_err, cconv_stream_t stream) {
  if (dtype != CCONV_DTYPE_BF16) return CCONV_ERR_UNSUPPORTED;
  const int rc = check_shared(num_seqs, num_groups, n_spec, num_q_heads, a.Hkv, D);
  if (rc != CCONV_OK) return rc;
  if (num_seqs == 0) return CCONV_OK;
  if (!attn_rows_ok(a, D, dtype, q, q_row_stride, out, out_row_stride, num_q_heads, block_table,
                    block_table_row_stride, table_width, seq_lens) ||
      (num_groups > 0 && (!cu_groups || !prefix_lens)))
    return CCONV_ERR_INVALID;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  const SharedPlan p =
      shared_plan(q8, sms, num_seqs, num_groups, 1 + n_spec, num_q_heads / a.Hkv, a.Hkv, D);
  if (!workspace || !mix_aligned16(workspace) || workspace_bytes < p.bytes)
    return CCONV_ERR_INVALID;
  attn_fill(a, p.own, D, q8 ? 1 : 2, q, q_row_stride, block_table, block_table_row_stride,
            table_width, seq_lens, num_seqs, n_spec, num_q_heads, scale, out, out_row_stride, lse,
            dev_err);
  char* const ws = static_cast<char*>(workspace);
  a.meta = reinterpret_cast<int32_t*>(ws);
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.cu_groups = cu_groups;
  a.prefix_lens = prefix_lens;
  a.groups = num_groups;
  a.unit_rows = D == 256 ? 128 : 256;
  a.prefix_tile = D == 256 ? 64 : 128;
  a.own_tile = (q8 ? 128 : 64) / a.hw;
  a.sms = sms;
  // Measured for heads of 128: a tile of two row tiles 2.5 us, of one 1.6; from 8 bits,
  // whose conversion bounds it, 2.8 either way; a start 8 to 10 us. A tile of the rest of up
  // to 8 rows takes an SM 0.9 us, about as many as its share of the memory's bandwidth
  // allows. (One of 16 rows over 8 bits takes 1.3 to 1.7, but mixed calls are no faster for
  // it: seven groups with 4 tokens 89 us, with 20 here 109, with 24 102, 64 requests mostly
  // behind their prefix 76, 87 and 98. With 32 rows, and heads of 64 and 256, they would be:
  // 200 us with 15, 147 with 32 for heads of 256.)
  a.start_places = q8 ? 3 : 8;
  a.pair_places = q8 ? 1 : 2;
  a.place_cost = (q8 ? 44 : 22) * (D == 64 ? 5 : 8) / 8;
  a.tile_cost = (q8 && a.rows == 8 ? 13 : 15) * D / 128;
  PrefixArgs x;
  x.a = a;
  x.rec = reinterpret_cast<Rec*>(ws + p.rec);
  x.po = reinterpret_cast<float*>(ws + p.po);
  x.ps = reinterpret_cast<float2*>(ws + p.ps);
  x.max_units = p.max_units;
  x.grid = sms;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  if (num_groups > 0)
    err = q8 ? (D == 64    ? launch_prefix<64, true>(x, st)
                : D == 128 ? launch_prefix<128, true>(x, st)
                           : launch_prefix<256, true>(x, st))
             : (D == 64    ? launch_prefix<64, false>(x, st)
                : D == 128 ? launch_prefix<128, false>(x, st)
                           : launch_prefix<256, false>(x, st));
  if (err != cudaSuccess) return CCONV_ERR_LAUNCH;
  err = q8 ? attn_launch_mma_q8(a, D, p.own.grid, true, st)
           : attn_launch_mma(a, D, p.own.grid, true, st);
  if (err != cudaSuccess) return CCONV_ERR_LAUNCH;
  err = D == 64    ? launch_shared_join<64>(x, st)
        : D == 128 ? launch_shared_join<128>(x, st)
                   : launch_shared_join<256>(x, st);
  return err == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}

}  // namespace
}  // namespace cconv

using namespace cconv;

extern "C" int64_t attn_decode_shared_workspace_bytes(int32_t num_seqs, int32_t num_groups,
                                                      int32_t n_spec, int32_t num_q_heads,
                                                      int32_t num_kv_heads, int32_t head_dim) {
  const int rc =
      check_shared(num_seqs, num_groups, n_spec, num_q_heads, num_kv_heads, head_dim);
  if (rc != CCONV_OK) return rc;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  int64_t most = 0;
  for (const bool q8 : {false, true})
    most = std::max(most, shared_plan(q8, sms, num_seqs, num_groups, 1 + n_spec,
                                      num_q_heads / num_kv_heads, num_kv_heads, head_dim).bytes);
  return most;
}

extern "C" int attn_decode_shared(const void* q, int64_t q_row_stride, kv_cache_t cache,
                                  const int32_t* block_table, int64_t block_table_row_stride,
                                  int32_t table_width, const int32_t* seq_lens, int32_t num_seqs,
                                  const int32_t* cu_groups, const int32_t* prefix_lens,
                                  int32_t num_groups, int32_t n_spec, int32_t num_q_heads,
                                  float scale, int32_t dtype, void* out, int64_t out_row_stride,
                                  float* lse, void* workspace, int64_t workspace_bytes,
                                  int32_t* dev_err, cconv_stream_t stream) {
  if (mix_dtype_bytes(dtype) == 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache(cache, dtype);
  if (rc != CCONV_OK) return rc;
  AttnArgs a = attn_cache_args(cache);
  return decode_shared(a, cache.head_dim, false, q, q_row_stride, block_table,
                       block_table_row_stride, table_width, seq_lens, num_seqs, cu_groups,
                       prefix_lens, num_groups, n_spec, num_q_heads, scale, dtype, out,
                       out_row_stride, lse, workspace, workspace_bytes, dev_err, stream);
}

extern "C" int attn_decode_shared_q8(const void* q, int64_t q_row_stride, kv_cache_q8_t cache,
                                     const int32_t* block_table, int64_t block_table_row_stride,
                                     int32_t table_width, const int32_t* seq_lens,
                                     int32_t num_seqs, const int32_t* cu_groups,
                                     const int32_t* prefix_lens, int32_t num_groups,
                                     int32_t n_spec, int32_t num_q_heads, float scale,
                                     int32_t dtype, void* out, int64_t out_row_stride, float* lse,
                                     void* workspace, int64_t workspace_bytes, int32_t* dev_err,
                                     cconv_stream_t stream) {
  if (mix_dtype_bytes(dtype) == 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache_q8(cache);
  if (rc != CCONV_OK) return rc;
  AttnArgs a = attn_cache_args(cache);
  a.ksc = cache.k_scale;
  a.vsc = cache.v_scale;
  a.c_page = cache.c_page, a.c_tok = cache.c_token, a.c_head = cache.c_head;
  return decode_shared(a, cache.head_dim, true, q, q_row_stride, block_table,
                       block_table_row_stride, table_width, seq_lens, num_seqs, cu_groups,
                       prefix_lens, num_groups, n_spec, num_q_heads, scale, dtype, out,
                       out_row_stride, lse, workspace, workspace_bytes, dev_err, stream);
}
