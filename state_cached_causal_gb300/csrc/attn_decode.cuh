// Paged attention of new tokens: work split, partial results and arguments
// shared by the kernels of attn_decode (attn_decode.cu, attn_mma.cu), of attn_decode_q8
// (attn_mma_q8.cu) and of the shared form (attn_shared.cu).
//
// A unit is a request with a group of `hw` kv heads (and a block of `rows` query
// rows of each); its cached tokens are cut into tiles of `tile` positions. All
// tiles of the call form one line -- request by request, unit by unit, tile by
// tile -- which the grid's blocks cut into equal runs, whatever the requests'
// lengths: the work is K and V bytes, and equal runs of them end together. A
// block walks its run as segments, one per unit. A segment that holds all the
// tiles of its unit is written out at once; of one that is cut the block stores
// the running maximum, sum and weighted values, at most two a block (its first
// segment if that began in another block, its last if that goes on in the
// next), and attn_join_kernel joins them.
#pragma once

#include "mixer.cuh"

namespace cconv {

struct AttnArgs {
  const char* q;
  int64_t q_rs;
  const char *kc, *vc;
  int64_t s_page, s_tok, s_head;
  int32_t num_pages, page_size;
  int32_t page_shift;   // log2(page_size), -1 if it is no power of two
  const int32_t* table;
  int64_t table_rs;
  int32_t table_width;
  const int32_t* seq_lens;
  int32_t B, q_len, Hq, Hkv, G;
  float scale;
  char* out;
  int64_t out_rs;
  float* lse;
  int32_t* meta;     // [B * units][2]: first and last block of a cut unit, or -1
  float* part;       // [grid][2][hw * rows][D + 2]: weighted values, maximum, sum
  int32_t hw;        // kv heads of a unit
  int32_t group_shift;  // log2 of the positions that one copy brings (attn_mma.cu)
  int32_t rblocks;   // row blocks of a head (rows of G * q_len taken separately)
  int32_t rows;      // rows of a block
  int32_t units;     // of a request: Hkv / hw * rblocks
  int32_t grid;      // blocks of the split kernel
  int32_t* dev_err;
  const uint8_t *ksc, *vsc;   // scales of a cache in 8 bits
  int64_t c_page, c_tok, c_head;
  // of attn_decode_shared (attn_shared.cu): groups, rows of a unit and positions of a
  // tile of a prefix, positions of a tile of the rest; places of a segment's start, of a
  // tile of two row tiles; SMs, and what a place of the prefixes' line and a tile of the
  // rest cost an SM, in sixteenths of a microsecond
  const int32_t *cu_groups, *prefix_lens;
  int32_t groups, unit_rows, prefix_tile, own_tile, start_places, pair_places;
  int32_t sms, place_cost, tile_cost;
};

// Blocks of the bf16 kernels that an SM holds at once, by their registers and
// shared memory (50 to 218 KB; with heads of 256 two places of the ring are over half of
// it already). A block of the kernel over a cache in 8 bits has a warp more.
__host__ __device__ constexpr int attn_mma_blocks(int D, int rows, bool q8) {
  return D == 256 || D * rows >= 4096 ? 1 : D * rows >= 2048 || q8 ? 2 : 3;
}

// Length of request b; -1 for one that is skipped.
__host__ __device__ __forceinline__ int attn_len(const AttnArgs& a, int b) {
  const int n = a.seq_lens[b];
  return (n < 0 || n > (int64_t)a.table_width * a.page_size) ? -1 : n;
}

// attn_decode_shared: the group that request b is of (-1: none), and the prefix of
// group g (0 where its bounds or its prefix are out of range).
__host__ __device__ __forceinline__ int attn_group(const AttnArgs& a, int b) {
  int lo = 0, hi = a.groups;              // the last group that begins at b or before
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_groups[mid] <= b)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int g = lo - 1;
  return g >= 0 && a.cu_groups[g + 1] > b ? g : -1;
}
__host__ __device__ __forceinline__ bool attn_group_ok(const AttnArgs& a, int first, int end,
                                                       int prefix) {
  return first >= 0 && first <= end && end <= a.B && prefix >= 0 &&
         prefix <= (int64_t)a.table_width * a.page_size;
}
__host__ __device__ __forceinline__ int attn_prefix(const AttnArgs& a, int g) {
  const int first = a.cu_groups[g], end = a.cu_groups[g + 1], p = a.prefix_lens[g];
  return attn_group_ok(a, first, end, p) ? p : 0;
}
// The positions of request b that the shared kernel takes (the rest begins there):
// its group's prefix if all its rows see the whole of that, else none.
__host__ __device__ __forceinline__ int attn_start(const AttnArgs& a, int b) {
  const int g = attn_group(a, b);
  if (g < 0) return 0;
  const int p = attn_prefix(a, g);
  return attn_len(a, b) - (a.q_len - 1) >= p ? p : 0;
}
// The positions of request b that lie behind that.
__host__ __device__ __forceinline__ int attn_behind(const AttnArgs& a, int b) {
  const int n = attn_len(a, b);
  return n > 0 ? n - attn_start(a, b) : 0;
}

// The position that tile 0 of request b begins at, and its tiles: at least one (an
// empty request still writes its rows). A copy of several positions begins at a
// multiple of them.
template <bool SHARED>
__device__ __forceinline__ int attn_base(const AttnArgs& a, int start) {
  return SHARED ? start >> a.group_shift << a.group_shift : 0;
}
template <bool SHARED>
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, int b, int tile) {
  int n = attn_len(a, b);
  if (SHARED && n > 0) n -= attn_base<SHARED>(a, attn_start(a, b));
  return n <= 0 ? 1 : (n + tile - 1) / tile;
}

// ---- prefixes on their line, and the SMs of the two kernels of attn_decode_shared ----

// Places of a unit (attn_shared.cu) on the line: start_places before its first tile (a
// segment's start -- Q, the first copies -- takes a block as long), then pair_places (1
// or 2) a tile where two row tiles take it, else one. A block takes the tiles whose first
// place is in its run, and no run is shorter than two.
struct AttnGroup {
  int first, prefix, tiles;
  int lead;                   // the first request that sees the prefix whole (-1: none)
  int64_t rows, units;        // rows of a kv head; units 0 without a prefix or a lead
  int64_t full;               // units of two whole row tiles, which come first
  int per_full, per, wide;    // places of one of these, of another, and of a tile of that
  int start, pair;

  __host__ __device__ __forceinline__ int64_t places() const {
    return full * per_full + (units - full) * per;
  }
  // the place of a unit's tile 0, and those of a tile
  __host__ __device__ __forceinline__ int64_t place_of(int64_t unit) const {
    return start + (unit < full ? unit * per_full : full * per_full + (unit - full) * per);
  }
  __host__ __device__ __forceinline__ int tile_places(int64_t unit) const {
    return unit < full ? pair : wide;
  }
};
// The first of requests first to end - 1 that sees a prefix whole, -1 if none does. (Four
// lengths at a time: a batch may begin with many that are finished.)
__host__ __device__ __forceinline__ int attn_lead(const AttnArgs& a, int first, int end,
                                                  int prefix) {
  const int least = prefix + a.q_len - 1, most = a.table_width * a.page_size;
#pragma unroll 1
  for (int b = first; b < end; b += 4) {
    int hit = 4;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
      const int n = a.seq_lens[b + k < end ? b + k : b];
      if (n >= least && n <= most) hit = k;
    }
    if (hit < 4) return b + hit;
  }
  return -1;
}
// (LED: it is known that there is a lead, which is not looked for)
template <bool LED = false>
__host__ __device__ __forceinline__ AttnGroup attn_group_of(const AttnArgs& a, int g) {
  AttnGroup r;
  r.first = a.cu_groups[g];
  const int end = a.cu_groups[g + 1], p = a.prefix_lens[g];
  const bool ok = attn_group_ok(a, r.first, end, p), two = a.unit_rows > 128;
  r.prefix = ok ? p : 0;
  r.tiles = (r.prefix + a.prefix_tile - 1) / a.prefix_tile;
  r.lead = ok && r.first < end ? r.first : -1;
  if (!LED && r.tiles > 0 && r.lead >= 0) r.lead = attn_lead(a, r.first, end, r.prefix);
  r.rows = ok ? (int64_t)(end - r.first) * (a.G * a.q_len) : 0;
  const int64_t blocks = (r.rows + a.unit_rows - 1) / a.unit_rows;     // of rows
  r.units = r.tiles > 0 && r.lead >= 0 ? blocks * a.Hkv : 0;
  r.full = two && r.units > 0 ? r.units - a.Hkv : 0;
  r.start = a.start_places;
  r.pair = a.pair_places;
  r.wide = two && r.rows - (blocks - 1) * a.unit_rows > 128 ? r.pair : 1;
  r.per = r.wide * r.tiles + r.start;
  r.per_full = r.pair * r.tiles + r.start;
  return r;
}

// The SMs that take the prefixes, the others taking the rest meanwhile: as the work of
// both is, by what an SM needs for it. `places` of the prefixes, `positions` of all
// requests that lie behind what they see of them; every block of both kernels comes to
// the same number. (Each request counts what it sees: 64 of 4000 positions in a group
// whose prefix is 4096 take 106 us, and took 1149 counted as if they saw it. One after the
// other on all SMs: 256 requests behind a long document 153 us against 146, groups in 8 bits
// 103 to 110 against 86, 64 requests whose own 8192 positions are most of the work 126
// against 116, 96 behind 1024 positions 67 against 57. With at most 5/8 of the SMs for the
// rest those 64 took 157.)
__host__ __device__ __forceinline__ int attn_prefix_sms(const AttnArgs& a, int64_t places,
                                                        int64_t positions) {
  if (places == 0) return 0;
  const int64_t tiles = (max(positions, (int64_t)0) / a.own_tile + a.B / 2) * a.units;
  const int64_t pc = places * a.place_cost, tc = tiles * a.tile_cost;
  const int64_t own = (a.sms * tc + pc + tc - 1) / max(pc + tc, (int64_t)1);
  return a.sms - (int)min(max(own, (int64_t)2), (int64_t)a.sms * 15 / 16);
}

// The block's run [p, end) of the line and the request that p lies in.
struct AttnRun {
  int64_t p, end, total;
  int64_t grid;         // blocks that have a run
  int b;                // request of p
  int64_t before;       // tiles (of one unit) of the requests before b
};

// Splits the line over the grid. Every thread of the block calls it; `sm` is
// shared scratch. Each thread counts a
// run of requests, and a scan over the threads places the block's start.
template <int THREADS, bool SHARED = false>
__device__ __forceinline__ bool attn_split(const AttnArgs& a, int tile, int64_t (&sm)[THREADS + 4],
                                           AttnRun& r) {
  const int tid = threadIdx.x;
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int64_t mine = 0;
  constexpr int kW = THREADS / 32;
  if constexpr (SHARED) {
    int64_t places = 0, positions = 0;
#pragma unroll 1
    for (int g = tid; g < a.groups; g += THREADS) places += attn_group_of(a, g).places();
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      mine += attn_tiles<true>(a, b, tile);
      positions += attn_behind(a, b);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      places += __shfl_xor_sync(0xffffffffu, places, d);
      positions += __shfl_xor_sync(0xffffffffu, positions, d);
    }
    if ((tid & 31) == 0) sm[kW + (tid >> 5)] = places, sm[2 * kW + (tid >> 5)] = positions;
  }
  if constexpr (!SHARED)
    for (int b = b0; b < b1; ++b) mine += attn_tiles<false>(a, b, tile);
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if ((tid & 31) >= d) incl += o;
  }
  if ((tid & 31) == 31) sm[tid >> 5] = incl;
  __syncthreads();
  int64_t base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w < (tid >> 5)) base += sm[w];
    sum += sm[w];
  }
  incl += base;
  const int64_t units = a.units;
  r.total = sum * units;
  int64_t blocks = gridDim.x;
  if constexpr (SHARED) {
    int64_t places = 0, positions = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) places += sm[kW + w], positions += sm[2 * kW + w];
    blocks = blocks / a.sms * (a.sms - attn_prefix_sms(a, places, positions));
  }
  // no run is empty: where there are fewer tiles than blocks, the blocks past
  // the tiles' number have none
  r.grid = min(blocks, r.total);
  r.p = blockIdx.x < r.grid ? blockIdx.x * r.total / r.grid : r.total;
  r.end = blockIdx.x < r.grid ? (blockIdx.x + 1) * r.total / r.grid : r.total;
  __syncthreads();
  // the thread whose requests hold p finds which one
  if (mine > 0 && r.p >= (incl - mine) * units && r.p < incl * units) {
    int64_t before = incl - mine;
    int b = b0;
    for (;; ++b) {
      const int n = attn_tiles<SHARED>(a, b, tile);
      if (r.p < (before + n) * units) break;
      before += n;
    }
    sm[0] = b;
    sm[1] = before;
  }
  __syncthreads();
  r.b = (int)sm[0];
  r.before = sm[1];
  return r.p < r.end;
}

// The block of the grid whose run holds this tile of the line.
__host__ __device__ __forceinline__ int attn_block_of(int64_t tile, int64_t total, int64_t grid) {
  return (int)(((tile + 1) * grid - 1) / total);
}

// One segment: unit `unit` of request b, tiles [j0, j1) of `tiles`; positions from
// `start` on, tile 0 beginning at `base`.
struct AttnSeg {
  int b, unit, len, tiles, j0, j1, start, base;
  bool whole;
  int64_t line;         // place of the unit's tile 0 on the line
};
template <bool SHARED = false>
__device__ __forceinline__ AttnSeg attn_segment(const AttnArgs& a, int tile, const AttnRun& r) {
  AttnSeg s;
  const int64_t units = a.units;
  s.b = r.b;
  s.len = attn_len(a, r.b);
  s.start = SHARED && s.len > 0 ? attn_start(a, r.b) : 0;
  s.base = attn_base<SHARED>(a, s.start);
  s.tiles = s.len - s.base <= 0 ? 1 : (s.len - s.base + tile - 1) / tile;
  const int64_t rel = r.p - r.before * units;
  s.unit = (int)(rel / s.tiles);
  s.j0 = (int)(rel % s.tiles);
  s.j1 = (int)min((int64_t)s.tiles, s.j0 + (r.end - r.p));
  s.line = r.before * units + (int64_t)s.unit * s.tiles;
  s.whole = !SHARED && s.j0 == 0 && s.j1 == s.tiles;
  return s;
}
__device__ __forceinline__ void attn_advance(const AttnArgs& a, const AttnSeg& s, AttnRun& r) {
  r.p += s.j1 - s.j0;
  if (s.j1 == s.tiles && s.unit == a.units - 1) {
    r.before += s.tiles;
    ++r.b;
  }
}

// Where the block's part of a cut segment goes (see above; attn_decode_shared joins
// every segment: from one to the next on the line the unit's number or the block's
// rises, so that their sum is a place of its own), and the note for the join,
// written by the block that holds the unit's first tile.
template <bool SHARED = false>
__device__ __forceinline__ float* attn_part(const AttnArgs& a, const AttnSeg& s, int D) {
  const int64_t place = SHARED ? (int64_t)s.b * a.units + s.unit + blockIdx.x
                               : (int64_t)blockIdx.x * 2 + (s.j0 == 0 ? 1 : 0);
  return a.part + place * a.hw * a.rows * (D + 2);
}
__device__ __forceinline__ void attn_note(const AttnArgs& a, const AttnSeg& s, const AttnRun& r) {
  if (s.j0 != 0) return;
  int32_t* m = a.meta + ((int64_t)s.b * a.units + s.unit) * 2;
  const bool cut = !s.whole && s.len >= 0;
  m[0] = cut ? attn_block_of(s.line, r.total, r.grid) : -1;
  m[1] = cut ? attn_block_of(s.line + s.tiles - 1, r.total, r.grid) : -1;
}

// Whether blocks c0 to c1 hold the parts of a cut unit: not if it was whole or
// skipped (-1), nor if no note of it was written, since a block was given up.
__host__ __device__ inline bool attn_joins(int32_t c0, int32_t c1, int32_t grid) {
  return c0 >= 0 && c0 <= c1 && c1 < grid;
}

// bf16 kernels over a cache in bf16 (attn_mma.cu) and in 8 bits (attn_mma_q8.cu); with
// `shared` they take each request from attn_start on, and all segments are joined.
cudaError_t attn_launch_mma(const AttnArgs& a, int D, int grid, bool shared, cudaStream_t st);
cudaError_t attn_launch_mma_q8(const AttnArgs& a, int D, int grid, bool shared, cudaStream_t st);

// ---- host side ----------------------------------------------------------------

constexpr int kAttnPlainRows = 8;     // query rows of a block of the plain kernel
constexpr int kAttnMaxGrid = 2048;    // blocks of the split kernels

struct AttnPlan {
  int hw, rblocks, rows, units, grid;
  int64_t meta_bytes, bytes;
};
inline AttnPlan attn_plan(int dtype, bool q8, int sms, int64_t B, int q_len, int G, int Hkv,
                          int D) {
  AttnPlan p;
  const int rows = G * q_len;
  p.hw = 1;
  if (dtype == CCONV_DTYPE_F32) {
    p.rows = kAttnPlainRows;
    p.grid = sms * (D == 64 ? 7 : D == 128 ? 5 : 2);   // blocks that an SM holds at once
  } else {
    // row tiles whose sums fit in registers
    p.rows = q8 && rows <= 8 ? 8 : rows <= 16 || D == 256 ? 16 : 32;
    p.hw = Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1;
    p.grid = sms * attn_mma_blocks(D, p.rows, q8);
  }
  p.grid = std::min(p.grid, kAttnMaxGrid);
  p.rblocks = (rows + p.rows - 1) / p.rows;
  p.units = Hkv / p.hw * p.rblocks;
  p.meta_bytes = (B * p.units * 8 + 15) / 16 * 16;
  p.bytes = p.meta_bytes + (int64_t)p.grid * 2 * p.hw * p.rows * (D + 2) * 4;
  return p;
}

inline int attn_check_sizes(int32_t num_seqs, int32_t n_spec, int32_t Hq, int32_t Hkv, int32_t D) {
  if (num_seqs < 0 || n_spec < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0)
    return CCONV_ERR_INVALID;
  if (n_spec > kMaxSpec || (int64_t)(Hq / Hkv) * (1 + n_spec) > 64 ||
      (D != 64 && D != 128 && D != 256))
    return CCONV_ERR_UNSUPPORTED;
  if ((int64_t)num_seqs * Hkv * 128 > INT32_MAX || (int64_t)num_seqs * (1 + n_spec) > INT32_MAX)
    return CCONV_ERR_INVALID;
  return CCONV_OK;
}

template <typename C>
AttnArgs attn_cache_args(const C& cache) {
  AttnArgs a = {};
  a.kc = static_cast<const char*>(cache.k);
  a.vc = static_cast<const char*>(cache.v);
  a.s_page = cache.s_page, a.s_tok = cache.s_token, a.s_head = cache.s_head;
  a.num_pages = cache.num_pages, a.page_size = cache.page_size;
  a.Hkv = cache.num_kv_heads;
  return a;
}

inline bool attn_rows_ok(const AttnArgs& a, int D, int dtype, const void* q, int64_t q_row_stride,
                         const void* out, int64_t out_row_stride, int32_t num_q_heads,
                         const int32_t* block_table, int64_t block_table_row_stride,
                         int32_t table_width, const int32_t* seq_lens) {
  const int V = 16 / mix_dtype_bytes(dtype);
  return mix_rows_ok(q, q_row_stride, (int64_t)num_q_heads * D, V) &&
         mix_rows_ok(out, out_row_stride, (int64_t)num_q_heads * D, V) && seq_lens &&
         table_width >= 0 && (table_width == 0 || block_table) &&
         block_table_row_stride >= table_width &&
         (int64_t)table_width * a.page_size <= INT32_MAX - 1024;
}

// Everything but the cache and the workspace; `bytes` of a cached value of the bf16
// kernels.
inline void attn_fill(AttnArgs& a, const AttnPlan& p, int D, int bytes, const void* q,
                      int64_t q_row_stride, const int32_t* block_table,
                      int64_t block_table_row_stride, int32_t table_width, const int32_t* seq_lens,
                      int32_t num_seqs, int32_t n_spec, int32_t num_q_heads, float scale,
                      void* out, int64_t out_row_stride, float* lse, int32_t* dev_err) {
  a.q = static_cast<const char*>(q);
  a.q_rs = q_row_stride;
  a.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (a.page_size == 1 << s) a.page_shift = s;
  a.table = block_table;
  a.table_rs = block_table_row_stride;
  a.table_width = table_width;
  a.seq_lens = seq_lens;
  a.B = num_seqs;
  a.q_len = 1 + n_spec;
  a.Hq = num_q_heads;
  a.G = num_q_heads / a.Hkv;
  a.scale = scale;
  a.out = static_cast<char*>(out);
  a.out_rs = out_row_stride;
  a.lse = lse;
  a.hw = p.hw;
  // positions that follow one another in memory come together, up to 1 KB or four
  a.group_shift = 0;
  if (a.s_tok == (int64_t)p.hw * D && (p.hw == 1 || a.s_head == D))
    while (a.group_shift < 2 && (p.hw * D * bytes << a.group_shift) < 1024 &&
           a.page_size % (2 << a.group_shift) == 0)
      ++a.group_shift;
  a.rblocks = p.rblocks;
  a.rows = p.rows;
  a.units = p.units;
  a.grid = p.grid;
  a.dev_err = dev_err;
}

// Launches a kernel of the shared form, beside the call's kernel before it if there is one
// (any other that lets its successor start early may still be writing what this reads).
template <typename K, typename A>
cudaError_t attn_launch_beside(bool beside, K kernel, const A& a, int more, int grid, int threads,
                               int smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, more);
}

}  // namespace cconv
