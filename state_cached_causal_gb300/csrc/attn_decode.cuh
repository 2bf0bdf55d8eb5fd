// Paged attention of new tokens: work split, partial results and arguments
// shared by the kernels of attn_decode (attn_decode.cu, attn_mma.cu).
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
};

// Blocks of the bf16 kernel that an SM holds at once, by their registers and
// shared memory (50 to 218 KB).
inline int attn_mma_blocks(int D, int rows) {
  return D * rows >= 4096 ? 1 : D * rows >= 2048 ? 2 : 3;
}

// Tiles of request b: at least one (an empty request still writes its rows).
// len < 0 marks a request that is skipped.
__device__ __forceinline__ int attn_len(const AttnArgs& a, int b) {
  const int n = a.seq_lens[b];
  return (n < 0 || n > (int64_t)a.table_width * a.page_size) ? -1 : n;
}
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, int b, int tile) {
  const int n = attn_len(a, b);
  return n <= 0 ? 1 : (n + tile - 1) / tile;
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
template <int THREADS>
__device__ __forceinline__ bool attn_split(const AttnArgs& a, int tile, int64_t (&sm)[THREADS + 4],
                                           AttnRun& r) {
  const int tid = threadIdx.x;
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += attn_tiles(a, b, tile);
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
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < (tid >> 5)) base += sm[w];
    sum += sm[w];
  }
  incl += base;
  const int64_t units = a.units;
  r.total = sum * units;
  // no run is empty: where there are fewer tiles than blocks, the blocks past
  // the tiles' number have none
  r.grid = min((int64_t)gridDim.x, r.total);
  r.p = blockIdx.x < r.grid ? blockIdx.x * r.total / r.grid : r.total;
  r.end = blockIdx.x < r.grid ? (blockIdx.x + 1) * r.total / r.grid : r.total;
  __syncthreads();
  // the thread whose requests hold p finds which one
  if (mine > 0 && r.p >= (incl - mine) * units && r.p < incl * units) {
    int64_t before = incl - mine;
    int b = b0;
    for (;; ++b) {
      const int n = attn_tiles(a, b, tile);
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
__device__ __forceinline__ int attn_block_of(int64_t tile, const AttnRun& r) {
  return (int)(((tile + 1) * r.grid - 1) / r.total);
}

// One segment: unit `unit` of request b, tiles [j0, j1) of `tiles`.
struct AttnSeg {
  int b, unit, len, tiles, j0, j1;
  bool whole;
  int64_t line;         // place of the unit's tile 0 on the line
};
__device__ __forceinline__ AttnSeg attn_segment(const AttnArgs& a, int tile, const AttnRun& r) {
  AttnSeg s;
  const int64_t units = a.units;
  s.b = r.b;
  s.len = attn_len(a, r.b);
  s.tiles = attn_tiles(a, r.b, tile);
  const int64_t rel = r.p - r.before * units;
  s.unit = (int)(rel / s.tiles);
  s.j0 = (int)(rel % s.tiles);
  s.j1 = (int)min((int64_t)s.tiles, s.j0 + (r.end - r.p));
  s.line = r.before * units + (int64_t)s.unit * s.tiles;
  s.whole = s.j0 == 0 && s.j1 == s.tiles;
  return s;
}
__device__ __forceinline__ void attn_advance(const AttnArgs& a, const AttnSeg& s, AttnRun& r) {
  r.p += s.j1 - s.j0;
  if (s.j1 == s.tiles && s.unit == a.units - 1) {
    r.before += s.tiles;
    ++r.b;
  }
}

// Where the block's part of a cut segment goes (see above), and the note for
// the join, written by the block that holds the unit's first tile.
__device__ __forceinline__ float* attn_part(const AttnArgs& a, const AttnSeg& s, int D) {
  return a.part + ((int64_t)blockIdx.x * 2 + (s.j0 == 0 ? 1 : 0)) * a.hw * a.rows * (D + 2);
}
__device__ __forceinline__ void attn_note(const AttnArgs& a, const AttnSeg& s, const AttnRun& r) {
  if (s.j0 != 0) return;
  int32_t* m = a.meta + ((int64_t)s.b * a.units + s.unit) * 2;
  const bool cut = !s.whole && s.len >= 0;
  m[0] = cut ? attn_block_of(s.line, r) : -1;
  m[1] = cut ? attn_block_of(s.line + s.tiles - 1, r) : -1;
}

// Whether blocks c0 to c1 hold the parts of a cut unit: not if it was whole or
// skipped (-1), nor if no note of it was written, since a block was given up.
__host__ __device__ inline bool attn_joins(int32_t c0, int32_t c1, int32_t grid) {
  return c0 >= 0 && c0 <= c1 && c1 < grid;
}

// bf16 kernel (attn_mma.cu)
cudaError_t attn_launch_mma(const AttnArgs& a, int D, int grid, cudaStream_t st);

}  // namespace cconv
