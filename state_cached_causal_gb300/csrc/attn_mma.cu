// attn_decode in bf16: the same split as attn_decode.cuh, with the products on
// the warp-level tensor instruction (m16n8k16).
//
// What bounds it is the cache's bytes: K and V are read once, for all query
// rows of a kv head together, and a row pair of 16 x 128 products per 256 bytes
// is far below any arithmetic limit. tcgen05 would need 64 rows or a transposed
// product to be fed; with 4 to 32 rows the warp-level form fits the rows as they
// are, keeps the softmax in the registers of the warp that made the scores, and
// the tensor pipe is mostly idle either way.
//
// A block of 4 warps keeps a ring of tiles of K and V in shared memory, filled
// by cp.async (16 bytes a request, rows swizzled by 16-byte unit so that
// ldmatrix meets no bank conflict), several tiles ahead. A tile is 64 rows: 64 /
// hw positions of hw kv heads, since the heads of a token lie side by side in
// the usual cache and one head alone would take 256 bytes of every kilobyte
// (3.96 TB/s so, against @HW@ with four heads together). Each warp takes 16
// rows, of one head: scores = Q K^T, running maximum and sum of its own, weights
// to bf16 in registers (the score layout of one product is the weight layout of
// the next), weighted values += P V. No barrier between warps but the ring's;
// warps of one head join their parts once per segment, through shared memory.
//
// Positions of a tile that lie behind the length or on a bad page are filled
// with zeros and masked.
#include "attn_decode.cuh"

#include <math.h>

namespace cconv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;           // rows of a tile (positions x heads); 16 a warp

template <int D>
struct Cfg {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kUnits = D / 8;                       // 16-byte units a row
  static constexpr int kTileBytes = kTile * kRowBytes;       // K or V of a tile
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr int kRing = kStages * 2 * kTileBytes;
};

// Byte of 16-byte unit u of row r: units are permuted within groups of eight.
template <int D>
__device__ __forceinline__ uint32_t at(int r, int u) {
  return (uint32_t)(r * Cfg<D>::kRowBytes + ((u ^ (r & 7)) << 4));
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// MT row tiles of 16. Q stays in registers where it fits beside the sums, else
// in shared memory (swizzled like K).
template <int D, int MT>
__global__ void __launch_bounds__(kThreads) attn_mma_kernel(const AttnArgs a) {
  using C = Cfg<D>;
  constexpr bool kQRegs = MT * D <= 128;
  extern __shared__ __align__(128) unsigned char attn_dyn[];
  __shared__ int64_t scan[kThreads + 4];
  __shared__ __align__(4) unsigned char there[C::kStages][kTile];   // positions that hold a token
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem = smem_addr(attn_dyn);
  // behind the ring: the joins of at most two heads, or the warps' own Q before
  float* const join = reinterpret_cast<float*>(attn_dyn + C::kRing);
  unsigned char* const sq = attn_dyn + C::kRing + warp * (MT * 16 * D * 2);
  AttnRun run;
  const int hw_shift = a.hw == 4 ? 2 : a.hw >> 1, tpos = kTile >> hw_shift;   // positions a tile
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!attn_split<kThreads>(a, tpos, scan, run)) return;
  const int rows_all = a.G * a.q_len;
  const float sl2 = a.scale * 1.4426950408889634f;

  // ---- loads: thread tid copies unit tid % kUnits of rows tid / kUnits + ..
  constexpr int kRowsAtOnce = kThreads / C::kUnits, kCopies = kTile / kRowsAtOnce;
  AttnRun ld = run;               // the load side runs ahead of the compute side
  AttnSeg ls = attn_segment(a, tpos, ld);
  int lj = ls.j0;
  auto load_tile = [&](int stage) {
    if (ld.p < ld.end) {
      const uint32_t kb = smem + stage * 2 * C::kTileBytes, vb = kb + C::kTileBytes;
      const int u = tid % C::kUnits, r0 = tid / C::kUnits;
      const int hkv0 = ls.unit / a.rblocks * a.hw;
      const int32_t* tab = a.table + (int64_t)ls.b * a.table_rs;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        // copies in the order of the cache: position by position, its heads
        const int k = r0 + i * kRowsAtOnce, hl = k & (a.hw - 1), pl = k >> hw_shift;
        const int r = hl * tpos + pl, pos = lj * tpos + pl;
        int page = -1;
        if (pos < ls.len) {
          page = tab[a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size];
          if (page < 0 || page >= a.num_pages) {
            flag_error(a.dev_err, CCONV_DERR_PAGE);
            page = -1;
          }
        }
        const bool in = page >= 0;
        const int tok = a.page_shift >= 0 ? pos & (a.page_size - 1) : pos % a.page_size;
        const int64_t off = in ? ((int64_t)page * a.s_page + (int64_t)tok * a.s_tok +
                                  (int64_t)(hkv0 + hl) * a.s_head + u * 8) * 2
                               : 0;
        if (u == 0) there[stage][r] = in;
        cp_async16(kb + at<D>(r, u), a.kc + off, in);
        cp_async16(vb + at<D>(r, u), a.vc + off, in);
      }
      if (++lj == ls.j1) {
        attn_advance(a, ls, ld);
        if (ld.p < ld.end) {
          ls = attn_segment(a, tpos, ld);
          lj = ls.j0;
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) load_tile(s);
  int stage = 0;

  while (run.p < run.end) {
    const AttnSeg sg = attn_segment(a, tpos, run);
    if (tid == 0) {
      attn_note(a, sg, run);
      if (sg.len < 0) flag_error(a.dev_err, CCONV_DERR_SEQ_LEN);
    }
    attn_advance(a, sg, run);
    // the warp's head and its first position of a tile
    const int hkv = sg.unit / a.rblocks * a.hw + warp * 16 / tpos;
    const int p0 = warp * 16 % tpos, r0 = sg.unit % a.rblocks * (MT * 16);
    const int rows = min(MT * 16, rows_all - r0);
    // ---- Q as left operands: row r is token (r0 + r) / G, head hkv * G + (r0 + r) % G
    auto q_row = [&](int r) {
      const int rr = r0 + r;
      return a.q + (((int64_t)sg.b * a.q_len + rr / a.G) * a.q_rs +
                    (int64_t)(hkv * a.G + rr % a.G) * D) * 2;
    };
    uint32_t q[kQRegs ? MT : 1][kQRegs ? D / 16 : 1][4];
    if constexpr (kQRegs) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = mt * 16 + half * 8 + (lane >> 2);
          const bool in = r < rows && sg.len > 0;
          const char* p = q_row(in ? r : 0) + (lane & 3) * 4;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              q[mt][ks][half + 2 * e] =
                  in ? *reinterpret_cast<const uint32_t*>(p + (ks * 16 + e * 8) * 2) : 0u;
        }
    } else {
      for (int i = lane; i < MT * 16 * C::kUnits; i += 32) {
        const int r = i / C::kUnits, u = i % C::kUnits;
        const bool in = r < rows && sg.len > 0;
        *reinterpret_cast<uint4*>(sq + at<D>(r, u)) =
            in ? ldg16(q_row(r) + u * 16) : make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
    float m[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.0f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.0f;
    }
    for (int j = sg.j0; j < sg.j1; ++j) {
      cp_async_wait<C::kStages - 2>();
      __syncthreads();                 // the tile is there; the oldest one has been read
      load_tile((stage + C::kStages - 1) % C::kStages);
      const uint32_t kb = smem + stage * 2 * C::kTileBytes, vb = kb + C::kTileBytes;
      const int cur = stage;
      stage = (stage + 1) % C::kStages;
      // ---- scores of the warp's 16 positions: two n-tiles of 8
      float s[MT][2][4] = {};
      const int kr = warp * 16 + (lane & 7) + ((lane >> 4) << 3), ku = (lane >> 3) & 1;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t b[4];                 // positions 0-7: k 0-7, k 8-15; positions 8-15: the same
        ldm4(b, kb + at<D>(kr, ks * 2 + ku));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if constexpr (kQRegs) {
            mma(s[mt][0], q[mt][ks], b[0], b[1]);
            mma(s[mt][1], q[mt][ks], b[2], b[3]);
          } else {
            uint32_t qa[4];
            ldm4(qa, smem_addr(sq) + at<D>(mt * 16 + (lane & 15), ks * 2 + (lane >> 4)));
            mma(s[mt][0], qa, b[0], b[1]);
            mma(s[mt][1], qa, b[2], b[3]);
          }
        }
      }
      // ---- mask, running maximum, weights
      const int pos0 = j * tpos + p0 + (lane & 3) * 2;   // + 8 n + {0, 1}
      const unsigned char* tr = there[cur] + warp * 16 + (lane & 3) * 2;
      const uint32_t th = (uint32_t)*reinterpret_cast<const uint16_t*>(tr) |
                          ((uint32_t)*reinterpret_cast<const uint16_t*>(tr + 8) << 16);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t pw[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = mt * 16 + half * 8 + (lane >> 2);
          const int seen = r < rows ? sg.len - a.q_len + 1 + (r0 + r) / a.G : 0;
          float x[4], mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = pos0 + (i >> 1) * 8 + (i & 1);
            x[i] = ((th >> (i * 8)) & 1u) && pos < seen ? sl2 * s[mt][i >> 1][half * 2 + (i & 1)]
                                                     : -INFINITY;
            mx = fmaxf(mx, x[i]);
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[mt][half], mx);
          const float base = mn == -INFINITY ? 0.0f : mn;
          const float corr = ex2(m[mt][half] - base);
          m[mt][half] = mn;
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = ex2(x[i] - base);
            sum += x[i];
          }
          l[mt][half] = fmaf(l[mt][half], corr, sum);
          pw[half] = pack_bf16x2(x[0], x[1]);
          pw[2 + half] = pack_bf16x2(x[2], x[3]);
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[mt][n][half * 2] *= corr;
            o[mt][n][half * 2 + 1] *= corr;
          }
        }
        // ---- weighted values
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t b[4];               // dims 0-7: positions 0-7, 8-15; dims 8-15: the same
          ldm4t(b, vb + at<D>(warp * 16 + (lane & 15), n * 2 + (lane >> 4)));
          mma(o[mt][2 * n], pw, b[0], b[1]);
          mma(o[mt][2 * n + 1], pw, b[2], b[3]);
        }
      }
    }
    // ---- the row sums over the quad, then the warps of one head join: those
    // behind the head's first one leave their part in shared memory, in turn
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        l[mt][half] += __shfl_xor_sync(0xffffffffu, l[mt][half], 1);
        l[mt][half] += __shfl_xor_sync(0xffffffffu, l[mt][half], 2);
      }
    const int per = kWarps >> hw_shift;              // warps of a head
    if (!kQRegs && per > 1) __syncthreads();         // every warp is done with its Q
#pragma unroll 1
    for (int w = 1; w < per; ++w) {
      float* const so = join + (warp / per) * (MT * 16 * (D + 4));
      if (warp % per == w) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float* p = so + (mt * 16 + half * 8 + (lane >> 2)) * (D + 4) + (lane & 3) * 2;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<float2*>(p + n * 8) =
                  make_float2(o[mt][n][half * 2], o[mt][n][half * 2 + 1]);
            if ((lane & 3) == 0) {
              p[D] = m[mt][half];
              p[D + 1] = l[mt][half];
            }
          }
      }
      __syncthreads();
      if (warp % per == 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float* row = so + (mt * 16 + half * 8 + (lane >> 2)) * (D + 4);
            const float mo = row[D], lo = row[D + 1];
            const float mm = fmaxf(m[mt][half], mo), base = mm == -INFINITY ? 0.0f : mm;
            const float f = ex2(m[mt][half] - base), fo = ex2(mo - base);
            m[mt][half] = mm;
            l[mt][half] = fmaf(l[mt][half], f, lo * fo);
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              const float2 v = *reinterpret_cast<const float2*>(row + n * 8 + (lane & 3) * 2);
              o[mt][n][half * 2] = fmaf(o[mt][n][half * 2], f, v.x * fo);
              o[mt][n][half * 2 + 1] = fmaf(o[mt][n][half * 2 + 1], f, v.y * fo);
            }
          }
      }
      __syncthreads();
    }
    if (sg.len < 0 || warp % per != 0) continue;
    float* const part = attn_part(a, sg, D) + (warp / per) * (MT * 16) * (D + 2);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + (lane >> 2), c = (lane & 3) * 2;
        if (r >= rows) continue;
        const float ll = l[mt][half], mn = m[mt][half] * 0.6931471805599453f;   // natural
        if (sg.whole) {
          const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
          const int64_t tok = (int64_t)sg.b * a.q_len + (r0 + r) / a.G;
          const int h = hkv * a.G + (r0 + r) % a.G;
          char* p = a.out + (tok * a.out_rs + (int64_t)h * D + c) * 2;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<uint32_t*>(p + n * 16) =
                pack_bf16x2(o[mt][n][half * 2] * inv, o[mt][n][half * 2 + 1] * inv);
          if (a.lse && c == 0) a.lse[tok * a.Hq + h] = ll > 0.0f ? mn + logf(ll) : -INFINITY;
        } else {
          float* p = part + r * (D + 2);
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2*>(p + n * 8 + c) =
                make_float2(o[mt][n][half * 2], o[mt][n][half * 2 + 1]);
          if (c == 0) {
            p[D] = mn;
            p[D + 1] = ll;
          }
        }
      }
  }
  cp_async_wait<0>();
}

static_assert(kTile == 16 * kWarps, "a warp takes 16 rows");

// Ring, and behind it the joins (none with a head a warp) or the warps' Q.
template <int D, int MT>
int smem_bytes(int hw) {
  const int join = (hw == 4 ? 0 : hw) * MT * 16 * (D + 4) * 4;
  const int q = MT * D <= 128 ? 0 : kWarps * MT * 16 * D * 2;
  return Cfg<D>::kRing + std::max(join, q);
}

template <int D, int MT>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t st) {
  const int smem = smem_bytes<D, MT>(a.hw);
  const cudaError_t e = cudaFuncSetAttribute(
      attn_mma_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_mma_kernel<D, MT><<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_launch_mma(const AttnArgs& a, int D, int grid, cudaStream_t st) {
  if (a.rows == 16)
    return D == 64 ? launch<64, 1>(a, grid, st) : D == 128 ? launch<128, 1>(a, grid, st)
                                                          : launch<256, 1>(a, grid, st);
  return D == 64 ? launch<64, 2>(a, grid, st) : launch<128, 2>(a, grid, st);
}

}  // namespace cconv
