// attn_decode_q8 in bf16: attention of new tokens over a cache in 8 bits, split as in
// attn_decode.cuh, with the products on the warp-level tensor instruction (m16n8k16).
//
// It is built as the kernel over a cache in bf16 (attn_mma.cu: a warp that copies
// positions into a ring, four that take 16 rows of a tile each), for half the bytes.
// What differs:
// - Values go to the products as fp16, which holds every e4m3 value, by one
//   instruction a pair. (bf16 would hold them too; that conversion takes four.) The
//   four bytes that ldmatrix leaves in a lane are two pairs of K's dims, so that Q is
//   laid out to match, and of V two dims of two positions, whose bytes are brought
//   beside one another first; the sums' columns then lie four side by side.
// - Q as fp16 has the power of two of its row's largest value taken out. Scores are
//   multiplied by that, by the scale and by their key's power of two.
// - A value's power of two 2^e goes to its weight: weights are 2^(s + e - M), with M
//   the running maximum of s + e, beside the running maximum m and sum of 2^(s - m).
//   No spread of the scales then costs range. Weights are fp16, 2^15 times as large,
//   so that those from 2^-29 of the largest on have all 11 bits. That is one rounding
//   more than none: 2^-12 of a result, whose own is 2^-9.
// - Scales are bytes that lie elsewhere; a warp of their own reads them into registers,
//   two tiles before they are needed, and puts them beside the tile. (With the copies
//   in one warp that warp's instructions were what bounded the kernel.)
// - A tile is 128 rows, 32 a warp, so that it has as many bytes.
#include "attn_decode.cuh"
#include "q8.cuh"
#include "tc.cuh"

#include <math.h>

namespace cconv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = (kWarps + 2) * 32;   // and a warp for the copies, one for scales
constexpr int kTile = 128;          // rows of a tile (positions x heads); 32 a warp
constexpr int kMaxStages = 4;
constexpr long long kWaitClocks = 4000000000LL;   // seconds; a copy takes microseconds
constexpr float kLift = 15.0f;      // log2 of what weights are multiplied by

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// All ones in the bytes that are NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) {
  return (((v & 0x7f7f7f7fu) + 0x01010101u & 0x80808080u) >> 7) * 0xffu;
}
// 2^-x of a row's largest magnitude m, which brings it to [2^14, 2^15), and x.
__device__ __forceinline__ float q_factor(float m, float& x) {
  const uint32_t e = __float_as_uint(m) >> 23;
  const bool plain = e >= 15 && e < 255;      // (smaller, or not finite: as it is)
  x = plain ? (float)e - (127 + 14) : 0.0f;
  return plain ? __uint_as_float((127 + 127 + 14 - e) << 23) : 1.0f;
}

// Bounded wait of a whole warp. A warp that it gives up leaves the kernel; what
// waits for that warp is given up in turn, so no barrier behind the first of these
// waits may be one without a limit.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, int phase, int32_t* err) {
  long long t0 = 0;
#pragma unroll 1
  for (uint32_t it = 1; !__any_sync(0xffffffffu, mbar_try(bar, phase)); ++it) {
    if ((it & 255u) == 0) {
      const long long now = clock64();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, now - t0 > kWaitClocks)) {
        flag_error(err, CCONV_DERR_TIMEOUT);
        return false;
      }
    }
  }
  __syncwarp();
  return true;
}

// What a warp that gives a wait up leaves the kernel by, so that no copy lands
// behind the block's end (as in attn_mma.cu), nor this kernel before the one that it
// runs beside.
__device__ __noinline__ void settle(uint64_t* full, int stages, int st, int ph, int32_t* err) {
  for (int i = 0; i < stages; ++i) wait_bar(&full[i], i < st ? ph ^ 1 : ph, err);
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// MT row tiles of 16. Q stays in registers where it fits beside the sums, else
// in shared memory.
template <int D, int MT, bool SHARED>
__global__ void __launch_bounds__(kThreads, attn_mma_blocks(D, MT * 16, true))
    attn_mma_q8_kernel(const AttnArgs a, const int stages) {
  constexpr bool kQRegs = MT == 1;
  constexpr int kQPitch = D * 2 + 16;
  extern __shared__ __align__(128) unsigned char attn_dyn[];
  __shared__ int64_t scan[kThreads + 4];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], met;
  __shared__ __align__(16) unsigned char there[kMaxStages][kTile];   // positions that hold a token
  // of K: its rows' powers of two; of V: their exponents; head by head
  __shared__ __align__(16) float scales[kMaxStages][2][kTile];
  __shared__ float row_x[kWarps][MT * 16];          // powers of two of Q's rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // position x of a tile lies at off(x) of its place: rows of a group side by side
  const int rowb = a.hw * D, gs = a.group_shift, group = 1 << gs;
  auto off = [&](int x) { return (uint32_t)(x * rowb + (x >> gs) * 16); };
  const int hw_shift = a.hw == 4 ? 2 : a.hw >> 1, tpos = kTile >> hw_shift;   // positions a tile
  const uint32_t half_stage = off(tpos);        // K, then V
  // behind the ring: the joins of at most two heads, or the warps' own Q before
  unsigned char* const behind = attn_dyn + stages * 2 * half_stage;
  float* const join = reinterpret_cast<float*>(behind);
  unsigned char* const sq = behind + warp * (MT * 16 * kQPitch);
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init(&met, kWarps);
    fence_mbar_init();
  }
  AttnRun run;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!attn_split<kThreads, SHARED>(a, tpos, scan, run)) return;
  const int rows_all = a.G * a.q_len;
  const float sl2 = a.scale * 1.4426950408889634f;

  if (warp == kWarps) {
    // ---- loads: lane l has the copies l, l + 32, .. of a tile: K and V of each
    // group of positions, whole or head by head. The pages of the copies after
    // these are looked up while these are issued.
    const int ps = a.s_head == D ? 0 : hw_shift;      // log2 of the copies of a position
    const uint32_t bytes = rowb >> ps;                // of a copy and position
    // the lane's copies: K or V, a head or all, positions pl0, pl0 + dpl, ..
    const int isv = lane & 1, piece = (lane >> 1) & ((1 << ps) - 1);
    const int pl0 = lane >> (1 + ps) << gs, dpl = 16 >> ps << gs;
    unsigned char* const dst0 = attn_dyn + isv * half_stage + piece * D;
    const bool notes = isv == 0 && piece == 0;
    int st = 0, ph = 1;               // (the first round's places are free)
    while (run.p < run.end) {
      const AttnSeg s = attn_segment<SHARED>(a, tpos, run);
      attn_advance(a, s, run);
      const int32_t* tab = a.table + (int64_t)s.b * a.table_rs;
      const char* const src0 = (isv ? a.vc : a.kc) +
                               (int64_t)(s.unit / a.rblocks * a.hw + piece) * a.s_head;
      // page of position pos, as the table has it
      auto look = [&](int pos, bool in) {
        return in && pos < s.len ? tab[a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size]
                                 : -1;
      };
      int ahead = look(s.base + s.j0 * tpos + pl0, pl0 < tpos);
      for (int j = s.j0; j < s.j1; ++j) {
        const uint32_t place = st * 2 * half_stage;
        const int t0 = s.base + j * tpos;
        int pl = pl0;
        for (int p = 0; p < tpos; p += dpl, pl += dpl) {       // (p: of lane 0)
          const int pos = t0 + pl, page = ahead;
          const bool in = pl < tpos;
          ahead = p + dpl < tpos ? look(pos + dpl, pl + dpl < tpos)
                                 : look(t0 + tpos + pl0, j + 1 < s.j1 && pl0 < tpos);
          int held = in ? min(group, max(s.len - pos, 0)) : 0;   // positions with a token
          if (held > 0 && (uint32_t)page >= (uint32_t)a.num_pages) {
            flag_error(a.dev_err, CCONV_DERR_PAGE);
            held = 0;
          }
          if (p == 0 && !wait_bar(&empty[st], ph, a.dev_err))
            return settle(full, stages, st, ph, a.dev_err);
          if (in) {
            // (positions before the request's first one are left out, too)
            const int skip = SHARED ? min(max(s.start - pos, 0), held) : 0;
            if (notes)
              for (int k = 0; k < group; ++k) there[st][pl + k] = k >= skip && k < held;
            unsigned char* const dst = dst0 + place + off(pl);
            if (held > skip) {
              const int tok = a.page_shift >= 0 ? pos & (a.page_size - 1) : pos % a.page_size;
              const uint32_t n = (held - skip) * bytes;
              mbar_expect(&full[st], n);
              bulk_load(dst + skip * bytes, src0 + page * a.s_page + (tok + skip) * a.s_tok, n,
                        &full[st]);
            }
            if (isv && held - skip < group) {
              for (uint32_t i = 0; i < group * bytes; i += 16)
                if (i < skip * bytes || i >= held * bytes)
                  *reinterpret_cast<uint4*>(dst + i) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async();      // before a later copy into the same place
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        if (++st == stages) st = 0, ph ^= 1;
      }
    }
    if (SHARED && blockIdx.x == 0)        // (as in attn_mma.cu)
      asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (warp == kWarps + 1) {
    // ---- scales: lane l has rows l, l + 32, .. of a tile, row r being position r % tpos
    // of head r / tpos. Those of a tile are requested two tiles before it, their pages
    // looked up one before that.
    int st = 0, ph = 1;
    while (run.p < run.end) {
      const AttnSeg s = attn_segment<SHARED>(a, tpos, run);
      attn_advance(a, s, run);
      const int32_t* tab = a.table + (int64_t)s.b * a.table_rs;
      const int head = s.unit / a.rblocks * a.hw;
      int page[4];
      auto look = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = s.base + j * tpos + ((lane + 32 * i) & (tpos - 1));
          page[i] = j < s.j1 && pos < s.len
                        ? tab[a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size]
                        : -1;
        }
      };
      struct Bytes {
        uint32_t k[4], v[4];
      };
      auto load = [&](int j) {
        Bytes c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i, pos = s.base + j * tpos + (r & (tpos - 1));
          c.k[i] = c.v[i] = 127;
          if ((uint32_t)page[i] < (uint32_t)a.num_pages) {
            const int tok = a.page_shift >= 0 ? pos & (a.page_size - 1) : pos % a.page_size;
            const int64_t at =
                page[i] * a.c_page + tok * a.c_tok + (int64_t)(head + r / tpos) * a.c_head;
            c.k[i] = a.ksc[at];
            c.v[i] = a.vsc[at];
          }
        }
        return c;
      };
      look(s.j0);
      Bytes c0 = load(s.j0);
      look(s.j0 + 1);
      Bytes c1 = load(s.j0 + 1);
      look(s.j0 + 2);
#pragma unroll 1
      for (int j = s.j0; j < s.j1; ++j) {
        const Bytes c2 = load(j + 2);
        look(j + 3);
        if (!wait_bar(&empty[st], ph, a.dev_err)) return settle(full, stages, st, ph, a.dev_err);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          scales[st][0][lane + 32 * i] = q8_scale(c0.k[i]);
          scales[st][1][lane + 32 * i] = (float)c0.v[i] - 127.0f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        if (++st == stages) st = 0, ph ^= 1;
        c0 = c1, c1 = c2;
      }
    }
    return;
  }
  int stage = 0, phase = 0, meets = 0;
  // The warps that compute, among themselves.
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&met);
    return wait_bar(&met, meets++ & 1, a.dev_err);
  };

  while (run.p < run.end) {
    const AttnSeg sg = attn_segment<SHARED>(a, tpos, run);
    if (tid == 0) {
      attn_note(a, sg, run);
      if (sg.len < 0) flag_error(a.dev_err, CCONV_DERR_SEQ_LEN);
    }
    attn_advance(a, sg, run);
    // the warp's head and its first position of a tile
    const int hl = warp * 32 / tpos, hkv = sg.unit / a.rblocks * a.hw + hl;
    const int p_warp = warp * 32 % tpos, r0 = sg.unit % a.rblocks * (MT * 16);
    const int rows = min(MT * 16, rows_all - r0);
    // ---- Q as left operands: row r is token (r0 + r) / G, head hkv * G + (r0 + r) % G.
    // Of 16 dims, 4 c + {0, 1} are where the product has 2 c + {0, 1}, and
    // 4 c + {2, 3} where it has 8 + 2 c + {0, 1}: as the bytes of K come.
    auto q_row = [&](int r) {
      const int rr = r0 + r;
      return a.q + (((int64_t)sg.b * a.q_len + rr / a.G) * a.q_rs +
                    (int64_t)(hkv * a.G + rr % a.G) * D) * 2;
    };
    uint32_t q[kQRegs ? MT : 1][kQRegs ? D / 16 : 1][4];
    float rf[MT][2];                    // what a row's scores are multiplied by
    if constexpr (kQRegs) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = mt * 16 + half * 8 + (lane >> 2);
          const bool in = r < rows && sg.len > 0;
          const char* p = q_row(in ? r : 0) + (lane & 3) * 8;
          uint2 raw[D / 16];
          float m = 0.0f;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            raw[ks] = in ? *reinterpret_cast<const uint2*>(p + ks * 32) : make_uint2(0u, 0u);
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(raw[ks].x << 16)),
                               fabsf(__uint_as_float(raw[ks].x & 0xffff0000u))));
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(raw[ks].y << 16)),
                               fabsf(__uint_as_float(raw[ks].y & 0xffff0000u))));
          }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          float x;
          const float f = q_factor(m, x);
          rf[mt][half] = x;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            q[mt][ks][half] = pack_f16x2(__uint_as_float(raw[ks].x << 16) * f,
                                         __uint_as_float(raw[ks].x & 0xffff0000u) * f);
            q[mt][ks][half + 2] = pack_f16x2(__uint_as_float(raw[ks].y << 16) * f,
                                             __uint_as_float(raw[ks].y & 0xffff0000u) * f);
          }
        }
    } else {
      constexpr int kLanes = D / 8;     // of a row, 8 dims each
#pragma unroll 1
      for (int i = lane; i < MT * 16 * kLanes; i += 32) {
        const int r = i / kLanes, u = i % kLanes;
        const bool in = r < rows && sg.len > 0;
        float f[8];
        unpack16<__nv_bfloat16>(in ? ldg16(q_row(r) + u * 16) : make_uint4(0u, 0u, 0u, 0u), f);
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        float x;
        const float k = q_factor(m, x);
        unsigned char* const to = sq + r * kQPitch + (u >> 1) * 32 + (u & 1) * 8;
        *reinterpret_cast<uint2*>(to) =
            make_uint2(pack_f16x2(f[0] * k, f[1] * k), pack_f16x2(f[4] * k, f[5] * k));
        *reinterpret_cast<uint2*>(to + 16) =
            make_uint2(pack_f16x2(f[2] * k, f[3] * k), pack_f16x2(f[6] * k, f[7] * k));
        if (u == 0) row_x[warp][r] = x;
      }
      __syncwarp();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          rf[mt][half] = row_x[warp][mt * 16 + half * 8 + (lane >> 2)];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) rf[mt][half] = ldexpf(sl2, (int)rf[mt][half]);
    // maxima of scores (m) and of scores with their value's power of two (mv)
    float m[MT][2], mv[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = mv[mt][0] = mv[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.0f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.0f;
    }
    for (int j = sg.j0; j < sg.j1; ++j) {
      if (!wait_bar(&full[stage], phase, a.dev_err))
        return settle(full, stages, stage, phase, a.dev_err);
      const uint32_t place = smem_addr(attn_dyn) + stage * 2 * half_stage + hl * D;
      const int cur = stage;
      if (++stage == stages) stage = 0, phase ^= 1;
      const uint32_t kb = place + off(p_warp), vb = kb + half_stage;
      const unsigned char* const tr = there[cur] + p_warp;
      const float* const ks = scales[cur][0] + hl * tpos + p_warp;
      const float* const vs = scales[cur][1] + hl * tpos + p_warp;
      // ---- scores of the warp's 32 positions: four n-tiles of 8
      float s[MT][4][4] = {};
      const uint32_t ka = kb + off((lane & 7) + ((lane >> 4) << 3)) + ((lane >> 3) & 1) * 16;
      const uint32_t step16 = off(16);
#pragma unroll
      for (int d = 0; d < D / 16; d += 2) {
        uint32_t b[2][4];              // positions 0-7: bytes 0-15, 16-31; positions 8-15: the same
        tc::ldmatrix4(b[0], ka + d * 16);
        tc::ldmatrix4(b[1], ka + step16 + d * 16);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint32_t b0 = e4m3x2_to_f16x2(b[g][t]), b1 = e4m3x2_to_f16x2(b[g][t] >> 16);
            const uint32_t b2 = e4m3x2_to_f16x2(b[g][2 + t]),
                           b3 = e4m3x2_to_f16x2(b[g][2 + t] >> 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if constexpr (kQRegs) {
                tc::mma16h(s[mt][2 * g], q[mt][d + t], b0, b1);
                tc::mma16h(s[mt][2 * g + 1], q[mt][d + t], b2, b3);
              } else {
                uint32_t qa[4];
                tc::ldmatrix4(qa, smem_addr(sq) + (mt * 16 + (lane & 15)) * kQPitch +
                                      (d + t) * 32 + (lane >> 4) * 16);
                tc::mma16h(s[mt][2 * g], qa, b0, b1);
                tc::mma16h(s[mt][2 * g + 1], qa, b2, b3);
              }
            }
          }
      }
      // the powers of two of the lane's eight positions: q0 + 8 n + {0, 1}
      const int q0 = (lane & 3) * 2;
      float ve[8];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float2 kf = *reinterpret_cast<const float2*>(ks + q0 + 8 * n);
        const float2 e = *reinterpret_cast<const float2*>(vs + q0 + 8 * n);
        ve[2 * n] = e.x;
        ve[2 * n + 1] = e.y;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][n][i] *= (i & 1 ? kf.y : kf.x);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[mt][i >> 2][i & 3] *= rf[mt][(i >> 1) & 1];
      // ---- masks, running maxima, weights
      const int pos0 = sg.base + j * tpos + p_warp;    // the first position
      // Draft tokens' positions are hidden from the rows before them by a weight of
      // zero, which a NaN among their values would get through: such values (`wild`)
      // are kept out of the product and added to the rows that see them.
      const int x0 = max(0, sg.len - a.q_len + 1 - pos0), x1 = min(32, sg.len - pos0);
      bool wild = false;
      if (x0 < x1) {
        for (int x = x0; x < x1; ++x)
          for (int i = lane; i < D / 4; i += 32)
            wild |= nan_bytes(lds32(vb + off(x) + i * 4)) != 0;
        wild = __any_sync(0xffffffffu, wild);
      }
      const uint4 all = *reinterpret_cast<const uint4*>(tr);
      const uint4 more = *reinterpret_cast<const uint4*>(tr + 16);
      if (pos0 + 31 > sg.len - a.q_len ||
          (all.x & all.y & all.z & all.w & more.x & more.y & more.z & more.w) != 0x01010101u) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = mt * 16 + half * 8 + (lane >> 2);
            const int seen = r < rows ? sg.len - a.q_len + 1 + (r0 + r) / a.G : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int x = q0 + (i >> 1) * 8 + (i & 1);
              if (!tr[x] || pos0 + x >= seen) s[mt][i >> 1][half * 2 + (i & 1)] = -INFINITY;
            }
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t pw[2][4];
        float corr[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[8], t[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = s[mt][i >> 1][half * 2 + (i & 1)];
            t[i] = x[i] + ve[i];
          }
          float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                           fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
          float tx = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])),
                           fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, 2));
          const float mn = fmaxf(m[mt][half], mx), tn = fmaxf(mv[mt][half], tx);
          const float base = mn == -INFINITY ? 0.0f : mn, tbase = tn == -INFINITY ? 0.0f : tn;
          corr[half] = tc::ex2(mv[mt][half] - tbase);
          float sum = 0.0f, more_sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            sum += tc::ex2(x[i] - base);
            more_sum += tc::ex2(x[i + 1] - base);
          }
          l[mt][half] = fmaf(l[mt][half], tc::ex2(m[mt][half] - base), sum + more_sum);
          m[mt][half] = mn;
          mv[mt][half] = tn;
          const float up = tbase - kLift;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            pw[g][half] = pack_f16x2(tc::ex2(t[4 * g] - up), tc::ex2(t[4 * g + 1] - up));
            pw[g][2 + half] = pack_f16x2(tc::ex2(t[4 * g + 2] - up), tc::ex2(t[4 * g + 3] - up));
          }
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[mt][n][0] *= corr[0];
            o[mt][n][1] *= corr[0];
            o[mt][n][2] *= corr[1];
            o[mt][n][3] *= corr[1];
          }
        }
        // ---- weighted values: of 16 dims, the even ones are one n-tile, the odd ones
        // another
        const uint32_t va = vb + off(lane & 15) + (lane >> 4) * 16;
        if (!wild) {
#pragma unroll
          for (int n = 0; n < D / 16; n += 2) {
            uint32_t b[2][4];          // dims 0-15: positions 0-7, 8-15; dims 16-31: the same
            tc::ldmatrix4_trans(b[0], va + n * 16);
            tc::ldmatrix4_trans(b[1], va + step16 + n * 16);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const uint32_t v0 = __byte_perm(b[g][2 * t], 0u, 0x3120),
                               v1 = __byte_perm(b[g][2 * t + 1], 0u, 0x3120);
                tc::mma16h(o[mt][2 * (n + t)], pw[g], e4m3x2_to_f16x2(v0), e4m3x2_to_f16x2(v1));
                tc::mma16h(o[mt][2 * (n + t) + 1], pw[g], e4m3x2_to_f16x2(v0 >> 16),
                           e4m3x2_to_f16x2(v1 >> 16));
              }
          }
        } else {
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {
            const uint32_t pg[4] = {g ? pw[1][0] : pw[0][0], g ? pw[1][1] : pw[0][1],
                                    g ? pw[1][2] : pw[0][2], g ? pw[1][3] : pw[0][3]};
#pragma unroll
            for (int n = 0; n < D / 16; n += 2) {
              uint32_t b[4];
              tc::ldmatrix4_trans(b, va + g * step16 + n * 16);
#pragma unroll
              for (int i = 0; i < 4; ++i) {        // positions 16 g + q0 + 8 (i & 1) + {0, 1}
                const int x = 16 * g + q0 + (i & 1) * 8;
                const uint32_t hidden =
                    (x >= x0 ? 0x00ff00ffu : 0u) | (x + 1 >= x0 ? 0xff00ff00u : 0u);
                b[i] = __byte_perm(b[i], 0u, 0x3120);
                b[i] &= ~(nan_bytes(b[i]) & hidden);
              }
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                tc::mma16h(o[mt][2 * (n + t)], pg, e4m3x2_to_f16x2(b[2 * t]),
                           e4m3x2_to_f16x2(b[2 * t + 1]));
                tc::mma16h(o[mt][2 * (n + t) + 1], pg, e4m3x2_to_f16x2(b[2 * t] >> 16),
                           e4m3x2_to_f16x2(b[2 * t + 1] >> 16));
              }
            }
          }
#pragma unroll 1
          for (int x = x0; x < x1; ++x)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int r = mt * 16 + half * 8 + (lane >> 2);
              if (r >= rows || pos0 + x >= sg.len - a.q_len + 1 + (r0 + r) / a.G) continue;
#pragma unroll
              for (int n = 0; n < D / 16; ++n) {     // dims 16 n + 4 c + {0, 1, 2, 3}
                const uint32_t v = nan_bytes(lds32(vb + off(x) + n * 16 + q0 * 2));
                const float nan = __uint_as_float(0x7fc00000u);
                if (v & 0xffu) o[mt][2 * n][half * 2] = nan;
                if (v & 0xff00u) o[mt][2 * n + 1][half * 2] = nan;
                if (v & 0xff0000u) o[mt][2 * n][half * 2 + 1] = nan;
                if (v & 0xff000000u) o[mt][2 * n + 1][half * 2 + 1] = nan;
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[cur]);
    }
    // ---- the row sums over the quad, and sums in units of 2^m again; then the warps of
    // one head join: those behind the head's first one leave their part in shared
    // memory, in turn
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        l[mt][half] += __shfl_xor_sync(0xffffffffu, l[mt][half], 1);
        l[mt][half] += __shfl_xor_sync(0xffffffffu, l[mt][half], 2);
        const float f = m[mt][half] == -INFINITY ? 1.0f
                                                 : exp2f(mv[mt][half] - m[mt][half] - kLift);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[mt][n][half * 2] *= f;
          o[mt][n][half * 2 + 1] *= f;
        }
      }
    const int per = kWarps >> hw_shift;              // warps of a head
    // (with Q in shared memory: every warp is done with its own)
    if (!kQRegs && per > 1 && !meet()) return settle(full, stages, stage, phase, a.dev_err);
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
      if (!meet()) return settle(full, stages, stage, phase, a.dev_err);
      if (warp % per == 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float* row = so + (mt * 16 + half * 8 + (lane >> 2)) * (D + 4);
            const float mo = row[D], lo = row[D + 1];
            const float mm = fmaxf(m[mt][half], mo), base = mm == -INFINITY ? 0.0f : mm;
            const float f = tc::ex2(m[mt][half] - base), fo = tc::ex2(mo - base);
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
      if (!meet()) return settle(full, stages, stage, phase, a.dev_err);
    }
    if (sg.len < 0 || warp % per != 0) continue;
    float* const part = attn_part<SHARED>(a, sg, D) + (warp / per) * (MT * 16) * (D + 2);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + (lane >> 2), c = (lane & 3) * 4;
        if (r >= rows) continue;
        const float ll = l[mt][half], mn = m[mt][half] * 0.6931471805599453f;   // natural
        if (sg.whole) {
          const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
          const int64_t tok = (int64_t)sg.b * a.q_len + (r0 + r) / a.G;
          const int h = hkv * a.G + (r0 + r) % a.G;
          char* p = a.out + (tok * a.out_rs + (int64_t)h * D + c) * 2;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            const float *e = o[mt][2 * n] + half * 2, *d = o[mt][2 * n + 1] + half * 2;
            *reinterpret_cast<uint2*>(p + n * 32) = make_uint2(
                pack_bf16x2(e[0] * inv, d[0] * inv), pack_bf16x2(e[1] * inv, d[1] * inv));
          }
          if (a.lse && c == 0) a.lse[tok * a.Hq + h] = ll != 0.0f ? mn + logf(ll) : -INFINITY;
        } else {
          float* p = part + r * (D + 2);
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            const float *e = o[mt][2 * n] + half * 2, *d = o[mt][2 * n + 1] + half * 2;
            *reinterpret_cast<float2*>(p + n * 16 + c) = make_float2(e[0], d[0]);
            *reinterpret_cast<float2*>(p + n * 16 + c + 2) = make_float2(e[1], d[1]);
          }
          if (c == 0) {
            p[D] = mn;
            p[D + 1] = ll;
          }
        }
      }
  }
}

static_assert(kTile == 32 * kWarps, "a warp takes 32 rows");

template <int D, int MT, bool SHARED>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t st) {
  // the ring, and behind it the joins (none with a head a warp) or the warps' Q
  const int tpos = kTile / a.hw, stage = 2 * (tpos * a.hw * D + (tpos >> a.group_shift) * 16);
  const int join = (a.hw == 4 ? 0 : a.hw) * MT * 16 * (D + 4) * 4;
  const int q = MT == 1 ? 0 : kWarps * MT * 16 * (D * 2 + 16);
  int stages = D == 64 ? 4 : 3;
  // as many as let the grid's blocks of an SM all be there (228 KB, less what the
  // kernel has besides)
  const int most = 228 * 1024 / attn_mma_blocks(D, MT * 16, true) - 10 * 1024;
  while (stages > 2 && stages * stage + std::max(join, q) > most) --stages;
  const int smem = stages * stage + std::max(join, q);
  static std::atomic<uint64_t> full;
  const void* const f = reinterpret_cast<const void*>(attn_mma_q8_kernel<D, MT, SHARED>);
  const cudaError_t e = mix_full_smem(f, full);
  if (e != cudaSuccess) return e;
  if constexpr (!SHARED) {
    attn_mma_q8_kernel<D, MT, SHARED><<<grid, kThreads, smem, st>>>(a, stages);
    return cudaGetLastError();
  } else {
    return attn_launch_beside(attn_mma_q8_kernel<D, MT, SHARED>, a, stages, grid, kThreads, smem,
                              st);
  }
}

template <bool SHARED>
cudaError_t launch_d(const AttnArgs& a, int D, int grid, cudaStream_t st) {
  if (a.rows == 16)
    return D == 64    ? launch<64, 1, SHARED>(a, grid, st)
           : D == 128 ? launch<128, 1, SHARED>(a, grid, st)
                      : launch<256, 1, SHARED>(a, grid, st);
  return D == 64 ? launch<64, 2, SHARED>(a, grid, st) : launch<128, 2, SHARED>(a, grid, st);
}

}  // namespace

cudaError_t attn_launch_mma_q8(const AttnArgs& a, int D, int grid, bool shared, cudaStream_t st) {
  return shared ? launch_d<true>(a, D, grid, st) : launch_d<false>(a, D, grid, st);
}

}  // namespace cconv
