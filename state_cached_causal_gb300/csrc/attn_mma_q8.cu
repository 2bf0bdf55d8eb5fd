// attn_decode_q8 in bf16: attention of new tokens over a cache in 8 bits, split as in
// attn_decode.cuh, with the products on the warp-level tensor instruction (m16n8k16).
//
// It is built as the kernel over a cache in bf16 (attn_mma.cu: a warp that copies
// positions into a ring, four that take their rows of a tile each), for half the bytes.
// What differs:
// - The products are the transposed ones, S^T = K Q^T and O^T = V^T P^T, whose narrow
//   side of 8 is the query rows': with 16 rows on the other side, half of the softmax
//   and of the sums was of rows that do not exist where a kv head has 4 or 8. The weights
//   are turned in registers (movmatrix).
// - Values go to the products as fp16, which holds every e4m3 value, by one
//   instruction a pair. (bf16 would hold them too; that conversion takes four.) The
//   four bytes that ldmatrix leaves in a lane are two pairs of K's dims, so that Q is
//   laid out to match, and of V two dims of two positions, whose bytes are brought
//   beside one another first.
// - Q as fp16 has the power of two of its row's largest value taken out. Scores are
//   multiplied by that, by the scale and by their key's power of two.
// - A value's power of two 2^e goes to its weight: weights are 2^(s + e - M + kLift), M
//   a reference that follows the largest s + e (and is left until that has passed it
//   by kSlack: lanes then need no more than a vote). The sum of 2^(s - M) is that of the
//   weights times 2^-e. Where some |e| is over 40 that could leave fp32's range: from
//   there on ("wide") the sum has a maximum of its own. Weights are fp16: 11 bits from
//   2^-22 of the largest on, 2^-33 of it at least. That is one rounding more than none:
//   2^-12 of a result, whose own is 2^-9. That holds for powers of two that are the
//   least ones of their rows. Others are allowed, so that a tile which raises the reference
//   is looked through first, and brought into that form (`fill_row`).
// - Scales are bytes that lie elsewhere; a warp of their own reads them into registers,
//   two tiles before they are needed, and puts them beside the tile. (With the copies
//   in one warp that warp's instructions were what bounded the kernel.)
// - A tile is 128 rows, 32 a warp, so that it has as many bytes.
//
// 256 requests of up to 8192 positions, 16 query heads on 4 kv heads of 128 (1.07 GB):
// 198 us, 5.4 TB/s. It is bound by the bytes, nearly: the copies alone, without the
// products, take 173 (in bf16 the cache takes 340). With rows as the products' side of
// 16 and one warp for copies and scales 270; with the scales in their own warp 216.
// 64 requests of 4 tokens (16 rows a kv head, 127 MB): 54 us: twice the softmax and the
// products a byte, whose latencies eight computing warps an SM do not hide (issue slots
// 37 %, and some of a warp's values spilled at 168 registers).
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
constexpr float kLift = 8.0f;       // log2 of what weights are multiplied by
constexpr float kSlack = 7.0f;      // how far the largest may pass the reference (fp16: 2^16)
constexpr float kMild = 40.0f;      // |e| of values whose sums need no maximum of their own

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
// Four e4m3 values as fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
// An 8 x 8 matrix of 16-bit values, a row's two in a lane, transposed.
__device__ __forceinline__ uint32_t turn(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
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

// Whether one of a row's D values has the magnitude that the largest one has where the
// scale is the least one: 224 and above (and none is NaN). Rolled: a block comes here a few
// times, and fetching the code was what it took (unrolled, 64 requests of 4 tokens 56 us;
// so 52; 50 without the look).
template <int D>
__device__ __forceinline__ bool row_full(uint32_t addr) {
  uint32_t full = 0u, nan = 0u;
#pragma unroll 1
  for (int i = 0; i < D; i += 16) {
    uint32_t v[4];
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr + i)
                 : "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      full |= (v[k] & 0x7f7f7f7fu) + 0x0a0a0a0au;       // (0x76 is 224)
      nan |= (v[k] & 0x7f7f7f7fu) + 0x01010101u;
    }
  }
  return (full & 0x80808080u) != 0u && (nan & 0x80808080u) == 0u;
}
// A row of `bytes` e4m3 values: if none is as large as above, they are multiplied by the
// power of two 2^x that brings the largest finite one there, and x is returned; kNothing
// for a row of zeros, 0 for any other.
constexpr float kNothing = 300.0f;
__device__ __noinline__ float fill_row(uint32_t addr, int bytes) {
  uint32_t most = 0u;
#pragma unroll 1
  for (int i = 0; i < bytes; i += 4) {
    const uint32_t v = lds32(addr + i);
    most = __vmaxu4(most, v & 0x7f7f7f7fu & ~nan_bytes(v));
  }
  most = __vmaxu4(most, most >> 16);
  const uint32_t b = max(most & 0xffu, most >> 8 & 0xffu);
  if (b >= 0x76u) return 0.0f;
  if (b == 0u) return kNothing;
  // 2^(e - 7) (1 + f / 8), below 2^-6 too; 448 is that of e = 15 and f = 6
  const int j = 31 - __clz(b), e = b < 8u ? j - 2 : (int)(b >> 3);
  const uint32_t f = (b < 8u ? b << (3 - j) : b) & 7u;
  const int x = (f < 7u ? 15 : 14) - e;
  const uint32_t x0 = (uint32_t)(x / 2 + 15) << 10, x1 = (uint32_t)(x - x / 2 + 15) << 10;
#pragma unroll 1
  for (int i = 0; i < bytes; i += 4) {
    uint32_t h[2], r[2];
    e4m3x4_to_f16(lds32(addr + i), h[0], h[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      asm("{\n\t.reg .b16 y;\n\t.reg .b32 a, x;\n\tmov.b32 x, {%2, %2};\n\t"
          "mul.rn.f16x2 a, %1, x;\n\tmov.b32 x, {%3, %3};\n\tmul.rn.f16x2 a, a, x;\n\t"
          "cvt.rn.satfinite.e4m3x2.f16x2 y, a;\n\tcvt.u32.u16 %0, y;\n\t}"
          : "=r"(r[k])
          : "r"(h[k]), "h"((uint16_t)x0), "h"((uint16_t)x1));
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr + i), "r"(r[0] | r[1] << 16) : "memory");
  }
  return (float)x;
}

// What a warp that gives a wait up leaves the kernel by, so that no copy lands
// behind the block's end (as in attn_mma.cu), nor this kernel before the one that it
// runs beside.
__device__ __noinline__ void settle(uint64_t* full, int stages, int st, int ph, int32_t* err) {
  for (int i = 0; i < stages; ++i) wait_bar(&full[i], i < st ? ph ^ 1 : ph, err);
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// NT row tiles of 8. Q stays in registers where it fits beside the sums, else in
// shared memory.
__host__ __device__ constexpr bool q_in_regs(int D, int NT) { return D * NT <= 256; }
template <int D, int NT, bool SHARED>
__global__ void __launch_bounds__(kThreads, attn_mma_blocks(D, NT * 8, true))
    attn_mma_q8_kernel(const AttnArgs a, const int stages) {
  constexpr bool kQRegs = q_in_regs(D, NT);
  constexpr int kRows = NT * 8, kQPitch = D * 2 + 16;
  extern __shared__ __align__(128) unsigned char attn_dyn[];
  __shared__ int64_t scan[kThreads + 4];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], met;
  __shared__ __align__(16) unsigned char there[kMaxStages][kTile];   // positions that hold a token
  // a row's K power of two and V exponent e, head by head; and whether all |e| are at
  // most kMild
  __shared__ __align__(16) float2 scales[kMaxStages][kTile];
  __shared__ bool mild[kMaxStages];
  __shared__ float row_x[kWarps][kRows];            // powers of two of Q's rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // position x of a tile lies at off(x) of its place: rows of a group side by side
  const int rowb = a.hw * D, gs = a.group_shift, group = 1 << gs;
  auto off = [&](int x) { return (uint32_t)(x * rowb + (x >> gs) * 16); };
  const int hw_shift = a.hw == 4 ? 2 : a.hw >> 1, tpos = kTile >> hw_shift;   // positions a tile
  const uint32_t half_stage = off(tpos);        // K, then V
  // behind the ring: the joins of at most two heads, or the warps' own Q before
  unsigned char* const behind = attn_dyn + stages * 2 * half_stage;
  float* const join = reinterpret_cast<float*>(behind);
  unsigned char* const sq = behind + warp * (kRows * kQPitch);
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
  // Q carries the scale's sign (and a scale of zero is the least normal number, which
  // leaves hidden scores at -inf)
  const float sl2 = fabsf(a.scale) * 1.4426950408889634f;
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;

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
        bool near = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = (float)c0.v[i] - 127.0f;
          near = near && fabsf(e) <= kMild;
          scales[st][lane + 32 * i] = make_float2(q8_scale(c0.k[i]), e);
        }
        near = __all_sync(0xffffffffu, near);
        if (lane == 0) mild[st] = near;
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
    const int p_warp = warp * 32 % tpos, r0 = sg.unit % a.rblocks * kRows;
    const int rows = min(kRows, rows_all - r0);
    // ---- Q as right operands: row r is token (r0 + r) / G, head hkv * G + (r0 + r) % G.
    // Of 16 dims, 4 c + {0, 1} are where the product has 2 c + {0, 1}, and
    // 4 c + {2, 3} where it has 8 + 2 c + {0, 1}: as the bytes of K come.
    auto q_row = [&](int r) {
      const int rr = r0 + r;
      return a.q + (((int64_t)sg.b * a.q_len + rr / a.G) * a.q_rs +
                    (int64_t)(hkv * a.G + rr % a.G) * D) * 2;
    };
    uint32_t q[kQRegs ? NT : 1][kQRegs ? D / 16 : 1][2];
    float rf[NT][2];                    // what scores of rows 8 nt + 2 c + {0, 1} are multiplied by
    if constexpr (kQRegs) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + (lane >> 2);
        const bool in = r < rows && sg.len > 0;
        const char* p = q_row(in ? r : 0) + (lane & 3) * 8;
        uint2 raw[D / 16];
        float m = 0.0f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          raw[ks] = in ? *reinterpret_cast<const uint2*>(p + ks * 32) : make_uint2(0u, 0u);
          raw[ks].x ^= flip, raw[ks].y ^= flip;
          m = fmaxf(m, fmaxf(fabsf(__uint_as_float(raw[ks].x << 16)),
                             fabsf(__uint_as_float(raw[ks].x & 0xffff0000u))));
          m = fmaxf(m, fmaxf(fabsf(__uint_as_float(raw[ks].y << 16)),
                             fabsf(__uint_as_float(raw[ks].y & 0xffff0000u))));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float x;
        const float f = q_factor(m, x);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          rf[nt][i] = __shfl_sync(0xffffffffu, x, ((lane & 3) * 2 + i) * 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          q[nt][ks][0] = pack_f16x2(__uint_as_float(raw[ks].x << 16) * f,
                                    __uint_as_float(raw[ks].x & 0xffff0000u) * f);
          q[nt][ks][1] = pack_f16x2(__uint_as_float(raw[ks].y << 16) * f,
                                    __uint_as_float(raw[ks].y & 0xffff0000u) * f);
        }
      }
    } else {
      constexpr int kLanes = D / 8;     // of a row, 8 dims each
#pragma unroll 8
      for (int i = lane; i < kRows * kLanes; i += 32) {
        const int r = i / kLanes, u = i % kLanes;
        const bool in = r < rows && sg.len > 0;
        uint4 raw = in ? ldg16(q_row(r) + u * 16) : make_uint4(0u, 0u, 0u, 0u);
        raw.x ^= flip, raw.y ^= flip, raw.z ^= flip, raw.w ^= flip;
        float f[8];
        unpack16<__nv_bfloat16>(raw, f);
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
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) rf[nt][i] = row_x[warp][nt * 8 + (lane & 3) * 2 + i];
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) rf[nt][i] = fmaxf(ldexpf(sl2, (int)rf[nt][i]), 0x1p-126f);
    // positions that row 8 nt + 2 c + i sees
    auto seen = [&](int nt, int i) {
      const int r = nt * 8 + (lane & 3) * 2 + i;
      return r < rows ? sg.len - a.q_len + 1 + (r0 + r) / a.G : 0;
    };
    // Of rows 8 nt + 2 c + {0, 1}: the reference of scores with their value's power of two
    // (mv), the lane's sum, and the sums of values at dims 16 n + 2 (lane / 4) + {0, 1}:
    // o[nt][n][row + 2 dim]. Once `wide`, m is the maximum of the scores themselves, and l
    // is relative to it; before, l is relative to mv - kLift.
    float m[NT][2], mv[NT][2], l[NT][2], o[NT][D / 16][4];
    bool wide = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = mv[nt][0] = mv[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) o[nt][n][0] = o[nt][n][1] = o[nt][n][2] = o[nt][n][3] = 0.0f;
    }
    for (int j = sg.j0; j < sg.j1; ++j) {
      if (!wait_bar(&full[stage], phase, a.dev_err))
        return settle(full, stages, stage, phase, a.dev_err);
      const uint32_t kb = smem_addr(attn_dyn) + stage * 2 * half_stage + hl * D + off(p_warp);
      const uint32_t vb = kb + half_stage;
      const int cur = stage;
      const unsigned char* const tr = there[cur] + p_warp;
      const float2* const sc = scales[cur] + hl * tpos + p_warp + (lane >> 2);
      if (++stage == stages) stage = 0, phase ^= 1;
      // ---- scores of the warp's 32 positions, two tiles of 16: s[nt][g][row + 2 h] is that
      // of position 16 g + 8 h + lane / 4
      float s[NT][2][4] = {};
      const uint32_t step16 = off(16);
      const uint32_t ka = kb + off(lane & 15) + (lane >> 4) * 16;
#pragma unroll
      for (int d = 0; d < D / 16; d += 2)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t b[4];               // bytes 0-15: positions 0-7, 8-15; bytes 16-31: the same
          tc::ldmatrix4(b, ka + g * step16 + d * 16);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t kf[4];
            e4m3x4_to_f16(b[2 * t], kf[0], kf[2]);
            e4m3x4_to_f16(b[2 * t + 1], kf[1], kf[3]);
            if constexpr (kQRegs) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                tc::mma16h(s[nt][g], kf, q[nt][d + t][0], q[nt][d + t][1]);
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; nt += 2) {
                uint32_t qb[4];        // rows 0-7: k 0-7, 8-15; rows 8-15: the same
                tc::ldmatrix4(qb, smem_addr(sq) +
                                      (nt * 8 + (lane & 7) + ((lane >> 4) << 3)) * kQPitch +
                                      (d + t) * 32 + ((lane >> 3) & 1) * 16);
                tc::mma16h(s[nt][g], kf, qb[0], qb[1]);
                tc::mma16h(s[nt + 1][g], kf, qb[2], qb[3]);
              }
            }
          }
        }
      // the scales of the lane's four positions: 8 i + lane / 4
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = sc[8 * i];
        e[i] = f.y;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][i >> 1][(i & 1) * 2] *= f.x;
          s[nt][i >> 1][(i & 1) * 2 + 1] *= f.x;
        }
      }
      // ---- masks, references, weights
      const int pos0 = sg.base + j * tpos + p_warp;    // the first position
      // Draft tokens' positions are hidden from the rows before them by a weight of
      // zero, which a NaN among their values would get through: the rows that see such
      // values (`wild`) get a NaN, and they become zero.
      const int x0 = max(0, sg.len - a.q_len + 1 - pos0), x1 = min(32, sg.len - pos0);
      bool wild = false;
      if (__builtin_expect(x0 < x1, 0)) {
#pragma unroll 1
        for (int x = x0; x < x1; ++x)
#pragma unroll 1
          for (int i = lane; i < D / 4; i += 32)
            wild |= nan_bytes(lds32(vb + off(x) + i * 4)) != 0;
        wild = __any_sync(0xffffffffu, wild);
      }
      const uint4 all = *reinterpret_cast<const uint4*>(tr);
      const uint4 more = *reinterpret_cast<const uint4*>(tr + 16);
      if (__builtin_expect(pos0 + 31 > sg.len - a.q_len ||
                               (all.x & all.y & all.z & all.w & more.x & more.y & more.z &
                                more.w) != 0x01010101u, 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int sees = seen(nt, k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int x = 8 * i + (lane >> 2);
              if (!tr[x] || pos0 + x >= sees) s[nt][i >> 1][(i & 1) * 2 + k] = -INFINITY;
            }
          }
      }
      bool far = !mild[cur];
      // scores with their value's power of two, and whether one passes its reference too far
      bool rises = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& t = s[nt][i >> 1][(i & 1) * 2 + k];
            t = fmaf(t, rf[nt][k], e[i]);
            top = fmaxf(top, t);
          }
          rises = rises || top > mv[nt][k] + kSlack || (mv[nt][k] == -INFINITY && top > mv[nt][k]);
        }
      rises = __any_sync(0xffffffffu, rises);
      if (__builtin_expect(rises, 0)) {
        // The reference stands for the largest products with values, so it follows powers
        // of two that are the least ones of their rows. A tile that raises it is brought
        // into that form (lane l has position l; these are this warp's alone): a row of
        // zeros, or of the smallest bytes, under a large power of two would otherwise
        // raise it past the weights of all others.
        const uint32_t mine = vb + off(lane);
        const bool low = !row_full<D>(mine) && tr[lane];
        if (__any_sync(0xffffffffu, low)) {
          const float up = low ? fill_row(mine, D) : 0.0f;
          fence_proxy_async();        // before a later copy into the same place
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = __shfl_sync(0xffffffffu, up, 8 * i + (lane >> 2));
            e[i] -= x;
            far = far || fabsf(e[i]) > kMild;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              s[nt][i >> 1][(i & 1) * 2] -= x;
              s[nt][i >> 1][(i & 1) * 2 + 1] -= x;
            }
          }
          far = __any_sync(0xffffffffu, far);
        }
      }
      if (__builtin_expect(!wide && far, 0)) {
        wide = true;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            m[nt][k] = mv[nt][k];
            l[nt][k] *= exp2f(-kLift);
          }
      }
      if (__builtin_expect(rises, 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float corr[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = fmaxf(fmaxf(s[nt][0][k], s[nt][0][2 + k]), fmaxf(s[nt][1][k], s[nt][1][2 + k]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(mv[nt][k], top);
            corr[k] = mn == -INFINITY ? 1.0f : tc::ex2(mv[nt][k] - mn);
            mv[nt][k] = mn;
            if (!wide) l[nt][k] *= corr[k];
          }
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            o[nt][n][0] *= corr[0];
            o[nt][n][1] *= corr[1];
            o[nt][n][2] *= corr[0];
            o[nt][n][3] *= corr[1];
          }
        }
      }
      if (__builtin_expect(wide, 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = s[nt][i >> 1][(i & 1) * 2 + k] - e[i];
            float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m[nt][k], top), base = mn == -INFINITY ? 0.0f : mn;
            l[nt][k] = fmaf(l[nt][k], tc::ex2(m[nt][k] - base),
                            (tc::ex2(x[0] - base) + tc::ex2(x[1] - base)) +
                                (tc::ex2(x[2] - base) + tc::ex2(x[3] - base)));
            m[nt][k] = mn;
          }
      }
      uint32_t pt[NT][4];               // weights of positions 8 i .. 8 i + 7 as right operands
      float inv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) inv[i] = wide ? 0.0f : tc::ex2(-e[i]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float up[2] = {mv[nt][0] == -INFINITY ? 0.0f : mv[nt][0] - kLift,
                             mv[nt][1] == -INFINITY ? 0.0f : mv[nt][1] - kLift};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w0 = tc::ex2(s[nt][i >> 1][(i & 1) * 2] - up[0]),
                      w1 = tc::ex2(s[nt][i >> 1][(i & 1) * 2 + 1] - up[1]);
          if (!wide) {
            l[nt][0] = fmaf(w0, inv[i], l[nt][0]);
            l[nt][1] = fmaf(w1, inv[i], l[nt][1]);
          }
          pt[nt][i] = turn(pack_f16x2(w0, w1));
        }
      }
      if (__builtin_expect(wild, 0)) {
#pragma unroll 1
        for (int x = x0; x < x1; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (pos0 + x >= seen(nt, k)) continue;
#pragma unroll
              for (int n = 0; n < D / 16; ++n) {     // dims 16 n + 2 (lane / 4) + {0, 1}
                const uint32_t v = nan_bytes(lds32(vb + off(x) + n * 16 + (lane >> 3) * 4)) >>
                                   (lane >> 2 & 1) * 16;
                const float nan = __uint_as_float(0x7fc00000u);
                if (v & 0xffu) o[nt][n][k] = nan;
                if (v & 0xff00u) o[nt][n][2 + k] = nan;
              }
            }
        __syncwarp();
        // (these positions' values of this head are this warp's alone)
#pragma unroll 1
        for (int x = x0; x < x1; ++x)
          for (int i = lane; i < D / 4; i += 32) {
            const uint32_t v = lds32(vb + off(x) + i * 4);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(vb + off(x) + i * 4), "r"(v & ~nan_bytes(v))
                         : "memory");
          }
        fence_proxy_async();          // before a later copy into the same place
        __syncwarp();
      }
      // ---- weighted values: of 16 dims, the even ones are rows 0-7 of a left operand, the
      // odd ones rows 8-15
      const uint32_t va = vb + off(lane & 15) + (lane >> 4) * 16;
#pragma unroll
      for (int n = 0; n < D / 16; n += 2)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t b[4];               // dims 0-15: positions 0-7, 8-15; dims 16-31: the same
          tc::ldmatrix4_trans(b, va + g * step16 + n * 16);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t v[4];
            e4m3x4_to_f16(__byte_perm(b[2 * t], 0u, 0x3120), v[0], v[1]);
            e4m3x4_to_f16(__byte_perm(b[2 * t + 1], 0u, 0x3120), v[2], v[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              tc::mma16h(o[nt][n + t], v, pt[nt][2 * g], pt[nt][2 * g + 1]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[cur]);
    }
    // ---- the row sums over the lanes, and all in units of 2^m; then the warps of one head
    // join: those behind the head's first one leave their part in shared memory, in turn
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], d);
        if (!wide) {
          m[nt][k] = mv[nt][k];
          l[nt][k] *= exp2f(-kLift);
        }
        const float g = m[nt][k] == -INFINITY ? 1.0f : exp2f(mv[nt][k] - m[nt][k] - kLift);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          o[nt][n][k] *= g;
          o[nt][n][2 + k] *= g;
        }
      }
    const int per = kWarps >> hw_shift;              // warps of a head
    // (with Q in shared memory: every warp is done with its own)
    if (!kQRegs && per > 1 && !meet()) return settle(full, stages, stage, phase, a.dev_err);
#pragma unroll 1
    for (int w = 1; w < per; ++w) {
      float* const so = join + (warp / per) * (kRows * (D + 4));
      if (warp % per == w) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float* p = so + (nt * 8 + (lane & 3) * 2 + k) * (D + 4);
#pragma unroll
            for (int n = 0; n < D / 16; ++n)
              *reinterpret_cast<float2*>(p + n * 16 + (lane >> 2) * 2) =
                  make_float2(o[nt][n][k], o[nt][n][2 + k]);
            if (lane < 4) {
              p[D] = m[nt][k];
              p[D + 1] = l[nt][k];
            }
          }
      }
      if (!meet()) return settle(full, stages, stage, phase, a.dev_err);
      if (warp % per == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float* row = so + (nt * 8 + (lane & 3) * 2 + k) * (D + 4);
            const float mo = row[D], lo = row[D + 1];
            const float mm = fmaxf(m[nt][k], mo), base = mm == -INFINITY ? 0.0f : mm;
            const float g = tc::ex2(m[nt][k] - base), go = tc::ex2(mo - base);
            m[nt][k] = mm;
            l[nt][k] = fmaf(l[nt][k], g, lo * go);
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              const float2 v = *reinterpret_cast<const float2*>(row + n * 16 + (lane >> 2) * 2);
              o[nt][n][k] = fmaf(o[nt][n][k], g, v.x * go);
              o[nt][n][2 + k] = fmaf(o[nt][n][2 + k], g, v.y * go);
            }
          }
      }
      if (!meet()) return settle(full, stages, stage, phase, a.dev_err);
    }
    if (sg.len < 0 || warp % per != 0) continue;
    float* const part = attn_part<SHARED>(a, sg, D) + (warp / per) * kRows * (D + 2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = nt * 8 + (lane & 3) * 2 + k, c = (lane >> 2) * 2;
        if (r >= rows) continue;
        const float ll = l[nt][k], mn = m[nt][k] * 0.6931471805599453f;   // natural
        if (sg.whole) {
          const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
          const int64_t tok = (int64_t)sg.b * a.q_len + (r0 + r) / a.G;
          const int h = hkv * a.G + (r0 + r) % a.G;
          char* p = a.out + (tok * a.out_rs + (int64_t)h * D + c) * 2;
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
            *reinterpret_cast<uint32_t*>(p + n * 32) =
                pack_bf16x2(o[nt][n][k] * inv, o[nt][n][2 + k] * inv);
          if (a.lse && c == 0) a.lse[tok * a.Hq + h] = ll != 0.0f ? mn + logf(ll) : -INFINITY;
        } else {
          float* p = part + r * (D + 2);
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
            *reinterpret_cast<float2*>(p + n * 16 + c) = make_float2(o[nt][n][k], o[nt][n][2 + k]);
          if (c == 0) {
            p[D] = mn;
            p[D + 1] = ll;
          }
        }
      }
  }
}

static_assert(kTile == 32 * kWarps, "a warp takes 32 rows");

template <int D, int NT, bool SHARED>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t st) {
  // the ring, and behind it the joins (none with a head a warp) or the warps' Q
  const int tpos = kTile / a.hw, stage = 2 * (tpos * a.hw * D + (tpos >> a.group_shift) * 16);
  const int join = (a.hw == 4 ? 0 : a.hw) * NT * 8 * (D + 4) * 4;
  const int q = q_in_regs(D, NT) ? 0 : kWarps * NT * 8 * (D * 2 + 16);
  int stages = D == 64 ? 4 : 3;
  // as many as let the grid's blocks of an SM all be there (228 KB, less what the
  // kernel has besides)
  const int most = 228 * 1024 / attn_mma_blocks(D, NT * 8, true) - 8 * 1024;
  while (stages > 2 && stages * stage + std::max(join, q) > most) --stages;
  const int smem = stages * stage + std::max(join, q);
  static std::atomic<uint64_t> full;
  const void* const f = reinterpret_cast<const void*>(attn_mma_q8_kernel<D, NT, SHARED>);
  const cudaError_t e = mix_full_smem(f, full);
  if (e != cudaSuccess) return e;
  if constexpr (!SHARED) {
    attn_mma_q8_kernel<D, NT, SHARED><<<grid, kThreads, smem, st>>>(a, stages);
    return cudaGetLastError();
  } else {
    return attn_launch_beside(a.groups > 0, attn_mma_q8_kernel<D, NT, SHARED>, a, stages, grid,
                              kThreads, smem, st);
  }
}

template <int NT, bool SHARED>
cudaError_t launch_d(const AttnArgs& a, int D, int grid, cudaStream_t st) {
  return D == 64    ? launch<64, NT, SHARED>(a, grid, st)
         : D == 128 ? launch<128, NT, SHARED>(a, grid, st)
                    : launch<256, NT < 2 ? NT : 2, SHARED>(a, grid, st);   // (16 rows at most)
}
template <bool SHARED>
cudaError_t launch_rows(const AttnArgs& a, int D, int grid, cudaStream_t st) {
  return a.rows == 8    ? launch_d<1, SHARED>(a, D, grid, st)
         : a.rows == 16 ? launch_d<2, SHARED>(a, D, grid, st)
                        : launch_d<4, SHARED>(a, D, grid, st);
}

}  // namespace

cudaError_t attn_launch_mma_q8(const AttnArgs& a, int D, int grid, bool shared, cudaStream_t st) {
  return shared ? launch_rows<true>(a, D, grid, st) : launch_rows<false>(a, D, grid, st);
}

}  // namespace cconv
