// attn_decode in bf16: the same split as attn_decode.cuh, with the products on
// the warp-level tensor instruction (m16n8k16).
//
// What bounds it is the cache's bytes: K and V are read once for up to 32 query
// rows of a kv head (16 for heads of 256) together, and a row pair of 16 x 128 products per 256 bytes
// is far below any arithmetic limit. tcgen05 would need 64 rows or a transposed
// product to be fed; with 4 to 32 rows the warp-level form fits the rows as they
// are, keeps the softmax in the registers of the warp that made the scores, and
// the tensor pipe is mostly idle either way. More rows are taken in blocks, and
// each of them reads K and V again (64 rows of a kv head: twice, 281 us for 128
// requests of up to 8192 positions and one kv head where 32 rows take 158; heads of
// 256 with 32 rows, twice: 302 us for 60 requests and 2 kv heads).
//
// A block of 4 warps keeps a ring of tiles of K and V in shared memory, several
// tiles ahead. A tile is 64 rows: 64 / hw positions of hw kv heads, since the
// heads of a token lie side by side in the usual cache: a position then comes in
// one bulk copy of hw * D values (else in hw of D values), a copy a thread. The
// copies cost a handful of instructions a tile; the first form, per-thread
// 16-byte copies of swizzled rows, took two thirds of the kernel's instructions
// and held it at 4.2 TB/s. Where a position is less than 1 KB and the next one lies
// behind it in memory, a copy brings two or four. Copies are 16 bytes further
// apart than their length, so that ldmatrix meets no bank conflict, or one of two
// or four positions: with a copy a position the copies were what bounded small
// rows. Each warp takes 16 rows, of
// one head: scores = Q K^T, running maximum and sum of its own, weights to two
// bf16 terms in registers (the score layout of one product is the weight layout of
// the next), weighted values += P V. No barrier between warps but the ring's; warps
// of one head join their parts once per segment, through shared memory.
//
// Measured, heads of 128, 4 kv heads, 16 query heads: 256 requests of 1 to 8192
// positions (2.1 GB) 340 us, 6.2 TB/s; one of 131072 (270 MB) 57 us with its join;
// 64 requests of up to 4096 with 4 tokens each (0.25 GB) 57 us. With
// 2 kv heads, 256 requests (1.06 GB): 186 us, 5.7 TB/s; with a copy a position,
// and a ring that left the grid's second block of an SM no room, 354 us.
//
// V of positions that lie behind the length or on a bad page is filled with
// zeros; their scores are masked, as are those that a draft token's row does not
// see. A tile that every row sees whole skips the masks, and sums are rescaled
// only when a maximum has risen.
#include "attn_decode.cuh"
#include "tc.cuh"

#include <math.h>

namespace cconv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = (kWarps + 1) * 32;   // and one warp that loads
constexpr int kTile = 64;           // rows of a tile (positions x heads); 16 a warp

constexpr int kMaxStages = 4;
constexpr long long kWaitClocks = 4000000000LL;   // seconds; a copy takes microseconds

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Two weights as two bf16 terms, each pair packed (x0 low): 16 bits of them, so
// that the one rounding of a result is its last. With one term (331 us for the 256
// requests) the results were 2.1e-3 of their norm off instead of 1.7e-3. The first
// term is cut, not rounded: the second one then is not negative, and is kept above
// zero for a weight that is, since otherwise the terms' products with an infinite
// value would make NaN.
__device__ __forceinline__ float rest(float x) {
  const float r = x - __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  return fmaxf(r, fminf(x, 0x1p-126f));
}
__device__ __forceinline__ void split_weights(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
  lo = pack_bf16x2(rest(x0), rest(x1));
}
// All ones in the halves of a bf16 pair that are infinite or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((v & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
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
// behind the block's end: the last tiles of all places, those from `st` on in the
// phase of parity ph, those before it in the next one. (A place that no such tile
// came to: at once for the loading warp, whose phases are the last ones begun; for
// the others when its time is up. Waiting here at the loading warp's usual end, too,
// took 5 us of 340; it ends with copies on their way, which the others wait for.)
__device__ __noinline__ void settle(uint64_t* full, int stages, int st, int ph, int32_t* err) {
  for (int i = 0; i < stages; ++i) wait_bar(&full[i], i < st ? ph ^ 1 : ph, err);
  asm volatile("griddepcontrol.wait;" ::: "memory");    // (as after_prefix)
}

// The shared form starts beside the end of the kernel that takes the prefixes and
// needs nothing of it, but is not over before it: what follows joins both. (One block
// waits; block 0 always has a run.)
__device__ __forceinline__ void after_prefix() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// MT row tiles of 16. Q stays in registers where it fits beside the sums, else
// in shared memory.
template <int D, int MT, bool SHARED>
__global__ void __launch_bounds__(kThreads) attn_mma_kernel(const AttnArgs a, const int stages) {
  constexpr bool kQRegs = MT == 1;
  constexpr int kQPitch = D * 2 + 16;
  extern __shared__ __align__(128) unsigned char attn_dyn[];
  __shared__ int64_t scan[kThreads + 4];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], met;
  __shared__ __align__(16) unsigned char there[kMaxStages][kTile];   // positions that hold a token
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // position x of a tile lies at off(x) of its place: rows of a group side by side
  const int rowb = a.hw * D * 2, gs = a.group_shift, group = 1 << gs;
  auto off = [&](int x) { return (uint32_t)(x * rowb + (x >> gs) * 16); };
  const int hw_shift = a.hw == 4 ? 2 : a.hw >> 1, tpos = kTile >> hw_shift;   // positions a tile
  const uint32_t half_stage = off(tpos);        // K, then V
  // behind the ring: the joins of at most two heads, or the warps' own Q before
  unsigned char* const behind = attn_dyn + stages * 2 * half_stage;
  float* const join = reinterpret_cast<float*>(behind);
  unsigned char* const sq = behind + warp * (MT * 16 * kQPitch);
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], 1);
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
    unsigned char* const dst0 = attn_dyn + isv * half_stage + piece * (D * 2);
    const bool notes = isv == 0 && piece == 0;
    int st = 0, ph = 1;               // (the first round's places are free)
    while (run.p < run.end) {
      const AttnSeg s = attn_segment<SHARED>(a, tpos, run);
      attn_advance(a, s, run);
      const int32_t* tab = a.table + (int64_t)s.b * a.table_rs;
      const char* const src0 =
          (isv ? a.vc : a.kc) +
          ((int64_t)(s.unit / a.rblocks * a.hw) * a.s_head + piece * a.s_head) * 2;
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
              bulk_load(dst + skip * bytes,
                        src0 + (page * a.s_page + (tok + skip) * a.s_tok) * 2, n, &full[st]);
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
    if (SHARED && blockIdx.x == 0) after_prefix();
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
    const int hl = warp * 16 / tpos, hkv = sg.unit / a.rblocks * a.hw + hl;
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
      for (int i = lane; i < MT * 16 * (D / 8); i += 32) {
        const int r = i / (D / 8), u = i % (D / 8);
        const bool in = r < rows && sg.len > 0;
        *reinterpret_cast<uint4*>(sq + r * kQPitch + u * 16) =
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
      if (!wait_bar(&full[stage], phase, a.dev_err))
        return settle(full, stages, stage, phase, a.dev_err);
      const uint32_t kb = smem_addr(attn_dyn) + stage * 2 * half_stage + off(p0) + hl * (D * 2);
      const uint32_t vb = kb + half_stage;
      const unsigned char* tr = there[stage] + p0;
      uint64_t* const read = &empty[stage];
      if (++stage == stages) stage = 0, phase ^= 1;
      // ---- scores of the warp's 16 positions: two n-tiles of 8
      float s[MT][2][4] = {};
      const uint32_t ka =
          kb + off((lane & 7) + ((lane >> 4) << 3)) + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t b[4];                 // positions 0-7: k 0-7, k 8-15; positions 8-15: the same
        tc::ldmatrix4(b, ka + ks * 32);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if constexpr (kQRegs) {
            tc::mma16(s[mt][0], q[mt][ks], b[0], b[1]);
            tc::mma16(s[mt][1], q[mt][ks], b[2], b[3]);
          } else {
            uint32_t qa[4];
            tc::ldmatrix4(qa, smem_addr(sq) + (mt * 16 + (lane & 15)) * kQPitch + ks * 32 +
                         (lane >> 4) * 16);
            tc::mma16(s[mt][0], qa, b[0], b[1]);
            tc::mma16(s[mt][1], qa, b[2], b[3]);
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[mt][i >> 2][i & 3] *= sl2;
      // ---- masks, running maximum, weights
      const int pos0 = sg.base + j * tpos + p0;    // the warp's first position
      // Draft tokens' positions are hidden from the rows before them by a weight
      // of zero, which an infinity or NaN among their values would get through:
      // such values (`wild`) are kept out of the product and added to the rows
      // that see them.
      const int x0 = max(0, sg.len - a.q_len + 1 - pos0), x1 = min(16, sg.len - pos0);
      bool wild = false;
      if (x0 < x1) {
        for (int x = x0; x < x1; ++x)
          for (int i = lane; i < D / 2; i += 32)
            wild |= not_finite(lds32(vb + off(x) + i * 4)) != 0;
        wild = __any_sync(0xffffffffu, wild);
      }
      const uint4 all = *reinterpret_cast<const uint4*>(tr);
      if (pos0 + 15 > sg.len - a.q_len ||
          (all.x & all.y & all.z & all.w) != 0x01010101u) {
        const int q0 = (lane & 3) * 2;             // + 8 n + {0, 1}
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = mt * 16 + half * 8 + (lane >> 2);
            const int seen = r < rows ? sg.len - a.q_len + 1 + (r0 + r) / a.G : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int q = q0 + (i >> 1) * 8 + (i & 1);
              if (!tr[q] || pos0 + q >= seen) s[mt][i >> 1][half * 2 + (i & 1)] = -INFINITY;
            }
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t pw[4], pl[4];
        float corr[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float s0 = s[mt][0][half * 2], s1 = s[mt][0][half * 2 + 1],
                      s2 = s[mt][1][half * 2], s3 = s[mt][1][half * 2 + 1];
          float mx = fmaxf(fmaxf(s0, s1), fmaxf(s2, s3));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[mt][half], mx);
          const float base = mn == -INFINITY ? 0.0f : mn;
          corr[half] = tc::ex2(m[mt][half] - base);
          m[mt][half] = mn;
          const float x0 = tc::ex2(s0 - base), x1 = tc::ex2(s1 - base), x2 = tc::ex2(s2 - base),
                      x3 = tc::ex2(s3 - base);
          l[mt][half] = fmaf(l[mt][half], corr[half], (x0 + x1) + (x2 + x3));
          split_weights(x0, x1, pw[half], pl[half]);
          split_weights(x2, x3, pw[2 + half], pl[2 + half]);
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
        // ---- weighted values
        const uint32_t va = vb + off(lane & 15) + (lane >> 4) * 16;
        if (!wild) {
#pragma unroll
          for (int n = 0; n < D / 16; n += 2) {
            uint32_t b[4], c[4];       // dims 0-7: positions 0-7, 8-15; dims 8-15: the same
            tc::ldmatrix4_trans(b, va + n * 32);
            tc::ldmatrix4_trans(c, va + n * 32 + 32);
            tc::mma16(o[mt][2 * n], pw, b[0], b[1]);
            tc::mma16(o[mt][2 * n + 1], pw, b[2], b[3]);
            tc::mma16(o[mt][2 * n + 2], pw, c[0], c[1]);
            tc::mma16(o[mt][2 * n + 3], pw, c[2], c[3]);
            tc::mma16(o[mt][2 * n], pl, b[0], b[1]);
            tc::mma16(o[mt][2 * n + 1], pl, b[2], b[3]);
            tc::mma16(o[mt][2 * n + 2], pl, c[0], c[1]);
            tc::mma16(o[mt][2 * n + 3], pl, c[2], c[3]);
          }
        } else {
          const int q0 = (lane & 3) * 2;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            tc::ldmatrix4_trans(b, va + n * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {          // positions q0 + 8 (i & 1) + {0, 1}
              const int x = q0 + (i & 1) * 8;
              const uint32_t hidden = (x >= x0 ? 0xffffu : 0u) | (x + 1 >= x0 ? 0xffff0000u : 0u);
              b[i] &= ~(not_finite(b[i]) & hidden);
            }
            tc::mma16(o[mt][2 * n], pw, b[0], b[1]);
            tc::mma16(o[mt][2 * n + 1], pw, b[2], b[3]);
            tc::mma16(o[mt][2 * n], pl, b[0], b[1]);
            tc::mma16(o[mt][2 * n + 1], pl, b[2], b[3]);
          }
#pragma unroll 1
          for (int x = x0; x < x1; ++x)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int r = mt * 16 + half * 8 + (lane >> 2);
              if (r >= rows || pos0 + x >= sg.len - a.q_len + 1 + (r0 + r) / a.G) continue;
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                uint32_t v = lds32(vb + off(x) + (n * 8 + q0) * 2);
                v &= not_finite(v);
                o[mt][n][half * 2] += __uint_as_float(v << 16);
                o[mt][n][half * 2 + 1] += __uint_as_float(v & 0xffff0000u);
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(read);
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
        const int r = mt * 16 + half * 8 + (lane >> 2), c = (lane & 3) * 2;
        if (r >= rows) continue;
        const float ll = l[mt][half], mn = m[mt][half] * 0.6931471805599453f;   // natural
        if (sg.whole) {
          const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
          const int64_t tok = (int64_t)sg.b * a.q_len + (r0 + r) / a.G;
          const int h = hkv * a.G + (r0 + r) % a.G;
          char* p = a.out + (tok * a.out_rs + (int64_t)h * D + c) * 2;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<uint32_t*>(p + n * 16) =
                pack_bf16x2(o[mt][n][half * 2] * inv, o[mt][n][half * 2 + 1] * inv);
          if (a.lse && c == 0) a.lse[tok * a.Hq + h] = ll != 0.0f ? mn + logf(ll) : -INFINITY;
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
}

static_assert(kTile == 16 * kWarps, "a warp takes 16 rows");

template <int D, int MT, bool SHARED>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t st) {
  // the ring, and behind it the joins (none with a head a warp) or the warps' Q
  const int tpos = kTile / a.hw, stage = 2 * (tpos * a.hw * D * 2 + (tpos >> a.group_shift) * 16);
  const int join = (a.hw == 4 ? 0 : a.hw) * MT * 16 * (D + 4) * 4;
  const int q = MT == 1 ? 0 : kWarps * MT * 16 * (D * 2 + 16);
  int stages = D == 64 ? 4 : 3;
  // as many as let the grid's blocks of an SM all be there (228 KB, less what the
  // kernel has besides)
  const int most = 228 * 1024 / attn_mma_blocks(D, MT * 16, false) - 3 * 1024;
  while (stages > 2 && stages * stage + std::max(join, q) > most) --stages;
  const int smem = stages * stage + std::max(join, q);
  static std::atomic<uint64_t> full;
  const void* const f = reinterpret_cast<const void*>(attn_mma_kernel<D, MT, SHARED>);
  const cudaError_t e = mix_full_smem(f, full);
  if (e != cudaSuccess) return e;
  if constexpr (!SHARED) {
    attn_mma_kernel<D, MT, SHARED><<<grid, kThreads, smem, st>>>(a, stages);
    return cudaGetLastError();
  } else {
    return attn_launch_beside(a.groups > 0, attn_mma_kernel<D, MT, SHARED>, a, stages, grid,
                              kThreads, smem, st);
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

cudaError_t attn_launch_mma(const AttnArgs& a, int D, int grid, bool shared, cudaStream_t st) {
  return shared ? launch_d<true>(a, D, grid, st) : launch_d<false>(a, D, grid, st);
}

}  // namespace cconv
