// Chunked gated delta rule on the tensor cores (bf16, heads of 128 x 128): the
// long sequences of gdn_fwd_varlen.
//
// With the tokens of a chunk of C = 64 and G_i the sum of their log decays up
// to i, the recurrence S_i = a_i S_{i-1} + b_i k_i (v_i - a_i S_{i-1}^T k_i)^T is
//   A_ij = b_i e^{G_i - G_j} k_i.k_j  (j < i),   T = (I + A)^-1,
//   R_i  = b_i (v_i - e^{G_i} S^T k_i),          N = T R,
//   o_i  = scale (e^{G_i} S^T q_i + sum_{j<=i} e^{G_i - G_j} (q_i.k_j) N_j),
//   S'   = e^{G_C} S + sum_j e^{G_C - G_j} k_j N_j^T,
// one chain of chunks per sequence and head. A block owns one chain. Everything
// that does not need S -- gates, norms, A, T, q.k -- is worked out one chunk
// ahead by four warps, so that the chain itself is four tensor products and
// the element-wise work between them.
//
// Orientation. All products with S are taken transposed, with the 128 columns
// of S (dv) as the M rows of the tensor-core instruction and the tokens (or dk)
// as N: S^T, R^T and N^T are then A operands, which tcgen05 reads from tensor
// memory, lane = column of S; a thread owns one column, writes its row of the
// operand there and never passes it through shared memory. The B operands are
// the staged tiles themselves: K and Q (rows = tokens) for S^T k and S^T q, the
// same K tile read along its other dimension for the state update, T and the
// scores for the two products inside the chunk.
//
// Precision. k, q and v are bf16 and exact. fp32 factors (S, R, T, N) enter as
// sums of two bf16 terms (about 16 bits; products lo * lo are left out), since
// the state must keep more than 8 bits over thousands of tokens: its error is
// 4e-6 of its norm against 64 bits where single bf16 factors give 2e-3. The
// two products that only feed the output, which is rounded to bf16 itself,
// take one term (2e-3). S is held in fp32 registers from the first chunk to
// the last. l2 norms enter as factors of the rows, so that raw rows are
// multiplied. G is kept as whole part + remainder (in powers of two): chunks
// with strong decays reach sums of several hundred, whose differences fp32
// alone would round by 1e-5.
//
// T is built by forward substitution of the two 32 x 32 diagonal blocks
// (a thread a column) and one block step for the rest, all in fp32: stable for
// any keys, unlike sums of powers of A, whose terms cancel for equal keys.
//
// Layout. K and Q of a chunk form one 128-row tile in the 128-byte swizzle (two
// panels of 64 dk each); rows behind the sequence's end are filled with zeros
// by the copies themselves (cp.async), so nothing of the neighbouring request
// -- NaN, say -- enters a product. Tensor memory columns: S (hi, lo by halves
// of dk; the state update's accumulator takes the same columns once S has been
// read) 0-127, S^T k 128-191 (then N), S^T q 192-255, R then the decayed N
// (hi, lo) 256-319, N 320-351, in-chunk output 352-415, [K; Q] K^T 416-479.
#include <stddef.h>

#include "gdn.cuh"
#include "tc.cuh"

namespace cconv {
namespace {

constexpr int kC = 64;                       // tokens of a chunk
constexpr int kD = 128;                      // dk = dv
constexpr int kStages = 3;
constexpr int kScanWarps = 8, kPrepWarps = 4;
constexpr int kWarpPrep0 = kScanWarps, kWarpMma = kWarpPrep0 + kPrepWarps,
              kWarpLoad = kWarpMma + 1;
constexpr int kThreadsC = (kWarpLoad + 1) * 32;

constexpr uint32_t kPanel = 128 * 128;       // 64 dk of [K; Q]: 128 rows x 128 bytes
constexpr uint32_t kKQBytes = 2 * kPanel;
constexpr uint32_t kVBytes = kC * kD * 2;
constexpr uint32_t kStageBytes = kKQBytes + kVBytes;
constexpr uint32_t kTBytes = kC * kC * 2;    // one 64 x 64 bf16 operand
constexpr uint32_t kTP = 3 * kTBytes;        // T hi, T lo, scores
constexpr int kAPitch = 68;                  // fp32 rows of A (16-byte aligned)

constexpr uint32_t kColS = 0, kColKS = 128, kColQS = 192, kColR = 256, kColN = 320, kColO = 352,
                   kColD1 = 416;

// A wait that has run out of this many clocks (seconds) gives the block up.
constexpr long long kWaitClocks = 4000000000LL;

struct alignas(16) Gates {   // read four at a time
  float rb[kC];      // beta
  float rc[kC];      // beta e^G / |k|
  float vd[kC];      // e^{G_C - G} / |k|
  float o1[kC];      // scale e^G / |q|
  float o2[kC];      // scale / |q|
  float ec;          // e^{G_C}
};

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t d1_full, g_full, t_full, tp_empty[2], arr_empty[2];
  uint64_t s_full, ks_full, qs_done, r_full, vn_full, vd_full, sd_full, o_full, o_empty, fin;
  uint32_t tmem;
  volatile int abort;
};

struct Smem {
  unsigned char stage[kStages][kStageBytes];   // 1024-byte aligned
  unsigned char tp[2][kTP];
  alignas(16) float A[kC][kAPitch];
  alignas(16) float X[32][36];            // A21 T11 of the block step
  Gates gates[2];
  alignas(16) float rk[kC];
  alignas(16) float g_hi[kC];
  alignas(16) float g_lo[kC];
  Ctl ctl;
};
static_assert(offsetof(Smem, tp) % 1024 == 0 && kStageBytes % 1024 == 0 && kTP % 1024 == 0 &&
                  kTBytes % 1024 == 0,
              "swizzled tiles start on 1024 bytes");
static_assert(sizeof(Gates) % 16 == 0 && offsetof(Smem, A) % 16 == 0 &&
                  offsetof(Smem, X) % 16 == 0 && offsetof(Smem, gates) % 16 == 0 &&
                  offsetof(Smem, rk) % 16 == 0 && offsetof(Smem, g_hi) % 16 == 0 &&
                  offsetof(Smem, g_lo) % 16 == 0 && offsetof(Smem, ctl) % 8 == 0,
              "16-byte accesses");

__device__ __forceinline__ uint32_t sw128(int row, int unit) {
  return (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
}

struct Wait {
  Ctl* ctl;
  int32_t* err;
  // Called by whole warps. False when the block is giving up.
  __device__ __forceinline__ bool operator()(uint64_t* bar, int phase) const {
    const bool done = mbar_try(bar, phase & 1);
    if (__any_sync(0xffffffffu, done)) return true;
    return loop(bar, phase & 1);
  }
  __device__ __noinline__ bool loop(uint64_t* bar, uint32_t parity) const {
    const long long t0 = clock64();
    for (uint32_t it = 0;; ++it) {
      if (__any_sync(0xffffffffu, mbar_try(bar, parity))) return true;
      if ((it & 63u) == 63u) {
        if (__any_sync(0xffffffffu, ctl->abort != 0)) return false;
        if (__any_sync(0xffffffffu, clock64() - t0 > kWaitClocks)) {
          ctl->abort = 1;
          if ((threadIdx.x & 31) == 0) flag_error(err, CCONV_DERR_TIMEOUT);
          return false;
        }
      }
    }
  }
};

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void prep_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kPrepWarps * 32) : "memory");
}

// ---- the warps that look one chunk ahead ----------------------------------

// Gates, norms, A, T and scores of every chunk. Thread p < 64 holds row p of
// K K^T and token p's gates, thread 64 + p row p of Q K^T.
__device__ __forceinline__ void prep_role(const GdnArgs& a, Smem& sm, const Wait& wait, int row0,
                                          int len, int h, int chunks, uint32_t tmem) {
  const int p = threadIdx.x - kWarpPrep0 * 32, lane = p & 31, warp = p >> 5;
  const bool is_k = p < kC;
  const int r = is_k ? p : p - kC;               // the thread's row
  const float A_log2 = -expf(a.A_log[h]) * 1.4426950408889634f;
  const float dtb = a.dt_bias[h];
  const __nv_bfloat16* ga = reinterpret_cast<const __nv_bfloat16*>(a.a) + h;
  const __nv_bfloat16* gb = reinterpret_cast<const __nv_bfloat16*>(a.b) + h;
  float na = 0.0f, nb = 0.0f;                    // the next chunk's gate inputs
  if (is_k && r < len) {
    na = elem(ga, (int64_t)(row0 + r) * a.a_rs);
    nb = elem(gb, (int64_t)(row0 + r) * a.b_rs);
  }
  for (int n = 0; n < chunks; ++n) {
    const int st = n % kStages, bf = n & 1;
    const int left = len - n * kC;                // tokens of this chunk (>= 64: whole)
    Gates& G = sm.gates[bf];
    // ---- gates (64 threads: two warps scan 64 tokens)
    double g = 0.0;
    float beta = 0.0f;
    if (is_k && r < left) {
      const float x = na + dtb;
      const float d = A_log2 * (fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))));
      // a decay below 2^-150 is zero in fp32 whatever follows (a NaN stays one)
      g = (double)(d < -150.0f ? -150.0f : d);
      beta = gdn_beta(nb);
    }
    if (is_k && left - kC > r) {
      na = elem(ga, (int64_t)(row0 + (n + 1) * kC + r) * a.a_rs);
      nb = elem(gb, (int64_t)(row0 + (n + 1) * kC + r) * a.b_rs);
    }
    if (warp < 2) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, g, d);
        if (lane >= d) g += o;
      }
      if (p == 31) {      // the first warp's sum, for the second one
        const double w = trunc(g);
        sm.X[0][0] = (float)w;
        sm.X[0][1] = (float)(g - w);
      }
    }
    // ---- the row's sum of squares
    if (!wait(&sm.ctl.full[st], n / kStages)) return;
    float ss = 0.0f;
    {
      const unsigned char* base = sm.stage[st];
      const int row = is_k ? r : kC + r;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        float f[8];
        unpack16<__nv_bfloat16>(
            *reinterpret_cast<const uint4*>(base + (u >> 3) * kPanel + sw128(row, u & 7)), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
      }
    }
    const float rn = a.l2norm ? 1.0f / sqrtf(ss + kGdnNormEps) : 1.0f;
    // the arrays of two chunks ago have been read
    if (n >= 2 && !wait(&sm.ctl.arr_empty[bf], (n >> 1) - 1)) return;
    prep_sync();
    if (is_k) {
      if (warp == 1) g += (double)sm.X[0][0] + (double)sm.X[0][1];
      const double w = trunc(g);
      sm.g_hi[r] = (float)w;
      sm.g_lo[r] = (float)(g - w);
      sm.rk[r] = rn;
      const float eg = exp2f((float)g);
      G.rb[r] = beta;
      G.rc[r] = beta * eg * rn;
    } else {
      G.o2[r] = a.scale * rn;
    }
    prep_sync();
    const float hi = sm.g_hi[r], lo = sm.g_lo[r];
    if (is_k)
      G.vd[r] = rn * exp2f((sm.g_hi[kC - 1] - hi) + (sm.g_lo[kC - 1] - lo));
    else
      G.o1[r] = a.scale * rn * exp2f(hi + lo);
    if (p == 0) G.ec = exp2f(sm.g_hi[kC - 1] + sm.g_lo[kC - 1]);
    warp_arrive(&sm.ctl.g_full);
    // ---- A and the scores from [K; Q] K^T
    if (!wait(&sm.ctl.d1_full, n)) return;
    tc::fence_after();
    if (n >= 2 && !wait(&sm.ctl.tp_empty[bf], (n >> 1) - 1)) return;
    unsigned char* const tp = sm.tp[bf];
    const uint32_t d1 = tmem + kColD1 + ((uint32_t)(warp * 32) << 16);
    const float fac = is_k ? beta * rn : 1.0f;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t x[32];
      tc::ld32(d1 + hf * 32, x);
      tc::wait_ld(x);
      float y[32];
#pragma unroll
      for (int j4 = 0; j4 < 8; ++j4) {
        const int j = hf * 32 + j4 * 4;
        const float4 rk4 = *reinterpret_cast<const float4*>(&sm.rk[j]);
        const float4 h4 = *reinterpret_cast<const float4*>(&sm.g_hi[j]);
        const float4 l4 = *reinterpret_cast<const float4*>(&sm.g_lo[j]);
        const float rkv[4] = {rk4.x, rk4.y, rk4.z, rk4.w}, hv[4] = {h4.x, h4.y, h4.z, h4.w},
                    lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int jj = j + e;
          const bool in = is_k ? jj < r : jj <= r;
          const float d = in ? exp2f((hi - hv[e]) + (lo - lv[e])) : 0.0f;
          y[j4 * 4 + e] = in ? fac * rkv[e] * d * __uint_as_float(x[j4 * 4 + e]) : 0.0f;
        }
      }
      if (is_k) {
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4)
          *reinterpret_cast<float4*>(&sm.A[r][hf * 32 + j4 * 4]) =
              make_float4(y[j4 * 4], y[j4 * 4 + 1], y[j4 * 4 + 2], y[j4 * 4 + 3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(tp + 2 * kTBytes + sw128(r, hf * 4 + u)) =
              make_uint4(pack_bf16x2(y[u * 8], y[u * 8 + 1]),
                         pack_bf16x2(y[u * 8 + 2], y[u * 8 + 3]),
                         pack_bf16x2(y[u * 8 + 4], y[u * 8 + 5]),
                         pack_bf16x2(y[u * 8 + 6], y[u * 8 + 7]));
      }
    }
    tc::fence_before();
    prep_sync();
    // ---- T: diagonal blocks (warps 0 and 1, a thread a column), stored as bf16
    // hi and lo; fp32 copies for the block step stay in A's own blocks
    auto put = [&](int i, int j, float v) {
      const uint32_t at = sw128(i, j >> 3) + (j & 7) * 2;
      const uint32_t hb = pack_bf16x2(v, 0.0f);
      *reinterpret_cast<uint16_t*>(tp + at) = (uint16_t)hb;
      *reinterpret_cast<uint16_t*>(tp + kTBytes + at) =
          (uint16_t)pack_bf16x2(v - __uint_as_float(hb << 16), 0.0f);
    };
    if (warp < 2) {
      const int b0 = warp * 32;
      float t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float acc[4] = {lane == i ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k4 = 0; k4 < i; k4 += 4) {
          const float4 v = *reinterpret_cast<const float4*>(&sm.A[b0 + i][b0 + k4]);
          acc[0] = fmaf(-v.x, t[k4], acc[0]);
          if (k4 + 1 < i) acc[1] = fmaf(-v.y, t[k4 + 1], acc[1]);
          if (k4 + 2 < i) acc[2] = fmaf(-v.z, t[k4 + 2], acc[2]);
          if (k4 + 3 < i) acc[3] = fmaf(-v.w, t[k4 + 3], acc[3]);
        }
        t[i] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        sm.A[b0 + i][b0 + lane] = t[i];
        put(b0 + i, b0 + lane, t[i]);
      }
    }
    prep_sync();
    // ---- T21 = -T22 (A21 T11): 8 outputs a thread, 2 rows x 4 columns
    {
      const int i0 = (p >> 3) * 2, j0 = (p & 7) * 4;
      float x[2][4] = {};
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float4 t = *reinterpret_cast<const float4*>(&sm.A[k][j0]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = sm.A[32 + i0 + e][k];
          x[e][0] = fmaf(v, t.x, x[e][0]);
          x[e][1] = fmaf(v, t.y, x[e][1]);
          x[e][2] = fmaf(v, t.z, x[e][2]);
          x[e][3] = fmaf(v, t.w, x[e][3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float4*>(&sm.X[i0 + e][j0]) =
            make_float4(x[e][0], x[e][1], x[e][2], x[e][3]);
      prep_sync();
      float y[2][4] = {};
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float4 t = *reinterpret_cast<const float4*>(&sm.X[k][j0]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = -sm.A[32 + i0 + e][32 + k];
          y[e][0] = fmaf(v, t.x, y[e][0]);
          y[e][1] = fmaf(v, t.y, y[e][1]);
          y[e][2] = fmaf(v, t.z, y[e][2]);
          y[e][3] = fmaf(v, t.w, y[e][3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t h0, h1, l0, l1;
        tc::split2(y[e][0], y[e][1], h0, l0);
        tc::split2(y[e][2], y[e][3], h1, l1);
        const uint32_t at = sw128(32 + i0 + e, j0 >> 3) + (j0 & 7) * 2;
        *reinterpret_cast<uint2*>(tp + at) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(tp + kTBytes + at) = make_uint2(l0, l1);
      }
    }
    fence_proxy_async();
    warp_arrive(&sm.ctl.t_full);
    prep_sync();     // X and A are free for the next chunk
  }
}

// ---- the warps on the chain -------------------------------------------------

template <typename ST>
__device__ __forceinline__ void scan_role(const GdnArgs& a, Smem& sm, const Wait& wait, int row0,
                                          int len, int h, int chunks, uint32_t tmem, bool init,
                                          int slot) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qd = warp & 3, hf = warp >> 2;
  const int col = qd * 32 + lane;                       // the thread's column of S
  const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
  ST* const sp = reinterpret_cast<ST*>(a.st) + (int64_t)(slot < 0 ? 0 : slot) * a.st_slot +
                 (int64_t)h * a.st_head + (int64_t)hf * 64 * kD + col;
  float S[64];                                          // dk hf * 64 + [0, 64)
#pragma unroll
  for (int i = 0; i < 64; ++i) S[i] = init ? elem(sp, i * kD) : 0.0f;
  __nv_bfloat16* const op = reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)h * kD + col;

  // outputs of chunk n
  auto outputs = [&](int n) -> bool {
    if (!wait(&sm.ctl.o_full, n)) return false;
    tc::fence_after();
    uint32_t x[32], y[32];
    tc::ld32(tl + kColQS + hf * 32, x);
    tc::ld32(tl + kColO + hf * 32, y);
    tc::wait_ld(x);
    tc::wait_ld(y);
    tc::fence_before();
    warp_arrive(&sm.ctl.o_empty);
    const Gates& G = sm.gates[n & 1];
    const int t0 = n * kC + hf * 32;
    __nv_bfloat16* o = op + (int64_t)(row0 + t0) * a.out_rs;
#pragma unroll
    for (int i4 = 0; i4 < 8; ++i4) {
      const float4 c1 = *reinterpret_cast<const float4*>(&G.o1[hf * 32 + i4 * 4]);
      const float4 c2 = *reinterpret_cast<const float4*>(&G.o2[hf * 32 + i4 * 4]);
      const float u[4] = {c1.x, c1.y, c1.z, c1.w}, w[4] = {c2.x, c2.y, c2.z, c2.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i4 * 4 + e;
        const float v = fmaf(u[e], __uint_as_float(x[i]), w[e] * __uint_as_float(y[i]));
        if (t0 + i < len) o[(int64_t)i * a.out_rs] = __float2bfloat16_rn(v);
      }
    }
    warp_arrive(&sm.ctl.arr_empty[n & 1]);
    return true;
  };
  // S = e^{G_C} S + update of chunk n
  auto advance = [&](int n, int part) {
    uint32_t x[32];
    tc::ld32(tl + kColS + hf * 64 + part * 32, x);
    tc::wait_ld(x);
    const float ec = sm.gates[n & 1].ec;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      S[part * 32 + i] = fmaf(ec, S[part * 32 + i], __uint_as_float(x[i]));
  };

  for (int n = 0; n < chunks; ++n) {
    const int st = n % kStages, bf = n & 1;
    // ---- S: add the last chunk's update, split, hand to the tensor cores
    if (n > 0) {
      if (!wait(&sm.ctl.sd_full, n - 1)) return;
      tc::fence_after();
      advance(n - 1, 0);
      advance(n - 1, 1);
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        tc::split2(S[part * 32 + 2 * i], S[part * 32 + 2 * i + 1], hi[i], lo[i]);
      tc::st16(tl + kColS + hf * 64 + part * 16, hi);
      tc::st16(tl + kColS + hf * 64 + 32 + part * 16, lo);
    }
    tc::wait_st();
    tc::fence_before();
    warp_arrive(&sm.ctl.s_full);
    if (n > 0 && !outputs(n - 1)) return;
    // ---- R
    if (!wait(&sm.ctl.g_full, n) || !wait(&sm.ctl.full[st], n / kStages) ||
        !wait(&sm.ctl.ks_full, n))
      return;
    tc::fence_after();
    const Gates& G = sm.gates[bf];
    {
      uint32_t x[32], hi[16], lo[16];
      tc::ld32(tl + kColKS + hf * 32, x);
      tc::wait_ld(x);
      const uint16_t* v = reinterpret_cast<const uint16_t*>(sm.stage[st] + kKQBytes) +
                          hf * 32 * kD + col;
#pragma unroll
      for (int i4 = 0; i4 < 8; ++i4) {
        const float4 b4 = *reinterpret_cast<const float4*>(&G.rb[hf * 32 + i4 * 4]);
        const float4 c4 = *reinterpret_cast<const float4*>(&G.rc[hf * 32 + i4 * 4]);
        const float b[4] = {b4.x, b4.y, b4.z, b4.w}, c[4] = {c4.x, c4.y, c4.z, c4.w};
        float r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float vv = __uint_as_float((uint32_t)v[(i4 * 4 + e) * kD] << 16);
          r[e] = fmaf(-c[e], __uint_as_float(x[i4 * 4 + e]), b[e] * vv);
        }
        tc::split2(r[0], r[1], hi[i4 * 2], lo[i4 * 2]);
        tc::split2(r[2], r[3], hi[i4 * 2 + 1], lo[i4 * 2 + 1]);
      }
      tc::st16(tl + kColR + hf * 16, hi);
      tc::st16(tl + kColR + 32 + hf * 16, lo);
    }
    tc::wait_st();
    tc::fence_before();
    warp_arrive(&sm.ctl.r_full);
    // ---- N
    if (!wait(&sm.ctl.vn_full, n)) return;
    tc::fence_after();
    {
      uint32_t x[32], hi[16], lo[16], on[16];
      tc::ld32(tl + kColKS + hf * 32, x);
      tc::wait_ld(x);
#pragma unroll
      for (int i4 = 0; i4 < 8; ++i4) {
        const float4 d4 = *reinterpret_cast<const float4*>(&G.vd[hf * 32 + i4 * 4]);
        const float v0 = __uint_as_float(x[i4 * 4]), v1 = __uint_as_float(x[i4 * 4 + 1]),
                    v2 = __uint_as_float(x[i4 * 4 + 2]), v3 = __uint_as_float(x[i4 * 4 + 3]);
        on[i4 * 2] = pack_bf16x2(v0, v1);
        on[i4 * 2 + 1] = pack_bf16x2(v2, v3);
        tc::split2(d4.x * v0, d4.y * v1, hi[i4 * 2], lo[i4 * 2]);
        tc::split2(d4.z * v2, d4.w * v3, hi[i4 * 2 + 1], lo[i4 * 2 + 1]);
      }
      tc::st16(tl + kColR + hf * 16, hi);
      tc::st16(tl + kColR + 32 + hf * 16, lo);
      tc::st16(tl + kColN + hf * 16, on);
    }
    tc::wait_st();
    tc::fence_before();
    warp_arrive(&sm.ctl.vd_full);
  }
  if (!wait(&sm.ctl.sd_full, chunks - 1)) return;
  tc::fence_after();
  advance(chunks - 1, 0);
  advance(chunks - 1, 1);
  if (slot >= 0)
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      const auto raw = f32_to_raw<ST>(S[i]);
      *reinterpret_cast<std::remove_const_t<decltype(raw)>*>(sp + i * kD) = raw;
    }
  outputs(chunks - 1);
}

// ---- the warp that issues the tensor products -------------------------------

__device__ __forceinline__ void mma_role(Smem& sm, const Wait& wait, int chunks, uint32_t tmem) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kId64 = tc::idesc(128, 64), kIdUpd = tc::idesc(128, 128, true);
  auto panel = [&](int st, int ks, int row) {   // 16 dk of rows [row, ..) of [K; Q]
    return smem_addr(sm.stage[st]) + (ks >> 2) * kPanel + (ks & 3) * 32 + row * 128;
  };
  auto scores = [&](int n) -> bool {            // [K; Q] K^T of chunk n
    const int st = n % kStages;
    if (!wait(&sm.ctl.full[st], n / kStages)) return false;
    tc::fence_after();
    if (lane == 0) {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint64_t d = tc::desc_sw128(panel(st, ks, 0), 16);
        tc::mma_ss(tmem + kColD1, d, d, kId64, ks > 0);
      }
      tc::commit(&sm.ctl.d1_full);
    }
    __syncwarp();
    return true;
  };
  if (!scores(0)) return;
  for (int n = 0; n < chunks; ++n) {
    const int st = n % kStages, bf = n & 1;
    const uint32_t tp = smem_addr(sm.tp[bf]);
    if (!wait(&sm.ctl.s_full, n)) return;
    tc::fence_after();
    if (lane == 0) {
#pragma unroll
      for (int t = 0; t < 2; ++t)               // S hi, S lo
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc::mma_ts(tmem + kColKS, tmem + kColS + (ks >> 2) * 64 + t * 32 + (ks & 3) * 8,
                     tc::desc_sw128(panel(st, ks, 0), 16), kId64, (t | ks) > 0);
      tc::commit(&sm.ctl.ks_full);
    }
    __syncwarp();
    if (n > 0 && !wait(&sm.ctl.o_empty, n - 1)) return;
    tc::fence_after();
    if (lane == 0) {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        tc::mma_ts(tmem + kColQS, tmem + kColS + (ks >> 2) * 64 + (ks & 3) * 8,
                   tc::desc_sw128(panel(st, ks, kC), 16), kId64, ks > 0);
      tc::commit(&sm.ctl.qs_done);
    }
    __syncwarp();
    if (!wait(&sm.ctl.r_full, n) || !wait(&sm.ctl.t_full, n)) return;
    tc::fence_after();
    if (lane == 0) {
#pragma unroll
      for (int t = 0; t < 3; ++t)               // R hi T hi, R lo T hi, R hi T lo
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc::mma_ts(tmem + kColKS, tmem + kColR + (t == 1 ? 32 : 0) + ks * 8,
                     tc::desc_sw128(tp + (t == 2 ? kTBytes : 0) + ks * 32, 16), kId64,
                     (t | ks) > 0);
      tc::commit(&sm.ctl.vn_full);
    }
    __syncwarp();
    if (n + 1 < chunks && !scores(n + 1)) return;
    if (!wait(&sm.ctl.vd_full, n) || !wait(&sm.ctl.qs_done, n)) return;
    tc::fence_after();
    if (lane == 0) {
#pragma unroll
      for (int t = 0; t < 2; ++t)               // K read along dk: 16 tokens a step
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc::mma_ts(tmem + kColS, tmem + kColR + t * 32 + ks * 8,
                     tc::desc_sw128(smem_addr(sm.stage[st]) + ks * 2048, kPanel), kIdUpd,
                     (t | ks) > 0);
      tc::commit(&sm.ctl.sd_full);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        tc::mma_ts(tmem + kColO, tmem + kColN + ks * 8,
                   tc::desc_sw128(tp + 2 * kTBytes + ks * 32, 16), kId64, ks > 0);
      tc::commit(&sm.ctl.o_full);
      tc::commit(&sm.ctl.empty[st]);
      tc::commit(&sm.ctl.tp_empty[bf]);
    }
    __syncwarp();
  }
}

// ---- the warp that stages K, Q and V ----------------------------------------

__device__ __forceinline__ void load_role(const GdnArgs& a, Smem& sm, const Wait& wait, int row0,
                                          int len, int h, int chunks) {
  const int lane = threadIdx.x & 31, u = lane & 15, r2 = lane >> 4;
  const int hk = h / (a.Hv / a.Hk);
  const char* kp = a.k + ((int64_t)row0 * a.k_rs + (int64_t)hk * kD) * 2 + u * 16;
  const char* qp = a.q + ((int64_t)row0 * a.q_rs + (int64_t)hk * kD) * 2 + u * 16;
  const char* vp = a.v + ((int64_t)row0 * a.v_rs + (int64_t)h * kD) * 2 + u * 16;
  for (int n = 0; n < chunks; ++n) {
    const int st = n % kStages;
    if (n >= kStages && !wait(&sm.ctl.empty[st], n / kStages - 1)) break;
    const uint32_t base = smem_addr(sm.stage[st]) + (u >> 3) * kPanel;
    const uint32_t vbase = smem_addr(sm.stage[st]) + kKQBytes + u * 16;
#pragma unroll 8
    for (int i = 0; i < kC / 2; ++i) {
      const int r = i * 2 + r2;
      const int64_t t = (int64_t)n * kC + r;
      const bool in = t < len;
      const int64_t tt = in ? t : 0;
      cp_async16(base + sw128(r, u & 7), kp + tt * a.k_rs * 2, in);
      cp_async16(base + sw128(kC + r, u & 7), qp + tt * a.q_rs * 2, in);
      cp_async16(vbase + r * (kD * 2), vp + tt * a.v_rs * 2, in);
    }
    cp_async_commit();
    if (n > 0) {
      cp_async_wait<1>();
      fence_proxy_async();
      warp_arrive(&sm.ctl.full[(n - 1) % kStages]);
    }
  }
  cp_async_wait<0>();      // also when giving up: nothing lands after the block ends
  fence_proxy_async();
  warp_arrive(&sm.ctl.full[(chunks - 1) % kStages]);
}

template <typename ST>
__global__ void __launch_bounds__(kThreadsC, 1) gdn_chunk_kernel(const GdnArgs a) {
  extern __shared__ __align__(1024) unsigned char gdn_dyn[];
  Smem& sm = *reinterpret_cast<Smem*>(
      gdn_dyn + ((1024u - (smem_addr(gdn_dyn) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5;
  const int h = blockIdx.x % a.Hv, s = blockIdx.x / a.Hv;
  // sequences that the recurrent kernel skips with an error are skipped there
  int row0, len;
  if (!gdn_bounds(a, s, row0, len) || len <= a.max_len) return;
  const int slot = a.state_idx[s];
  if (slot >= a.num_slots) {
    if (h == 0 && tid == 0) flag_error(a.dev_err, CCONV_DERR_SLOT_RANGE);
    return;
  }
  const bool init = slot >= 0 && (!a.has_init || a.has_init[s]);
  const int chunks = (len + kC - 1) / kC;

  if (tid == 0) {
    Ctl& c = sm.ctl;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.tp_empty[i], 1);
      mbar_init(&c.arr_empty[i], kScanWarps);
    }
    mbar_init(&c.d1_full, 1);
    mbar_init(&c.g_full, kPrepWarps);
    mbar_init(&c.t_full, kPrepWarps);
    mbar_init(&c.s_full, kScanWarps);
    mbar_init(&c.ks_full, 1);
    mbar_init(&c.qs_done, 1);
    mbar_init(&c.r_full, kScanWarps);
    mbar_init(&c.vn_full, 1);
    mbar_init(&c.vd_full, kScanWarps);
    mbar_init(&c.sd_full, 1);
    mbar_init(&c.o_full, 1);
    mbar_init(&c.o_empty, kScanWarps);
    mbar_init(&c.fin, 1);
    c.abort = 0;
    fence_mbar_init();
  }
  // the upper right quarter of T is zero in both buffers
  for (int i = tid; i < 2 * 2 * 32 * 4; i += kThreadsC) {
    const int u = i & 3, r = (i >> 2) & 31, m = (i >> 7) & 1, b = i >> 8;
    *reinterpret_cast<uint4*>(sm.tp[b] + m * kTBytes + sw128(r, 4 + u)) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async();
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sm.ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sm.ctl.tmem;
  const Wait wait{&sm.ctl, a.dev_err};

  if (warp < kScanWarps) {
    scan_role<ST>(a, sm, wait, row0, len, h, chunks, tmem, init, slot);
  } else if (warp < kWarpMma) {
    prep_role(a, sm, wait, row0, len, h, chunks, tmem);
  } else if (warp == kWarpMma) {
    mma_role(sm, wait, chunks, tmem);
    // every product that was issued ends before tensor memory is given back
    if ((tid & 31) == 0) tc::commit(&sm.ctl.fin);
    __syncwarp();
    const long long t0 = clock64();
    while (!mbar_try(&sm.ctl.fin, 0))
      if (clock64() - t0 > kWaitClocks) {
        flag_error(a.dev_err, CCONV_DERR_TIMEOUT);
        break;
      }
  } else {
    load_role(a, sm, wait, row0, len, h, chunks);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <typename ST>
cudaError_t launch_chunk(const GdnArgs& a, cudaStream_t st) {
  constexpr size_t smem = sizeof(Smem) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  const cudaError_t e = cudaFuncSetAttribute(
      gdn_chunk_kernel<ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  gdn_chunk_kernel<ST><<<(unsigned)(a.B * a.Hv), kThreadsC, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gdn_launch_chunk(const GdnArgs& a, int state_dtype, cudaStream_t st) {
  return state_dtype == CCONV_DTYPE_F32 ? launch_chunk<float>(a, st)
                                        : launch_chunk<__nv_bfloat16>(a, st);
}

}  // namespace cconv
