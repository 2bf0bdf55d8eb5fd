// Chunked gated delta rule on the tensor cores (bf16, heads of 128 x 128): the
// long sequences of gdn_fwd_varlen.
//
// With the tokens of a chunk of C = 64 and G_i the sum of their log decays up
// to i, the recurrence S_i = a_i S_{i-1} + b_i k_i (v_i - a_i S_{i-1}^T k_i)^T is
//   A_ij = b_i e^{G_i - G_j} k_i.k_j  (j < i),   T = (I + A)^-1,
//   R_i  = b_i (v_i - e^{G_i} S^T k_i),          N = T R,
//   o_i  = scale (e^{G_i} S^T q_i + sum_{j<=i} e^{G_i - G_j} (q_i.k_j) N_j),
//   S'   = e^{G_C} S + sum_j e^{G_C - G_j} k_j N_j^T,
// one chain of chunks per sequence and head. Everything that does not need S --
// gates, norms, A, T, T V, q.k -- is worked out ahead of the chain by other
// warps, so that a link of it is three tensor products, one after the other
// (S^T k, T R, the update), and the element-wise work between them.
//
// Orientation. All products with S are taken transposed, with the 128 columns
// of S (dv) as the M rows of the tensor-core instruction and the tokens (or dk)
// as N: S^T, R^T and N^T are then A operands, which tcgen05 reads from tensor
// memory, lane = column of S; a thread owns one column, writes its row of the
// operand there and never passes it through shared memory. The B operands are
// the staged tiles themselves: K and Q (rows = tokens) for S^T k and S^T q, the
// same K tile read along its other dimension for the state update, T and the
// scores for the two products inside the chunk. V enters once, as (T V)^T, with
// V as the A operand from shared memory and before the chain arrives; T R then
// adds -T e^G S^T k to it.
//
// Precision. k, q and v are bf16 and exact. fp32 factors (S, R, T, N, the scores)
// enter as sums of two bf16 terms (about 16 bits; products lo * lo are left out),
// since the state must keep more than 8 bits over thousands of tokens: its error
// is 4e-6 of its norm against 64 bits, where single bf16 factors give 2e-3. The
// outputs are rounded once, when they are stored: 1.7e-3 of their norm against 64
// bits, 1.4e-4 against the rounded ones of 64 bits. (With one term for the scores
// and for S in S^T q they were 2.3e-3 off; 887 us at 16384 tokens then, 929 now.)
// S is held in fp32 registers from the first chunk to the last. l2 norms enter as factors of the rows, so that
// raw rows are multiplied. G is kept as whole part + remainder (in powers of
// two): chunks with strong decays reach sums of several hundred, whose
// differences fp32 alone would round by 1e-5.
//
// T is built by forward substitution of its four 16 x 16 diagonal blocks, in
// fp32, and products of blocks for the rest: stable for any keys, unlike sums
// of powers of A, whose terms cancel for equal keys.
//
// Roles (28 warps, registers dealt by setmaxnreg): 16 scan warps hold S and the
// chain, four work out A and the scores, two T, one issues every tcgen05.mma,
// one loads and works the gates out, four write the outputs and take the norms.
// They meet at mbarriers alone, each wait with a time limit, after which the
// block gives up and the launch reports it.
//
// Layout. K and Q of a chunk form one 128-row tile in the 128-byte swizzle (two
// panels of 64 dk each). Whole chunks come as tensor-map boxes; in a sequence's
// last, partial one the rows behind its end are filled with zeros by the copies
// themselves (cp.async), so nothing of the neighbouring request -- NaN, say --
// enters a product. Tensor memory columns: S 0-127, per 16 dk 8 columns hi and 8
// lo (the update's accumulator takes the same columns once S has been read),
// S^T k 128-191 (then N hi, lo), S^T q 192-255, R and then the decayed N (hi,
// lo) 256-319, T V + T R 320-383, in-chunk output 384-447, [K; Q] K^T 448-511.
//
// What bounds it. A chain is serial: at 16384 tokens of one request 256 links of
// 3.6 us, 0.93 ms, on 32 of the SMs (one a head); its bytes would take 0.06 ms
// and its products less. With 16 requests of up to 2048 tokens and 32 heads the
// 512 chains fill the GPU: 0.28 ms, where bytes take 0.07; the longest chains and
// the whole work weigh alike there. Inside a link every wait is short, and the
// roles' code together (72 KB) is larger than the instruction caches near the
// schedulers, so code size counts: unrolled loops and waits of 161 KB took 0.61
// ms for the 16 requests and 128 single tokens that take 0.37 now, and what is
// not on the chain stays rolled. Token by token (gdn_step.cu) the long chain
// takes 21.5 ms.
#include <cuda.h>
#include <math.h>
#include <stddef.h>

#include <mutex>

#include "gdn.cuh"
#include "tc.cuh"

namespace cconv {
namespace {

constexpr int kC = 64;                       // tokens of a chunk
constexpr int kD = 128;                      // dk = dv
constexpr int kStages = 3;
// Warpgroups: four on the chain, one for A and the scores, one of two warps for
// T, one that issues the tensor products and one that loads, and one for the
// outputs; registers a thread of each (their sum is the block's 896 x 72).
constexpr int kScanWarps = 16, kPrepWarps = 4, kInvWarps = 2, kOutWarps = 4;
constexpr int kWarpPrep0 = kScanWarps, kWarpInv0 = kWarpPrep0 + kPrepWarps,
              kWarpMma = kWarpInv0 + kInvWarps, kWarpLoad = kWarpMma + 1,
              kWarpOut0 = kWarpLoad + 1;
constexpr int kThreadsC = (kWarpOut0 + kOutWarps) * 32;
constexpr int kRegsScan = 72, kRegsPrep = 88, kRegsRest = 72, kRegsOut = 56;
static_assert(kThreadsC == 896 && 4 * kRegsScan + kRegsPrep + kRegsRest + kRegsOut <= 7 * 72,
              "a split over the block's own registers would wait forever");

constexpr uint32_t kPanel = 128 * 128;       // 64 dk of [K; Q]: 128 rows x 128 bytes
constexpr uint32_t kKQBytes = 2 * kPanel;
constexpr uint32_t kVPanel = kC * 128;       // 64 dv of V
constexpr uint32_t kVBytes = kC * kD * 2;    // V, later the chunk's outputs [64][128]
constexpr uint32_t kStageBytes = kKQBytes + kVBytes;
constexpr uint32_t kTBytes = kC * kC * 2;    // one 64 x 64 bf16 operand
constexpr uint32_t kDiagBytes = 16 * 128;    // four 16 x 16 blocks side by side
constexpr uint32_t kTP = 3 * kTBytes + kDiagBytes;   // T hi, T lo, scores (see p_lo)
constexpr int kMaxSeqs = 640;                // sequences of a launch
constexpr int kB = 16;                       // blocks of A and T
constexpr int kCoefs = 4;                    // chunks whose factors are kept

constexpr uint32_t kColS = 0, kColKS = 128, kColN = kColKS, kColQS = 192, kColR = 256,
                   kColVN = 320, kColO = 384, kColD1 = 448;

// A wait of this many nanoseconds gives the block up.
constexpr long long kWaitNs = 2000000000LL;

// Per-token factors of a chunk for the warps on the chain (read four at a time).
struct alignas(16) Coef {
  float rc[kC];      // -e^G / |k|
  float vd[kC];      // e^{G_C - G} / |k|
  float o1[kC];      // scale e^G / |q|
  float ec;          // e^{G_C}
};
// Gates of a chunk: sum of log2 decays (whole part, remainder) and beta.
struct alignas(16) Gate {
  float hi[kC], lo[kC], beta[kC];
};

struct Maps {
  CUtensorMap k, q, v;   // [tokens, heads * 128], boxes of 64 x 64 in the 128-byte swizzle
};

// A of a chunk: diagonal blocks in fp32, the blocks left of them as bf16 hi and
// lo (block (i, k) at i (i - 1) / 2 + k); 16-byte units permuted by row so that
// rows written or read together fall into different banks.
struct alignas(16) Blocks {
  float d[kC * kB];
  uint16_t hi[6 * kB * kB], lo[6 * kB * kB];
};
__device__ __forceinline__ int a_diag(int row, int unit) {          // index of 4 floats
  return row * kB + ((unit ^ ((row >> 1) & 3)) << 2);
}
__device__ __forceinline__ int a_left(int i, int k, int row, int unit) {   // of 8 bf16
  return ((i * (i - 1) / 2 + k) * kB + row) * kB + ((unit ^ ((row >> 2) & 1)) << 3);
}

__device__ __forceinline__ uint32_t sw128(int row, int unit) {
  return (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
}

// Scores: 10 blocks of 16 x 16 on and below the diagonal, in two bf16 terms. The
// first terms lie where they belong, block (I, J) in rows I and columns J of the
// tile; the second ones of the six blocks below the diagonal in the tile's free
// half, (I, J) in rows I - J - 1 and columns 3 - J, so that those of one J lie one
// below the other, as a product takes them; the second ones of the diagonal in a
// tile of 16 rows behind. Offset of row `row`, unit `unit` of a second term:
__device__ __forceinline__ uint32_t p_lo(int I, int J, int row, int unit) {
  return J < I ? sw128((I - J - 1) * kB + row, (3 - J) * 2 + unit)
               : kTBytes + sw128(row, J * 2 + unit);
}

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t gate_empty[2], tp_empty[2], coef_full[kCoefs], coef_empty[kCoefs];
  uint64_t rn_full[kStages], v_full[kStages], v_empty[kStages];
  uint64_t a_full[2], a_empty[2], t_full[2], p_full[2];
  uint64_t d1_full, d1_empty, prep_meet, inv_meet;
  uint64_t s_full[2], sd_full[2];
  uint64_t ks_full, qs_done, r_full, vn_full, vd_full, o_full, o_empty, fin;
  uint32_t tmem;
};

struct Smem {
  unsigned char stage[kStages][kStageBytes];   // 1024-byte aligned
  unsigned char tp[2][kTP];
  Blocks A[2];
  alignas(16) float tab[4][kC];                // e^{G_(16I-1) - G_j} / |k_j|, j < 16 I
  alignas(16) float rn[kStages][2 * kC];        // 1 / |k|, 1 / |q|
  Coef coef[kCoefs];
  Gate gate[2];
  uint16_t order[kMaxSeqs];   // the launch's long sequences, longest first
  int count, total;           // how many; chunks of this block's chains
  Ctl ctl;
};
static_assert(offsetof(Smem, tp) % 1024 == 0 && kStageBytes % 1024 == 0 && kTP % 1024 == 0 &&
                  kTBytes % 1024 == 0 && kVPanel % 1024 == 0,
              "swizzled tiles start on 1024 bytes");
static_assert(sizeof(Coef) % 16 == 0 && sizeof(Gate) % 16 == 0 && sizeof(Blocks) % 16 == 0 &&
                  offsetof(Smem, A) % 16 == 0 &&
                  offsetof(Smem, tab) % 16 == 0 && offsetof(Smem, rn) % 16 == 0 &&
                  offsetof(Smem, coef) % 16 == 0 && offsetof(Smem, gate) % 16 == 0 &&
                  offsetof(Smem, ctl) % 8 == 0,
              "16-byte accesses");

// A wait of a whole warp on a phase: false when it has run out of time, and the
// role gives up (what waits for it runs out of time in turn). Few instructions,
// and in line: the block's code is larger than the instruction caches near the
// schedulers, so every role pays for the size of all; and a call would spill
// the state's registers around it.
struct Wait {
  __device__ __forceinline__ bool operator()(uint64_t* bar, int phase) const {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 t0, t1;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "mov.u64 t0, %globaltimer;\n"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "mov.u64 t1, %globaltimer;\n\t"
        "sub.u64 t1, t1, t0;\n\t"
        "setp.lt.u64 q, t1, %3;\n\t"
        "@q bra AGAIN;\n"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"((uint32_t)(phase & 1)), "n"(kWaitNs)
        : "memory");
    return __all_sync(0xffffffffu, ok != 0);
  }
};

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Meeting point of a role's warps (a barrier of the block that can be given up).
struct Meet {
  uint64_t* bar;
  int phase;
  __device__ __forceinline__ bool operator()(const Wait& wait) {
    warp_arrive(bar);
    return wait(bar, phase++);
  }
};
template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- which chains a block takes ----------------------------------------------

// The chains of a launch, longest sequence first, a head after the other, are
// dealt to the blocks back and forth, so that each gets some of every length.
// Neighbouring heads, which share K and Q, run at the same time.
struct Chain {
  int row0, len, chunks, h, slot;
  bool init;
};
__device__ __forceinline__ bool chain_at(const GdnArgs& a, const Smem& sm, int k, Chain& c) {
  const uint32_t i = k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (i >= (uint32_t)sm.count * a.Hv) return false;   // (less than 2^31: a host check)
  const uint32_t r = i / (uint32_t)a.Hv;
  const int s = sm.order[r];
  c.h = (int)(i - r * a.Hv);
  c.row0 = a.cu[s];
  c.len = a.cu[s + 1] - c.row0;
  c.chunks = (c.len + kC - 1) / kC;
  c.slot = a.state_idx[s];
  c.init = c.slot >= 0 && (!a.has_init || a.has_init[s]);
  return true;
}

// Fills order, count and total. All threads; `lens` is scratch of kMaxSeqs.
__device__ __forceinline__ void order_chains(const GdnArgs& a, Smem& sm, int* lens) {
  const int s = threadIdx.x;
  static_assert(kThreadsC >= kMaxSeqs, "a thread a sequence");
  int len = 0;
  if (s < a.B) {
    int row0;
    // (a bad cu_seqlens entry is reported by the recurrent kernel)
    if (!gdn_bounds(a, s, row0, len) || len <= a.max_len) len = 0;
    if (len > 0 && a.state_idx[s] >= a.num_slots) {
      if (blockIdx.x == 0) flag_error(a.dev_err, CCONV_DERR_SLOT_RANGE);
      len = 0;
    }
  }
  if (s < kMaxSeqs) lens[s] = len;
  const int count = __syncthreads_count(len > 0);
  if (len > 0) {
    int rank = 0;
    for (int i = 0; i < a.B; ++i) {
      const int o = lens[i];
      rank += o > len || (o == len && i < s);
    }
    sm.order[rank] = (uint16_t)s;
  }
  if (s == 0) sm.count = count;
  __syncthreads();
  if (s < 32) {
    int sum = 0;
    Chain c;
    for (int k = s; chain_at(a, sm, k, c); k += 32) sum += c.chunks;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (s == 0) sm.total = sum;
  }
  __syncthreads();
}

// ---- the warp that loads K, Q and V and works the gates out -----------------

// Per chunk: requests its rows, works its gates out while they come. Whole
// chunks come as tensor-map boxes; the last, partial one row by row, with
// zeros behind the sequence's end. Gates: two tokens a lane (lane, lane + 32);
// their sums are kept as whole part and remainder in (-1, 0], exact to 2^-24 of
// the remainder however long the sum.
__device__ __forceinline__ bool load_role(const GdnArgs& a, const Maps& maps, Smem& sm,
                                          const Wait& wait) {
  const int lane = threadIdx.x & 31, u = lane & 15, r2 = lane >> 4;
  const __nv_bfloat16* const ga0 = reinterpret_cast<const __nv_bfloat16*>(a.a);
  const __nv_bfloat16* const gb0 = reinterpret_cast<const __nv_bfloat16*>(a.b);
  int boxed = 0, v_boxed = 0;   // last chunks that came as boxes
  int g = 0;                    // chunks of the block so far
  Chain c;
  for (int k = 0; chain_at(a, sm, k, c); ++k) {
    const int row0 = c.row0, len = c.len, h = c.h;
    const int hk = h / (a.Hv / a.Hk);
    const char* kp = a.k + ((int64_t)row0 * a.k_rs + (int64_t)hk * kD) * 2 + u * 16;
    const char* qp = a.q + ((int64_t)row0 * a.q_rs + (int64_t)hk * kD) * 2 + u * 16;
    const char* vp = a.v + ((int64_t)row0 * a.v_rs + (int64_t)h * kD) * 2 + u * 16;
    const float A_log2 = -expf(a.A_log[h]) * 1.4426950408889634f;
    const float dtb = a.dt_bias[h];
    const __nv_bfloat16* ga = ga0 + h;
    const __nv_bfloat16* gb = gb0 + h;
    if (c.init) {             // the chain's state, for the warps that will read it
      const char* sp = a.st + ((int64_t)c.slot * a.st_slot + (int64_t)h * a.st_head) * a.st_bytes;
      for (int i = lane * 128; i < kD * kD * a.st_bytes; i += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(sp + i));
    }
    for (int n = 0; n < c.chunks; ++n, ++g) {
      const int st = g % kStages;
      if (g >= kStages && !wait(&sm.ctl.empty[st], g / kStages - 1)) goto quit;
      const int tok = n * kC + lane;
      float na[2], nb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = tok + i * 32;
        na[i] = t < len ? elem(ga, (int64_t)(row0 + t) * a.a_rs) : 0.0f;
        nb[i] = t < len ? elem(gb, (int64_t)(row0 + t) * a.b_rs) : 0.0f;
      }
      // K and Q, then, when the outputs have left its place, V
      const bool whole = len - n * kC >= kC;
      const int y = row0 + n * kC;
      const uint32_t at = smem_addr(sm.stage[st]);
      auto rows = [&](uint32_t dst, uint32_t pitch, const char* src, int64_t stride) {
#pragma unroll 1
        for (int i = r2; i < kC; i += 2) {
          const bool in = n * kC + i < len;
          cp_async16(dst + (u >> 3) * pitch + sw128(i, u & 7),
                     src + (int64_t)(in ? n * kC + i : 0) * stride * 2, in);
        }
      };
      if (whole) {
        boxed = g + 1;
        if (lane == 0) {
          mbar_arrive_tx(&sm.ctl.full[st], kKQBytes);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            tc::tma_load_2d(at + p * kPanel, &maps.k, hk * kD + p * 64, y, &sm.ctl.full[st]);
            tc::tma_load_2d(at + p * kPanel + kC * 128, &maps.q, hk * kD + p * 64, y,
                            &sm.ctl.full[st]);
          }
        }
      } else {
        rows(at, kPanel, kp, a.k_rs);
        rows(at + kC * 128, kPanel, qp, a.q_rs);
        cp_async_commit();
      }
      if (g >= 2 && !wait(&sm.ctl.gate_empty[g & 1], (g >> 1) - 1)) {
        warp_arrive(&sm.ctl.full[st]);
        goto quit;
      }
      Gate& G = sm.gate[g & 1];
      float w0 = 0.0f, f0 = 0.0f;                    // sums so far
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const bool in = tok + i * 32 < len;
        const float x = (i == 0 ? na[0] : na[1]) + dtb;
        float gl = A_log2 * gdn_softplus(x);
        // a decay below 2^-150 is zero in fp32 whatever follows (a NaN stays one)
        gl = in ? (gl < -150.0f ? -150.0f : gl) : 0.0f;
        float w = truncf(gl), f = gl - w;
        auto add = [&](float ow, float of) {
          const float s = f + of, c = truncf(s);
          w += ow + c;
          f = s - c;
        };
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
          const float ow = __shfl_up_sync(0xffffffffu, w, d);
          const float of = __shfl_up_sync(0xffffffffu, f, d);
          if (lane >= d) add(ow, of);
        }
        add(w0, f0);
        w0 = __shfl_sync(0xffffffffu, w, 31);
        f0 = __shfl_sync(0xffffffffu, f, 31);
        G.hi[i * 32 + lane] = w;
        G.lo[i * 32 + lane] = f;
        G.beta[i * 32 + lane] = in ? gdn_beta(i == 0 ? nb[0] : nb[1]) : 0.0f;
      }
      if (!whole) {
        cp_async_wait<0>();
        fence_proxy_async();
        if (lane == 0) mbar_arrive(&sm.ctl.full[st]);
      }
      warp_arrive(&sm.ctl.full[st]);
      if (g >= kStages && !wait(&sm.ctl.v_empty[st], g / kStages - 1)) goto quit;
      if (whole) {
        v_boxed = g + 1;
        if (lane == 0) {
          mbar_arrive_tx(&sm.ctl.v_full[st], kVBytes);
#pragma unroll
          for (int p = 0; p < 2; ++p)
            tc::tma_load_2d(at + kKQBytes + p * kVPanel, &maps.v, h * kD + p * 64, y,
                            &sm.ctl.v_full[st]);
        }
      } else {
        rows(at + kKQBytes, kVPanel, vp, a.v_rs);
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async();
        warp_arrive(&sm.ctl.v_full[st]);
      }
    }
  }
  return true;
quit:                       // given up: no copy lands after the block ends
  cp_async_wait<0>();
  for (int i = max(boxed - kStages, 0); i < boxed; ++i)
    wait(&sm.ctl.full[i % kStages], i / kStages);
  for (int i = max(v_boxed - kStages, 0); i < v_boxed; ++i)
    wait(&sm.ctl.v_full[i % kStages], i / kStages);
  return false;
}

// ---- the warps that look one chunk ahead ------------------------------------

// Four pairs of fp32 as bf16 hi and lo.
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo) {
  tc::split2(x[0], x[1], hi.x, lo.x);
  tc::split2(x[2], x[3], hi.y, lo.y);
  tc::split2(x[4], x[5], hi.z, lo.z);
  tc::split2(x[6], x[7], hi.w, lo.w);
}

// The 16 x 16 blocks of T below the diagonal, by two warps. With U = T^T, which
// is how T is stored for the tensor cores,
//   U_Ji = -(sum_{J <= k < i} U_Jk A_ik^T) U_ii
// is taken in two levels of 32 x 32 blocks: first U_01 (warp 0) and U_23 (warp 1),
// then, for J = 0 and 1, X_2 = sum_k U_Jk A_2k^T and X_3 = sum_k U_Jk A_3k^T over k =
// J .. 1, and U_J2 = -X_2 U_22, U_J3 = -(X_2 U_23 + X_3 U_33). Factors and A are
// read as they lie in shared memory; X passes to its second product in
// registers, where the output layout of one warp product is the input layout
// of the next. Products of hi and lo parts as everywhere (lo * lo left out), the
// mixed ones in a sum of their own: shorter chains.
struct Sum {
  float x[2][4], m[2][4];       // hi * hi, mixed; two tiles of 8 columns
};
template <bool PAIRS>
__device__ __forceinline__ void mul_add(Sum& s, const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                        const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
  // right operand of tile nt: registers 2 nt, 2 nt + 1 (PAIRS) or nt, nt + 2
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int i0 = PAIRS ? 2 * nt : nt, i1 = PAIRS ? 2 * nt + 1 : nt + 2;
    tc::mma16(s.x[nt], ah, bh[i0], bh[i1]);
    tc::mma16(s.m[nt], ah, bl[i0], bl[i1]);
    tc::mma16(s.m[nt], al, bh[i0], bh[i1]);
  }
}
// The sum times `sign` as a left operand, hi and lo.
__device__ __forceinline__ void to_left(const Sum& s, float sign, uint32_t (&h)[4],
                                        uint32_t (&l)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    tc::split2(sign * (s.x[e >> 1][(e & 1) * 2] + s.m[e >> 1][(e & 1) * 2]),
               sign * (s.x[e >> 1][(e & 1) * 2 + 1] + s.m[e >> 1][(e & 1) * 2 + 1]), h[e], l[e]);
}
struct TWarp {
  const Blocks& A;
  unsigned char* tp;
  int lane, lrow, lu;           // lane; its row and unit of a block for ldmatrix
  __device__ __forceinline__ void left(int J, int k, uint32_t (&h)[4], uint32_t (&l)[4]) const {
    const uint32_t at = smem_addr(tp) + sw128(J * kB + lrow, k * 2 + lu);       // U_Jk
    tc::ldmatrix4(h, at);
    tc::ldmatrix4(l, at + kTBytes);
  }
  __device__ __forceinline__ void right(int i, int k, uint32_t (&h)[4], uint32_t (&l)[4]) const {
    const uint32_t at = smem_addr(tp) + sw128(i * kB + lrow, k * 2 + lu);       // U_ik
    tc::ldmatrix4_trans(h, at);
    tc::ldmatrix4_trans(l, at + kTBytes);
  }
  __device__ __forceinline__ void a_right(int i, int k, uint32_t (&h)[4],
                                          uint32_t (&l)[4]) const {             // A_ik^T
    const int at = a_left(i, k, lrow, lu);
    tc::ldmatrix4(h, smem_addr(&A.hi[at]));
    tc::ldmatrix4(l, smem_addr(&A.lo[at]));
  }
  // U_Ji, from its left-operand form
  __device__ __forceinline__ void put(int J, int i, const uint32_t (&h)[4],
                                      const uint32_t (&l)[4]) const {
    const int r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {      // rows r, r + 8 (e & 1) of tile e >> 1
      const uint32_t at = sw128(J * kB + r + (e & 1) * 8, i * 2 + (e >> 1)) + c * 2;
      *reinterpret_cast<uint32_t*>(tp + at) = h[e];
      *reinterpret_cast<uint32_t*>(tp + kTBytes + at) = l[e];
    }
  }
};
__device__ __forceinline__ bool t_blocks(const TWarp& w, int warp, Meet& meet, const Wait& wait) {
  uint32_t uh[4], ul[4], bh[4], bl[4], xh[4], xl[4];
  {                                    // U_01 or U_23
    const int J = warp * 2;
    Sum x = {}, y = {};
    w.left(J, J, uh, ul);
    w.a_right(J + 1, J, bh, bl);
    mul_add<false>(x, uh, ul, bh, bl);
    w.right(J + 1, J + 1, bh, bl);
    to_left(x, 1.0f, xh, xl);
    mul_add<true>(y, xh, xl, bh, bl);
    to_left(y, -1.0f, xh, xl);
    w.put(J, J + 1, xh, xl);
  }
  if (!meet(wait)) return false;
  const int J = warp;
  Sum x2 = {}, x3 = {};
#pragma unroll 1
  for (int k = J; k < 2; ++k) {
    w.left(J, k, uh, ul);
    w.a_right(2, k, bh, bl);
    mul_add<false>(x2, uh, ul, bh, bl);
    w.a_right(3, k, bh, bl);
    mul_add<false>(x3, uh, ul, bh, bl);
  }
  Sum y2 = {}, y3 = {};
  to_left(x2, 1.0f, xh, xl);
  w.right(2, 2, bh, bl);
  mul_add<true>(y2, xh, xl, bh, bl);
  w.right(2, 3, bh, bl);
  mul_add<true>(y3, xh, xl, bh, bl);
  to_left(x3, 1.0f, uh, ul);
  w.right(3, 3, bh, bl);
  mul_add<true>(y3, uh, ul, bh, bl);
  to_left(y2, -1.0f, xh, xl);
  w.put(J, 2, xh, xl);
  to_left(y3, -1.0f, xh, xl);
  w.put(J, 3, xh, xl);
  return true;
}

// Factors, A and the scores of every chunk. Thread p < 64 holds row p of K K^T,
// thread 64 + p row p of Q K^T.
__device__ __forceinline__ bool prep_role(const GdnArgs& a, Smem& sm, const Wait& wait,
                                          int chunks, uint32_t tmem) {
  const int p = threadIdx.x - kWarpPrep0 * 32, warp = p >> 5;
  const bool is_k = p < kC;
  const int r = p & (kC - 1), blk = r / kB;       // the thread's row and its block
  Meet meet{&sm.ctl.prep_meet, 0};
  for (int n = 0; n < chunks; ++n) {
    const int st = n % kStages, bf = n & 1;
    Coef& C = sm.coef[n % kCoefs];
    const Gate& G = sm.gate[bf];
    if (!wait(&sm.ctl.full[st], n / kStages) || !wait(&sm.ctl.rn_full[n % kStages], n / kStages))
      return false;
    const float* const rns = sm.rn[n % kStages];
    const float rn = rns[p];
    if (n >= kCoefs && !wait(&sm.ctl.coef_empty[n % kCoefs], n / kCoefs - 1)) return false;
    // ---- factors
    const float hi = G.hi[r], lo = G.lo[r];
    const float eg = tc::ex2(hi + lo);
    if (is_k) {
      C.rc[r] = -eg * rn;
      C.vd[r] = rn * tc::ex2((G.hi[kC - 1] - hi) + (G.lo[kC - 1] - lo));
      if (r == kC - 1) C.ec = eg;
    } else {
      C.o1[r] = a.scale * rn * eg;
    }
    {
      const float rk = rns[r];
#pragma unroll
      for (int I = 1; I < 4; ++I)
        if ((I == 3) == is_k && r < I * kB)
          sm.tab[I][r] = rk * tc::ex2((G.hi[I * kB - 1] - hi) + (G.lo[I * kB - 1] - lo));
    }
    const float fac = is_k ? rn : a.scale * rn;
    const float off =
        blk > 0 ? fac * tc::ex2((hi - G.hi[blk * kB - 1]) + (lo - G.lo[blk * kB - 1])) : 0.0f;
    warp_arrive(&sm.ctl.coef_full[n % kCoefs]);
    // the row's factors of the diagonal block, zero above it (in registers: worked
    // out where they are used, in half of a warp's lanes at a time, they made 16384
    // tokens 1317 us)
    float e[kB];
#pragma unroll
    for (int j4 = 0; j4 < kB; j4 += 4) {
      const int j = blk * kB + j4;
      const float4 h4 = *reinterpret_cast<const float4*>(&G.hi[j]);
      const float4 l4 = *reinterpret_cast<const float4*>(&G.lo[j]);
      const float4 k4 = *reinterpret_cast<const float4*>(&rns[j]);
      float d[4], f[4];
      fma_x2(d[0], d[1], l4.x, l4.y, -1.0f, -1.0f, lo, lo);
      fma_x2(d[2], d[3], l4.z, l4.w, -1.0f, -1.0f, lo, lo);
      fma_x2(f[0], f[1], h4.x, h4.y, -1.0f, -1.0f, hi, hi);
      fma_x2(f[2], f[3], h4.z, h4.w, -1.0f, -1.0f, hi, hi);
      fma_x2(d[0], d[1], f[0], f[1], 1.0f, 1.0f, d[0], d[1]);
      fma_x2(d[2], d[3], f[2], f[3], 1.0f, 1.0f, d[2], d[3]);
      mul_x2(f[0], f[1], k4.x, k4.y, fac, fac);
      mul_x2(f[2], f[3], k4.z, k4.w, fac, fac);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = tc::ex2(j + i <= r ? d[i] : -INFINITY);
      mul_x2(e[j4], e[j4 + 1], d[0], d[1], f[0], f[1]);
      mul_x2(e[j4 + 2], e[j4 + 3], d[2], d[3], f[2], f[3]);
    }
    if (!meet(wait)) return false;
    // ---- A and the scores from [K; Q] K^T: row r times the factors of its columns
    if (!wait(&sm.ctl.d1_full, n)) return false;
    tc::fence_after();
    if (n >= 2 && !wait(is_k ? &sm.ctl.a_empty[bf] : &sm.ctl.tp_empty[bf], (n >> 1) - 1))
      return false;
    unsigned char* const scores = sm.tp[bf] + 2 * kTBytes;
    const uint32_t d1 = tmem + kColD1 + ((uint32_t)(warp * 32) << 16);
    // (the last block that one of the warp's rows has)
    const int last = (warp & 1) * 2 + 1;
#pragma unroll 1
    for (int J = 0; J <= last; ++J) {
      uint32_t x[16];
      tc::ld16(d1 + J * 16, x);
      tc::wait_ld(x);
      if (J <= blk) {
        // left of the diagonal: e^{G_i - G_j} as two factors at most 1 around the
        // start of the row's block
        float y[16];
#pragma unroll
        for (int j4 = 0; j4 < 16; j4 += 4) {
          const float4 t = *reinterpret_cast<const float4*>(&sm.tab[blk][J * kB + j4]);
          const bool left = J < blk;
          mul_x2(y[j4], y[j4 + 1], left ? off * t.x : e[j4], left ? off * t.y : e[j4 + 1],
                 __uint_as_float(x[j4]), __uint_as_float(x[j4 + 1]));
          mul_x2(y[j4 + 2], y[j4 + 3], left ? off * t.z : e[j4 + 2], left ? off * t.w : e[j4 + 3],
                 __uint_as_float(x[j4 + 2]), __uint_as_float(x[j4 + 3]));
        }
        if (is_k && J == blk) {
#pragma unroll
          for (int j4 = 0; j4 < 16; j4 += 4)
            *reinterpret_cast<float4*>(&sm.A[bf].d[a_diag(r, j4 >> 2)]) =
                make_float4(y[j4], y[j4 + 1], y[j4 + 2], y[j4 + 3]);
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint4 h, l;
            split8(y + u * 8, h, l);
            if (is_k) {
              const int at = a_left(blk, J, r & (kB - 1), u);
              *reinterpret_cast<uint4*>(&sm.A[bf].hi[at]) = h;
              *reinterpret_cast<uint4*>(&sm.A[bf].lo[at]) = l;
            } else {
              *reinterpret_cast<uint4*>(scores + sw128(r, J * 2 + u)) = h;
              *reinterpret_cast<uint4*>(scores + p_lo(blk, J, r & (kB - 1), u)) = l;
            }
          }
        }
      }
      __syncwarp();
    }
    tc::fence_before();
    warp_arrive(&sm.ctl.d1_empty);
    if (is_k) {
      warp_arrive(&sm.ctl.a_full[bf]);
    } else {
      fence_proxy_async();
      warp_arrive(&sm.ctl.p_full[bf]);
    }
    warp_arrive(&sm.ctl.gate_empty[bf]);
    if (!meet(wait)) return false;     // tab and rn are free for the next chunk
  }
  return true;
}

// T of every chunk, by two warps: forward substitution of the four diagonal
// blocks (a lane a column, two blocks a warp), then the blocks below them. What
// is built is T with its columns scaled by beta, (diag(1 / beta) + A)^-1 for the
// A without beta that the scores' warps wrote: rows t_i = beta_i (e_i - sum_k
// A_ik t_k), without a division, so that beta = 0 needs nothing of its own.
__device__ __forceinline__ bool inv_role(Smem& sm, const Wait& wait, int chunks) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kWarpInv0;
  const int blk = warp * 2 + (lane >> 4), c = lane & (kB - 1), b0 = blk * kB;
  Meet meet{&sm.ctl.inv_meet, 0};
  for (int n = 0; n < chunks; ++n) {
    const int bf = n & 1;
    const Gate& G = sm.gate[bf];
    unsigned char* const tp = sm.tp[bf];
    if (!wait(&sm.ctl.a_full[bf], n >> 1)) return false;
    if (n >= 2 && !wait(&sm.ctl.tp_empty[bf], (n >> 1) - 1)) return false;
    const Blocks& A = sm.A[bf];
    float t[kB];
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      float acc[4] = {c == i ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k4 = 0; k4 < i; k4 += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&A.d[a_diag(b0 + i, k4 >> 2)]);
        acc[0] = fmaf(-v.x, t[k4], acc[0]);
        if (k4 + 1 < i) acc[1] = fmaf(-v.y, t[k4 + 1], acc[1]);
        if (k4 + 2 < i) acc[2] = fmaf(-v.z, t[k4 + 2], acc[2]);
        if (k4 + 3 < i) acc[3] = fmaf(-v.w, t[k4 + 3], acc[3]);
      }
      t[i] = G.beta[b0 + i] * ((acc[0] + acc[1]) + (acc[2] + acc[3]));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint4 h, l;
      split8(t + u * 8, h, l);
      *reinterpret_cast<uint4*>(tp + sw128(b0 + c, blk * 2 + u)) = h;
      *reinterpret_cast<uint4*>(tp + kTBytes + sw128(b0 + c, blk * 2 + u)) = l;
    }
    __syncwarp();     // (the first level reads the warp's own blocks)
    if (!t_blocks(TWarp{A, tp, lane, lane & 15, lane >> 4}, warp, meet, wait)) return false;
    fence_proxy_async();
    warp_arrive(&sm.ctl.t_full[bf]);
    warp_arrive(&sm.ctl.a_empty[bf]);
    warp_arrive(&sm.ctl.gate_empty[bf]);
  }
  return true;
}

// ---- the warps on the chain -------------------------------------------------

// Thread: column `col` of S, dk p * 64 + qt * 16 + [0, 16) in S[p * 16 ..], p =
// 0, 1: the two halves of dk pass through the update and the split one after
// the other, while the tensor cores work on the other one. Of a chunk's tokens
// the thread has qt * 16 + [0, 16). (Four warps a quadrant of lanes: what a warp
// does between two products is short then; with two, the chain was a third
// longer.)
template <typename ST>
__device__ __forceinline__ bool scan_role(const GdnArgs& a, Smem& sm, const Wait& wait,
                                          uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qd = warp & 3, qt = warp >> 2;
  const int col = qd * 32 + lane;
  const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
  const uint32_t ts = tl + kColS + qt * 16;
  float S[32];

  // S = e^{G_C} S + update of chunk n, one half
  auto advance = [&](int n, int p) -> bool {
    if (!wait(&sm.ctl.sd_full[p], n)) return false;
    tc::fence_after();
    uint32_t x[16];
    tc::ld16(ts + p * 64, x);
    const float ec = sm.coef[n % kCoefs].ec;
    tc::wait_ld(x);
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      fma_x2(S[p * 16 + i], S[p * 16 + i + 1], ec, ec, S[p * 16 + i], S[p * 16 + i + 1],
             __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
    return true;
  };
  // the thread's 16 tokens times their factors, split, to kColR
  auto scaled = [&](const uint32_t(&x)[16], const float* f) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 c = *reinterpret_cast<const float4*>(f + qt * 16 + i);
      float q[4];
      mul_x2(q[0], q[1], c.x, c.y, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
      mul_x2(q[2], q[3], c.z, c.w, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
      tc::split2(q[0], q[1], hi[i / 2], lo[i / 2]);
      tc::split2(q[2], q[3], hi[i / 2 + 1], lo[i / 2 + 1]);
    }
    tc::st8(tl + kColR + qt * 8, hi);
    tc::st8(tl + kColR + 32 + qt * 8, lo);
  };

  int n = 0;                                      // chunks of the block so far
  Chain ch;
  for (int k = 0; chain_at(a, sm, k, ch); ++k) {
    ST* const sp = reinterpret_cast<ST*>(a.st) +
                   (int64_t)(ch.slot < 0 ? 0 : ch.slot) * a.st_slot + (int64_t)ch.h * a.st_head +
                   (int64_t)qt * 16 * kD + col;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      S[i] = ch.init ? elem(sp, ((i >> 4) * 64 + (i & 15)) * kD) : 0.0f;
    for (int m = 0; m < ch.chunks; ++m, ++n) {
      const Coef& C = sm.coef[n % kCoefs];
      // ---- S: add the last chunk's update, split, hand to the tensor cores
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (m > 0 && !advance(n - 1, p)) return false;
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tc::split2(S[p * 16 + 2 * i], S[p * 16 + 2 * i + 1], hi[i], lo[i]);
        tc::st8(ts + p * 64, hi);
        tc::st8(ts + p * 64 + 8, lo);
        tc::wait_st();
        tc::fence_before();
        warp_arrive(&sm.ctl.s_full[p]);
      }
      if (m > 0) warp_arrive(&sm.ctl.coef_empty[(n - 1) % kCoefs]);
      // ---- R
      if (!wait(&sm.ctl.coef_full[n % kCoefs], n / kCoefs) || !wait(&sm.ctl.ks_full, n))
        return false;
      tc::fence_after();
      uint32_t x[16];
      tc::ld16(tl + kColKS + qt * 16, x);
      tc::wait_ld(x);
      scaled(x, C.rc);
      tc::wait_st();
      tc::fence_before();
      warp_arrive(&sm.ctl.r_full);
      // ---- N
      if (!wait(&sm.ctl.vn_full, n)) return false;
      tc::fence_after();
      tc::ld16(tl + kColVN + qt * 16, x);
      tc::wait_ld(x);
      scaled(x, C.vd);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        tc::split2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), hi[i], lo[i]);
      tc::st8(tl + kColN + qt * 8, hi);
      tc::st8(tl + kColN + 32 + qt * 8, lo);
      tc::wait_st();
      tc::fence_before();
      warp_arrive(&sm.ctl.vd_full);
    }
    if (!advance(n - 1, 0) || !advance(n - 1, 1)) return false;
    warp_arrive(&sm.ctl.coef_empty[(n - 1) % kCoefs]);
    if (ch.slot >= 0)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const auto raw = f32_to_raw<ST>(S[i]);
        *reinterpret_cast<std::remove_const_t<decltype(raw)>*>(
            sp + ((i >> 4) * 64 + (i & 15)) * kD) = raw;
      }
  }
  return true;
}

// Outputs: a warp takes 32 columns, 16 tokens at a time, turns them round in
// the chunk's V, which has been used, and stores 16-byte units. In between the
// same warps take the norms of the chunk three further on (a thread a row).
__device__ __forceinline__ bool out_role(const GdnArgs& a, Smem& sm, const Wait& wait,
                                         int chunks, uint32_t tmem) {
  const int qd = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
  auto norms = [&](int m) -> bool {
    if (m >= chunks) return true;
    if (!wait(&sm.ctl.full[m % kStages], m / kStages)) return false;
    const int p = threadIdx.x - kWarpOut0 * 32;         // row of [K; Q]
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
    if (a.l2norm) {
#pragma unroll 4
      for (int u = 0; u < 16; ++u) {
        const uint4 x = *reinterpret_cast<const uint4*>(sm.stage[m % kStages] + (u >> 3) * kPanel +
                                                        sw128(p, u & 7));
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float a0 = __uint_as_float(q[e] << 16), a1 = __uint_as_float(q[e] & 0xffff0000u);
          const float b0 = __uint_as_float(q[e + 1] << 16),
                      b1 = __uint_as_float(q[e + 1] & 0xffff0000u);
          fma_x2(s0, s1, a0, a1, a0, a1, s0, s1);
          fma_x2(s2, s3, b0, b1, b0, b1, s2, s3);
        }
      }
    }
    sm.rn[m % kStages][p] = a.l2norm ? rsqrtf((s0 + s1) + (s2 + s3) + kGdnNormEps) : 1.0f;
    warp_arrive(&sm.ctl.rn_full[m % kStages]);
    return true;
  };
  for (int m = 0; m < kStages; ++m)
    if (!norms(m)) return false;
  int n = 0;                                      // chunks of the block so far
  Chain ch;
  for (int k = 0; chain_at(a, sm, k, ch); ++k) {
    char* const op = a.out + ((int64_t)ch.row0 * a.out_rs + (int64_t)ch.h * kD + qd * 32) * 2 +
                     (lane & 3) * 16;
    for (int m = 0; m < ch.chunks; ++m, ++n) {
      if (!wait(&sm.ctl.o_full, n)) return false;
      tc::fence_after();
      unsigned char* const box = sm.stage[n % kStages] + kKQBytes + qd * 4096;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        uint32_t x[16], y[16];
        tc::ld16(tl + kColQS + g * 16, x);
        tc::ld16(tl + kColO + g * 16, y);
        tc::wait_ld(x);
        tc::wait_ld(y);
        if (g == 3) {
          tc::fence_before();
          warp_arrive(&sm.ctl.o_empty);
        }
        uint16_t* const o = reinterpret_cast<uint16_t*>(box + g * 1024) + lane;
        const float* f = sm.coef[n % kCoefs].o1 + g * 16;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 c = *reinterpret_cast<const float4*>(f + i);
          float v[4];
          fma_x2(v[0], v[1], c.x, c.y, __uint_as_float(x[i]), __uint_as_float(x[i + 1]),
                 __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
          fma_x2(v[2], v[3], c.z, c.w, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]),
                 __uint_as_float(y[i + 2]), __uint_as_float(y[i + 3]));
          const uint32_t p0 = pack_bf16x2(v[0], v[1]), p1 = pack_bf16x2(v[2], v[3]);
          o[i * 32] = (uint16_t)p0;
          o[(i + 1) * 32] = (uint16_t)(p0 >> 16);
          o[(i + 2) * 32] = (uint16_t)p1;
          o[(i + 3) * 32] = (uint16_t)(p1 >> 16);
        }
      }
      warp_arrive(&sm.ctl.coef_empty[n % kCoefs]);
      char* ot = op + ((int64_t)m * kC + (lane >> 2)) * a.out_rs * 2;
      const int left = ch.len - m * kC - (lane >> 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 q = *reinterpret_cast<const uint4*>(box + (i * 32 + lane) * 16);
        if (i * 8 < left) *reinterpret_cast<uint4*>(ot) = q;
        ot += a.out_rs * 16;
      }
      fence_proxy_async();
      warp_arrive(&sm.ctl.v_empty[n % kStages]);
      if (!norms(n + kStages)) return false;
    }
  }
  return true;
}

// ---- the warp that issues the tensor products -------------------------------

// On the chain: S^T k (16 products of N = 64, 512 clocks), T R (12, 384), the
// update (16, 512). Beside it: S^T q, in-chunk outputs, and, while the chain's
// warps work on S, T V of this chunk and the scores of the next ones.
__device__ __forceinline__ bool mma_role(Smem& sm, const Wait& wait, int chunks, uint32_t tmem) {
  constexpr uint32_t kId = tc::idesc(128, 64), kIdT = tc::idesc(128, 64, false, true),
                     kIdV = tc::idesc(128, 64, true, true);
  // descriptors of the first stage and T buffer; others lie a constant further
  // (their addresses are counted in units of 16 bytes). K, Q, scores: K-major;
  // K for the update: 64 dk of 16 tokens, MN-major, like V and U.
  const uint64_t kq0 = tc::desc_sw128(smem_addr(sm.stage[0]), 16);
  const uint64_t v0 = tc::desc_sw128(smem_addr(sm.stage[0]) + kKQBytes, kVPanel);
  const uint64_t t0 = tc::desc_sw128(smem_addr(sm.tp[0]), 16);
  auto panel = [](int ks, int row) {            // 16 dk of rows [row, ..) of [K; Q]
    return ((ks >> 2) * kPanel + (ks & 3) * 32 + row * 128) >> 4;
  };
  // Steps of a chunk: S^T k of the first half of dk, of the second (with S^T q),
  // T R, update. The pipe is free while the chain's warps work: T V of this chunk
  // is issued while S is worked on, the scores of the next chunk that has none
  // while R or N is, each as soon as its operands are there (and at the latest
  // before T R, which needs both). Issued before S^T k, the scores held it up by
  // 500 clocks.
  int scored = 0, tved = 0;                     // chunks whose products are issued
#pragma unroll 1
  for (int step = 0; step < 4 * chunks; ++step) {
    const int n = step >> 2, sub = step & 3, st = n % kStages;
    const uint64_t kq = kq0 + ((st * kStageBytes) >> 4), tp = t0 + (((n & 1) * kTP) >> 4);
    const bool must = sub == 2;
    // polls: bounded like the waits, by the one behind this loop or, before T R,
    // by those inside
    bool again = sub != 1;
#pragma unroll 1
    for (int poll = 0; again; ++poll) {
      uint64_t* const full = &sm.ctl.full[scored % kStages];
      if ((must || step == 0) && scored <= n) {
        if (!wait(full, scored / kStages) || (scored > 0 && !wait(&sm.ctl.d1_empty, scored - 1)))
          return false;
      }
      if (scored < chunks && (sub >= 2 || step == 0 || poll > 0) &&
          __any_sync(0xffffffffu, tc::mbar_ready(full, (scored / kStages) & 1)) &&
          (scored == 0 ||
           __any_sync(0xffffffffu, tc::mbar_ready(&sm.ctl.d1_empty, (scored - 1) & 1)))) {
        tc::fence_after();
        const uint64_t d = kq0 + (((scored % kStages) * kStageBytes) >> 4);
        if (tc::elect()) {                      // [K; Q] K^T
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_ss(tmem + kColD1, d + panel(ks, 0), d + panel(ks, 0), kId, ks > 0);
          tc::commit(&sm.ctl.d1_full);
        }
        __syncwarp();
        ++scored;
      }
      // (chunk n - 1's N has been read: its update, which needed it, is issued)
      if (must && scored > n &&
          (!wait(&sm.ctl.t_full[n & 1], n >> 1) || !wait(&sm.ctl.v_full[st], n / kStages)))
        return false;
      if (tved == n && scored > n &&
          __any_sync(0xffffffffu, tc::mbar_ready(&sm.ctl.t_full[n & 1], (n >> 1) & 1)) &&
          __any_sync(0xffffffffu, tc::mbar_ready(&sm.ctl.v_full[st], (n / kStages) & 1))) {
        tc::fence_after();
        const uint64_t v = v0 + ((st * kStageBytes) >> 4);
        if (tc::elect()) {                      // (T V)^T, V read along dv
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_ss(tmem + kColVN, v + ((ks * 2048) >> 4),
                         tp + ((t * kTBytes + ks * 2048) >> 4), kIdV, (t | ks) > 0);
        }
        __syncwarp();
        ++tved;
      }
      again = must ? tved == n
                   : sub == 0 && (step == 0 ? scored == 0
                                            : poll < 4096 && !__any_sync(0xffffffffu,
                                                  tc::mbar_ready(&sm.ctl.s_full[0], n & 1)));
    }
    if (sub < 2) {
      if (!wait(&sm.ctl.full[st], n / kStages) || !wait(&sm.ctl.s_full[sub], n)) return false;
      // N of the last chunk lies where S^T k goes
      if (sub == 0 && n > 0 && !wait(&sm.ctl.o_full, n - 1)) return false;
      tc::fence_after();
      const uint32_t s0 = tmem + kColS + sub * 64;
      const uint64_t kp = kq + ((sub * kPanel) >> 4);
      if (tc::elect()) {
#pragma unroll
        for (int t = 0; t < 2; ++t)             // S hi, S lo
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)
            tc::mma_ts(tmem + kColKS, s0 + k4 * 16 + t * 8,
                       kp + panel(k4, 0), kId, (sub | t | k4) > 0);
        if (sub == 1) tc::commit(&sm.ctl.ks_full);
      }
      __syncwarp();
      if (sub == 1) {
        if (n > 0 && !wait(&sm.ctl.o_empty, n - 1)) return false;
        tc::fence_after();
        if (tc::elect()) {
#pragma unroll
          for (int t = 0; t < 2; ++t)           // S hi, S lo
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc::mma_ts(tmem + kColQS, tmem + kColS + ks * 16 + t * 8, kq + panel(ks, kC), kId,
                         (t | ks) > 0);
          tc::commit(&sm.ctl.qs_done);
        }
        __syncwarp();
      }
    } else if (sub == 2) {
      if (!wait(&sm.ctl.r_full, n)) return false;
      tc::fence_after();
      if (tc::elect()) {
#pragma unroll
        for (int t = 0; t < 3; ++t)             // R hi T hi, R lo T hi, R hi T lo
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_ts(tmem + kColVN, tmem + kColR + (t == 1 ? 32 : 0) + ks * 8,
                       tp + (((t == 2 ? kTBytes : 0) + ks * 2048) >> 4), kIdT, true);
        tc::commit(&sm.ctl.vn_full);
      }
      __syncwarp();
    } else {
      if (!wait(&sm.ctl.p_full[n & 1], n >> 1) || !wait(&sm.ctl.vd_full, n) ||
          !wait(&sm.ctl.qs_done, n))
        return false;
      tc::fence_after();
      if (tc::elect()) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // K read along dk, 64 at a time
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_ts(tmem + kColS + part * 64, tmem + kColR + t * 32 + ks * 8,
                         kq + ((part * kPanel + ks * 2048) >> 4), kIdT, (t | ks) > 0);
          tc::commit(&sm.ctl.sd_full[part]);
        }
        tc::commit(&sm.ctl.empty[st]);
        // in-chunk outputs: tokens j of a block ks reach the tokens i of that block
        // and of those behind it, i.e. rows [16 ks, 64) of the scores
#pragma unroll
        for (int t = 0; t < 2; ++t)             // N hi P hi, N lo P hi
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_ts(tmem + kColO + ks * kB, tmem + kColN + t * 32 + ks * 8,
                       tp + ((2 * kTBytes + ks * (kB * 128 + 32)) >> 4),
                       tc::idesc(128, kC - ks * kB), (t | ks) > 0);
#pragma unroll
        for (int ks = 0; ks < 3; ++ks)          // N hi P lo, below the diagonal
          tc::mma_ts(tmem + kColO + (ks + 1) * kB, tmem + kColN + ks * 8,
                     tp + ((2 * kTBytes + (3 - ks) * 32) >> 4),
                     tc::idesc(128, kC - (ks + 1) * kB), true);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)          // on it
          tc::mma_ts(tmem + kColO + ks * kB, tmem + kColN + ks * 8,
                     tp + ((3 * kTBytes + ks * 32) >> 4), tc::idesc(128, kB), true);
        tc::commit(&sm.ctl.o_full);
        tc::commit(&sm.ctl.tp_empty[n & 1]);
      }
      __syncwarp();
    }
  }
  return true;
}

template <typename ST>
__global__ void __launch_bounds__(kThreadsC, 1)
    gdn_chunk_kernel(const GdnArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char gdn_dyn[];
  Smem& sm = *reinterpret_cast<Smem*>(
      gdn_dyn + ((1024u - (smem_addr(gdn_dyn) & 1023u)) & 1023u));
  const int tid = threadIdx.x;
  // (read from one lane: values that the compiler then knows to be the same in
  // the whole warp, and keeps in uniform registers, where tcgen05.mma wants them)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // the short sequences' kernel, which needs nothing of this one, may start as
  // SMs become free (22.5 -> 20.1 us for one request of 77 tokens; SMs kept free
  // for it from the start took as much from the chains as it gained)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  order_chains(a, sm, reinterpret_cast<int*>(sm.stage[0]));
  const int chunks = __shfl_sync(0xffffffffu, sm.total, 0);
  if (chunks == 0) return;

  if (tid == 0) {
    Ctl& c = sm.ctl;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&c.full[i], 2);                // rows, gates
      mbar_init(&c.empty[i], 1);
      mbar_init(&c.v_full[i], 1);
      mbar_init(&c.rn_full[i], kOutWarps);
      mbar_init(&c.v_empty[i], kOutWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.gate_empty[i], kPrepWarps + kInvWarps);
      mbar_init(&c.tp_empty[i], 1);
      mbar_init(&c.a_full[i], 2);
      mbar_init(&c.p_full[i], 2);
      mbar_init(&c.t_full[i], kInvWarps);
      mbar_init(&c.a_empty[i], kInvWarps);
      mbar_init(&c.s_full[i], kScanWarps);
      mbar_init(&c.sd_full[i], 1);
    }
    mbar_init(&c.d1_full, 1);
    for (int i = 0; i < kCoefs; ++i) {
      mbar_init(&c.coef_full[i], kPrepWarps);
      mbar_init(&c.coef_empty[i], kScanWarps + kOutWarps);
    }
    mbar_init(&c.prep_meet, kPrepWarps);
    mbar_init(&c.inv_meet, kInvWarps);
    mbar_init(&c.d1_empty, kPrepWarps);
    mbar_init(&c.ks_full, 1);
    mbar_init(&c.qs_done, 1);
    mbar_init(&c.r_full, kScanWarps);
    mbar_init(&c.vn_full, 1);
    mbar_init(&c.vd_full, kScanWarps);
    mbar_init(&c.o_full, 1);
    mbar_init(&c.o_empty, kOutWarps);
    mbar_init(&c.fin, 1);
    fence_mbar_init();
  }
  // blocks of U left of the diagonal are zero in both buffers: rows [16, 64),
  // units before the row's block
  for (int i = tid; i < 2 * 2 * 48 * 8; i += kThreadsC) {
    const int u = i & 7, r = kB + (i >> 3) % 48, m = (i / 384) & 1, b = i / 768;
    if (u < r / kB * 2)
      *reinterpret_cast<uint4*>(sm.tp[b] + m * kTBytes + sw128(r, u)) =
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.ctl.tmem, 0);
  const Wait wait;
  bool ok = true;

  if (warp < kScanWarps) {
    ok = scan_role<ST>(a, sm, wait, tmem);
  } else if (warp < kWarpInv0) {
    more_regs<kRegsPrep>();
    ok = prep_role(a, sm, wait, chunks, tmem);
  } else if (warp < kWarpOut0) {
    if (warp < kWarpMma) {
      ok = inv_role(sm, wait, chunks);
    } else if (warp == kWarpMma) {
      ok = mma_role(sm, wait, chunks, tmem);
      // every product that was issued ends before tensor memory is given back
      if (tc::elect()) tc::commit(&sm.ctl.fin);
      __syncwarp();
      if (!wait(&sm.ctl.fin, 0)) ok = false;
    } else {
      ok = load_role(a, maps, sm, wait);
    }
  } else {
    fewer_regs<kRegsOut>();
    ok = out_role(a, sm, wait, chunks, tmem);
  }
  if (!ok && (tid & 31) == 0) flag_error(a.dev_err, CCONV_DERR_TIMEOUT);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool encode_rows(CUtensorMap* m, const char* p, int64_t cols, int64_t rows, int64_t stride) {
  const EncodeTiledFn enc = encode_fn();
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64u, (cuuint32_t)kC};
  const cuuint32_t step[2] = {1u, 1u};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<char*>(p), dims, strides,
                    box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename ST>
cudaError_t launch_chunk(const GdnArgs& a, cudaStream_t st) {
  constexpr size_t smem = sizeof(Smem) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a block");
  static std::atomic<uint64_t> full;
  const cudaError_t e = mix_full_smem(reinterpret_cast<const void*>(gdn_chunk_kernel<ST>), full);
  if (e != cudaSuccess) return e;
  Maps maps;
  if (!encode_rows(&maps.k, a.k, (int64_t)a.Hk * kD, a.T, a.k_rs) ||
      !encode_rows(&maps.q, a.q, (int64_t)a.Hk * kD, a.T, a.q_rs) ||
      !encode_rows(&maps.v, a.v, (int64_t)a.Hv * kD, a.T, a.v_rs))
    return cudaErrorInvalidValue;
  const int sms = mix_sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  GdnArgs b = a;
  b.st_bytes = sizeof(ST);
  for (int s = 0; s < a.B; s += kMaxSeqs) {     // a launch orders at most kMaxSeqs sequences
    b.B = std::min(kMaxSeqs, a.B - s);
    b.state_idx = a.state_idx + s;
    b.cu = a.cu + s;
    b.has_init = a.has_init ? a.has_init + s : nullptr;
    const int grid = (int)std::min<int64_t>(sms, (int64_t)b.B * a.Hv);
    gdn_chunk_kernel<ST><<<grid, kThreadsC, smem, st>>>(b, maps);
    const cudaError_t le = cudaGetLastError();
    if (le != cudaSuccess) return le;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t gdn_launch_chunk(const GdnArgs& a, int state_dtype, cudaStream_t st) {
  return state_dtype == CCONV_DTYPE_F32 ? launch_chunk<float>(a, st)
                                        : launch_chunk<__nv_bfloat16>(a, st);
}

}  // namespace cconv
