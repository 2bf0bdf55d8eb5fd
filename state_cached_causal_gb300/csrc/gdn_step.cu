// gdn_fwd_varlen and gdn_update: host entry points, and the recurrent kernel
// of the gated delta rule.
//
// A token costs 6*dk*dv flops of a [dk, dv] state that has to come from and go
// to HBM: a decode step is bound by those bytes (64 KB each way for a 128 x
// 128 fp32 head), not by its arithmetic. So a block keeps a tile of the state
// in registers from its load to its store, and takes its tokens past it.
//
// The state's columns are independent of each other: column c of S needs k, q
// and element c of v alone. An item is 32 columns (kCols) of one head of one
// sequence, all dk rows, 128 threads of 4 columns by dk/16 rows: one request of
// 32 heads is 128 items. Blocks, seven an SM, take one item after the other. What
// the next item needs -- its state, its first tokens' q, k, v and gates, and the
// index entries of the item after it -- is requested (cp.async) before they
// work on this one, so that a token meets no load of its own: 112 KB of state are
// on their way to an SM at any time.
//
// What bounds it: HBM, as far as an item's own chain of reductions and barriers
// (5 us) lets seven of them keep it busy. 64 requests of 32 heads of 128 x 128 in
// fp32 (270 MB): 52.3 us, 5.2 TB/s; 128 requests of 4 tokens, a state stored for
// each (1355 MB): 234 us, 5.8 TB/s. With bf16 states, half the bytes and the same
// instructions (68 % of the issue slots): 45.8 and 201 us. On the way: a block an item 57.8 us; items
// one after the other, the state requested ahead 54.4 (247); q, k, v, gates and
// indices ahead too 59.0 with eight blocks of 64 registers, 52.2 with seven of 72,
// 55.6 with six; a division for the head of an item in place of a multiplication
// costs 15 us; eight neighbouring rows a thread in place of every 16th 7 us.
//
// Per token one reduction over the rows gives both products with the old
// state, x = S^T k and y = S^T q, and the rest follows from them:
//   r = beta (v - alpha x),  S' = alpha S + k r^T,  o = alpha y + (q.k) r
// The norms of q and k enter as factors, so that raw q and k are used.
#include "gdn.cuh"

#include <mutex>

namespace cconv {

int mix_sm_count() {
  static int count[64];
  static std::mutex m;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(m);
  if (count[dev] == 0 &&
      cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    count[dev] = 0;
  return count[dev];
}

cudaError_t mix_full_smem(const void* f, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
  cudaFuncAttributes at;
  e = cudaFuncGetAttributes(&at, f);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             227 * 1024 - (int)at.sharedSizeBytes);
  if (e != cudaSuccess)
    cudaGetLastError();                  // this call's error, not the next one's
  else if (dev < 64)
    done |= 1ull << dev;
  return e;
}

namespace {

constexpr int kCols = 32;      // state columns of a block
constexpr int kTok = 4;        // tokens staged at a time
constexpr int kStepBlocks = 7; // of an SM
constexpr int kStepThreads = 128;
constexpr int kStepMax = 8;    // longest sequence of this kernel where the chunked one serves

// What the host's index arrays say of an item, in shared memory.
struct StepDesc {
  int cu[2], acc;              // cu_seqlens of the sequence, or the accepted tokens
  float A_log, dt_bias;        // of the head
  int slot[kMaxSpec + 1];      // state slots: one, or one for each token
};
// The line of items: sequence by sequence, head by head, 2^shift blocks of columns.
struct StepLine {
  int items, shift;
  uint64_t inv;                // 2^64 / Hv, rounded up (0 for Hv = 1)
  __device__ __forceinline__ int seq(int i) const {
    const int j = i >> shift;
    return inv ? (int)__umul64hi((uint64_t)j, inv) : j;
  }
};
struct StepItem {
  int s, h, blk, row0, len, slot_in, slot_out;
  bool skip, init;
};
// Item i: its sequence, head and columns, and the slots to start from and (not
// for gdn_update, which has one for each token) to end in. Reports bad indices.
__device__ __forceinline__ void step_item(const GdnArgs& a, int i, const StepLine& ln,
                                          const StepDesc& d, bool has_init, bool report,
                                          StepItem& t) {
  t.s = ln.seq(i);
  t.h = (i >> ln.shift) - t.s * a.Hv;
  t.blk = i & ((1 << ln.shift) - 1);
  t.skip = true;
  t.init = false;
  const bool first = report && t.blk == 0 && t.h == 0 && threadIdx.x == 0;
  if (a.cu) {
    t.row0 = d.cu[0];
    t.len = d.cu[1] - d.cu[0];
    if (t.row0 < 0 || d.cu[1] < t.row0 || d.cu[1] > a.T) {
      if (first) flag_error(a.dev_err, CCONV_DERR_CU_SEQLENS);
      return;
    }
  } else {
    t.row0 = t.s * a.q_len;
    t.len = a.q_len;
  }
  if (a.max_len > 0 && t.len > a.max_len) return;
  bool bad = false;
  if (a.cu) {
    t.slot_in = t.slot_out = d.slot[0];
    bad = t.slot_in >= a.num_slots;
  } else {
    int acc = 1;
    if (a.q_len > 1) {
      acc = d.acc;
      if (acc < 1 || acc > a.q_len) {
        if (first) flag_error(a.dev_err, CCONV_DERR_NUM_ACCEPTED);
        return;
      }
    }
    for (int k = 0; k < a.q_len; ++k) bad |= d.slot[k] >= a.num_slots;
    t.slot_in = d.slot[acc - 1];
    t.slot_out = -1;
  }
  if (bad) {
    if (first) flag_error(a.dev_err, CCONV_DERR_SLOT_RANGE);
    return;
  }
  t.init = t.slot_in >= 0 && has_init;
  // an empty sequence leaves its slot, or clears it
  t.skip = t.len == 0 && (t.init || t.slot_out < 0);
}

template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}

template <typename T, typename ST, int DK>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks)
gdn_step_kernel(const GdnArgs a, const int dv, const StepLine ln) {
  constexpr int R = DK / 16;                     // rows of a thread
  constexpr int kUnit = 4 * sizeof(ST);          // bytes of its 4 columns of a row
  constexpr int kRow = 2 * DK + kCols;           // a token's k, q and columns of v
  constexpr int kUK = DK * sizeof(T) / 16, kUV = kCols * sizeof(T) / 16, kUnits = 2 * kUK + kUV;
  __shared__ __align__(16) unsigned char stage[R][kStepThreads][kUnit];
  __shared__ __align__(16) unsigned char toks[2][kTok][kRow * sizeof(T)];
  __shared__ StepDesc desc[3];
  __shared__ float sgate[kTok][2];
  __shared__ float4 sred[2][2][4][8];            // [token parity][x, y][warp][column quad]
  __shared__ float4 ssum[2][4];                  // [token parity][warp]: k.k, q.q, q.k
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = ln.items, rep = a.Hv / a.Hk;
  const int cq = (lane & 7) * 4;                     // the thread's 4 columns of the item
  const int rg = warp * 4 + (lane >> 3);             // rows rg + 16 i
  auto state_of = [&](const StepItem& t, int slot) {
    return reinterpret_cast<ST*>(a.st) + (int64_t)slot * a.st_slot + (int64_t)t.h * a.st_head +
           t.blk * kCols + cq + rg * dv;
  };
  // Requests: of item i's description, of an item's state, of a few of its tokens.
  auto describe = [&](int i, StepDesc& d) {
    if (i >= items) return;
    const int s = ln.seq(i), h = (i >> ln.shift) - s * a.Hv, n = a.cu ? 1 : a.q_len;
    auto get = [](void* to, const void* from) { cp_async_small<4>(smem_addr(to), from); };
    if (tid < n) get(&d.slot[tid], a.state_idx + (int64_t)s * n + tid);
    if (tid >= 32 && tid < 34 && a.cu) get(&d.cu[tid - 32], a.cu + s + tid - 32);
    if (tid == 64 && a.q_len > 1) get(&d.acc, a.num_acc + s);
    if (tid == 96) get(&d.A_log, a.A_log + h);
    if (tid == 97) get(&d.dt_bias, a.dt_bias + h);
  };
  auto starts = [&](int i) {
    return i < items && (!a.has_init || a.has_init[ln.seq(i)] != 0);
  };
  auto request = [&](const StepItem& t) {
    if (t.skip || !t.init) return;
    const ST* p = state_of(t, t.slot_in);
#pragma unroll
    for (int i = 0; i < R; ++i) cp_async_small<kUnit>(smem_addr(stage[i][tid]), p + 16 * i * dv);
  };
  float ga = 0.0f, gb = 0.0f;                    // raw gates of the next batch's token `tid`
  auto tokens = [&](const StepItem& t, int t0, int buf) {
    if (t.skip) return;
    const int n = min(kTok, t.len - t0);
    const int64_t row0 = (int64_t)t.row0 + t0;
    const int hk = rep == 1 ? t.h : t.h / rep;
    for (int u = tid; u < n * kUnits; u += kStepThreads) {
      const int j = u / kUnits, w = u - j * kUnits;
      const int64_t row = row0 + j;
      const char* p = w < kUK ? a.k + (row * a.k_rs + hk * DK) * sizeof(T) + w * 16
                      : w < 2 * kUK
                          ? a.q + (row * a.q_rs + hk * DK) * sizeof(T) + (w - kUK) * 16
                          : a.v + (row * a.v_rs + t.h * dv + t.blk * kCols) * sizeof(T) +
                                (w - 2 * kUK) * 16;
      cp_async_small<16>(smem_addr(toks[buf][j]) + w * 16, p);
    }
    if (tid < n) {
      ga = elem<T>(reinterpret_cast<const T*>(a.a), (row0 + tid) * a.a_rs + t.h);
      gb = elem<T>(reinterpret_cast<const T*>(a.b), (row0 + tid) * a.b_rs + t.h);
    }
  };
  auto arrived = [&] {
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
  };
  const int step = gridDim.x;
  describe(blockIdx.x, desc[0]);
  describe(blockIdx.x + step, desc[1]);
  bool ini = starts(blockIdx.x), ini_nx = starts(blockIdx.x + step);
  arrived();
  {
    StepItem it;
    step_item(a, blockIdx.x, ln, desc[0], ini, false, it);
    request(it);
    tokens(it, 0, 0);
  }
  int pb = 0, d = 0;
  arrived();
#pragma unroll 1
  for (int i = blockIdx.x; i < items; i += step) {
    StepItem it;
    step_item(a, i, ln, desc[d], ini, true, it);
    float S[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (it.init)
        load4<ST>(reinterpret_cast<const ST*>(stage[r][tid]), S[r]);
      else
        S[r][0] = S[r][1] = S[r][2] = S[r][3] = 0.0f;
    }
    const int dn = d == 2 ? 0 : d + 1, d2 = dn == 2 ? 0 : dn + 1;
    const bool more = i + step < items;
    bool ini_n2 = false;
    bool last;
    int t0 = 0;
#pragma unroll 1
    do {
      const int n = it.skip ? 0 : min(kTok, it.len - t0);
      last = it.skip || t0 + kTok >= it.len;
      if (tid < n) {
        sgate[tid][0] = expf(gdn_log_decay(ga, desc[d].A_log, desc[d].dt_bias));
        sgate[tid][1] = gdn_beta(gb);
      }
      // requests of what comes next, in flight while these tokens are worked on
      if (t0 == 0 || last) {
        StepItem nx;
        nx.skip = true;
        if (more) step_item(a, i + step, ln, desc[dn], ini_nx, false, nx);
        if (t0 == 0) {
          request(nx);
          describe(i + 2 * step, desc[d2]);
          ini_n2 = starts(i + 2 * step);
        }
        if (last) tokens(nx, 0, pb ^ 1);
      }
      if (!last) tokens(it, t0 + kTok, pb ^ 1);
      cp_async_commit();
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        const T* const tk = reinterpret_cast<const T*>(toks[pb][t]);
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f}, kr[R];
        float kk = 0.0f, qq = 0.0f, qk = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          kr[r] = elem<T>(tk, rg + 16 * r);
          const float qv = elem<T>(tk, DK + rg + 16 * r);
          kk = fmaf(kr[r], kr[r], kk);
          qq = fmaf(qv, qv, qq);
          qk = fmaf(qv, kr[r], qk);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            x[c] = fmaf(kr[r], S[r][c], x[c]);
            y[c] = fmaf(qv, S[r][c], y[c]);
          }
        }
#pragma unroll
        for (int m = 8; m < 32; m <<= 1) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            x[c] += __shfl_xor_sync(0xffffffffu, x[c], m);
            y[c] += __shfl_xor_sync(0xffffffffu, y[c], m);
          }
          kk += __shfl_xor_sync(0xffffffffu, kk, m);
          qq += __shfl_xor_sync(0xffffffffu, qq, m);
          qk += __shfl_xor_sync(0xffffffffu, qk, m);
        }
        // two copies of the exchange by token parity: one barrier a token
        if (lane < 8) {
          sred[t & 1][0][warp][lane] = make_float4(x[0], x[1], x[2], x[3]);
          sred[t & 1][1][warp][lane] = make_float4(y[0], y[1], y[2], y[3]);
        }
        if (lane == 8) ssum[t & 1][warp] = make_float4(kk, qq, qk, 0.0f);
        __syncthreads();
        float4 X = make_float4(0.f, 0.f, 0.f, 0.f), Y = X;
        kk = qq = qk = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 u = sred[t & 1][0][w][lane & 7], z = sred[t & 1][1][w][lane & 7];
          X.x += u.x, X.y += u.y, X.z += u.z, X.w += u.w;
          Y.x += z.x, Y.y += z.y, Y.z += z.z, Y.w += z.w;
          const float4 p = ssum[t & 1][w];
          kk += p.x, qq += p.y, qk += p.z;
        }
        const float rk = a.l2norm ? 1.0f / sqrtf(kk + kGdnNormEps) : 1.0f;
        const float rq = (a.l2norm ? 1.0f / sqrtf(qq + kGdnNormEps) : 1.0f) * a.scale;
        const float al = sgate[t][0], be = sgate[t][1];
        const float ark = al * rk, arq = al * rq, kq = rq * rk * qk;
        float vt[4];
        load4<T>(tk + 2 * DK + cq, vt);
        const float r4[4] = {be * (vt[0] - ark * X.x), be * (vt[1] - ark * X.y),
                             be * (vt[2] - ark * X.z), be * (vt[3] - ark * X.w)};
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float kn = kr[r] * rk;
#pragma unroll
          for (int c = 0; c < 4; ++c) S[r][c] = fmaf(kn, r4[c], al * S[r][c]);
        }
        if (tid < 8) {
          const float o[4] = {fmaf(kq, r4[0], arq * Y.x), fmaf(kq, r4[1], arq * Y.y),
                              fmaf(kq, r4[2], arq * Y.z), fmaf(kq, r4[3], arq * Y.w)};
          store4<T>(reinterpret_cast<T*>(a.out) + ((int64_t)it.row0 + t0 + t) * a.out_rs +
                        (int64_t)it.h * dv + it.blk * kCols + cq, o);
        }
        const int so = a.cu ? (t0 + t + 1 == it.len ? it.slot_out : -1) : desc[d].slot[t0 + t];
        if (so >= 0) {
          ST* p = state_of(it, so);
#pragma unroll
          for (int r = 0; r < R; ++r) store4<ST>(p + 16 * r * dv, S[r]);
        }
      }
      pb ^= 1;
      t0 += kTok;
      arrived();
    } while (!last);
    if (!it.skip && it.len == 0) {      // cleared
      ST* p = state_of(it, it.slot_out);
#pragma unroll
      for (int r = 0; r < R; ++r) store4<ST>(p + 16 * r * dv, S[r]);
    }
    ini = ini_nx;
    ini_nx = ini_n2;
    d = dn;
  }
  // This kernel may run beside the chunked one, which was launched before it:
  // what follows both waits for this grid alone, so one of its blocks waits for
  // the other grid's end. (No block of that one waits for anything here.)
  if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T, typename ST>
cudaError_t launch_step_t(const GdnArgs& a, int dk, int dv, cudaStream_t st) {
  const int sms = mix_sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  const int items = a.B * a.Hv * (dv / kCols);     // (at most 2^31 - 1: a host check)
  const StepLine ln = {items, dv == 64 ? 1 : 2, a.Hv == 1 ? 0 : ~0ull / (unsigned)a.Hv + 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(items, sms * kStepBlocks));
  cfg.blockDim = dim3(kStepThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.max_len > 0 ? 1 : 0;            // beside the chunked kernel
  return dk == 64 ? cudaLaunchKernelEx(&cfg, gdn_step_kernel<T, ST, 64>, a, dv, ln)
                  : cudaLaunchKernelEx(&cfg, gdn_step_kernel<T, ST, 128>, a, dv, ln);
}

}  // namespace

cudaError_t gdn_launch_step(const GdnArgs& a, int dtype, int state_dtype, int dk, int dv,
                            cudaStream_t st) {
  if (dtype == CCONV_DTYPE_F32)
    return state_dtype == CCONV_DTYPE_F32 ? launch_step_t<float, float>(a, dk, dv, st)
                                          : launch_step_t<float, __nv_bfloat16>(a, dk, dv, st);
  return state_dtype == CCONV_DTYPE_F32
             ? launch_step_t<__nv_bfloat16, float>(a, dk, dv, st)
             : launch_step_t<__nv_bfloat16, __nv_bfloat16>(a, dk, dv, st);
}

// Checks of everything the two entry points share; fills `o`.
static int gdn_args(const void* q, int64_t q_rs, const void* k, int64_t k_rs, const void* v,
                    int64_t v_rs, const void* a, int64_t a_rs, const void* b, int64_t b_rs,
                    const float* A_log, const float* dt_bias, const gdn_state_t& st,
                    const int32_t* state_idx, const uint8_t* has_init, int32_t num_seqs,
                    int64_t rows, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv, float scale,
                    int32_t l2norm, int32_t dtype, void* out, int64_t out_rs, int32_t* dev_err,
                    GdnArgs& o) {
  const int e = mix_dtype_bytes(dtype), se = mix_dtype_bytes(st.dtype);
  if (e == 0 || se == 0) return CCONV_ERR_INVALID;
  if (num_seqs < 0 || rows < 0 || rows > INT32_MAX || Hk <= 0 || Hv <= 0 || Hv % Hk != 0 ||
      dk <= 0 || dv <= 0)
    return CCONV_ERR_INVALID;
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return CCONV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return CCONV_OK;
  const int V = 16 / e;
  if (!A_log || !dt_bias || !state_idx) return CCONV_ERR_INVALID;
  if (rows > 0) {
    if (!mix_rows_ok(q, q_rs, (int64_t)Hk * dk, V) || !mix_rows_ok(k, k_rs, (int64_t)Hk * dk, V) ||
        !mix_rows_ok(v, v_rs, (int64_t)Hv * dv, V) ||
        !mix_rows_ok(out, out_rs, (int64_t)Hv * dv, V))
      return CCONV_ERR_INVALID;
    if (!a || !b || a_rs < Hv || b_rs < Hv || reinterpret_cast<uintptr_t>(a) % e ||
        reinterpret_cast<uintptr_t>(b) % e)
      return CCONV_ERR_INVALID;
  }
  if (!st.p || !mix_aligned16(st.p) || st.num_slots <= 0 || st.s_head < (int64_t)dk * dv ||
      st.s_slot <= 0 || st.s_head % (16 / se) || st.s_slot % (16 / se))
    return CCONV_ERR_INVALID;
  // items of the recurrent kernel (and a grid more) are counted in 32 bits
  if ((int64_t)num_seqs * Hv * (dv / kCols) > INT32_MAX / 2) return CCONV_ERR_INVALID;
  o.q = static_cast<const char*>(q);
  o.k = static_cast<const char*>(k);
  o.v = static_cast<const char*>(v);
  o.a = static_cast<const char*>(a);
  o.b = static_cast<const char*>(b);
  o.q_rs = q_rs, o.k_rs = k_rs, o.v_rs = v_rs, o.a_rs = a_rs, o.b_rs = b_rs, o.out_rs = out_rs;
  o.A_log = A_log;
  o.dt_bias = dt_bias;
  o.out = static_cast<char*>(out);
  o.st = static_cast<char*>(st.p);
  o.st_slot = st.s_slot;
  o.st_head = st.s_head;
  o.num_slots = st.num_slots;
  o.state_idx = state_idx;
  o.has_init = has_init;
  o.B = num_seqs;
  o.T = (int32_t)rows;
  o.Hk = Hk;
  o.Hv = Hv;
  o.scale = scale;
  o.l2norm = l2norm != 0;
  o.dev_err = dev_err;
  o.max_len = 0;
  return CCONV_OK;
}

}  // namespace cconv

using namespace cconv;

extern "C" int gdn_fwd_varlen(const void* q, int64_t q_row_stride, const void* k,
                              int64_t k_row_stride, const void* v, int64_t v_row_stride,
                              const void* a, int64_t a_row_stride, const void* b,
                              int64_t b_row_stride, const float* A_log, const float* dt_bias,
                              gdn_state_t states, const int32_t* state_idx,
                              const int32_t* cu_seqlens, const uint8_t* has_init,
                              int32_t num_seqs, int32_t num_tokens, int32_t num_k_heads,
                              int32_t num_v_heads, int32_t dk, int32_t dv, float scale,
                              int32_t qk_l2norm, int32_t dtype, void* out,
                              int64_t out_row_stride, int32_t* dev_err, cconv_stream_t stream) {
  GdnArgs o;
  const int rc = gdn_args(q, q_row_stride, k, k_row_stride, v, v_row_stride, a, a_row_stride, b,
                          b_row_stride, A_log, dt_bias, states, state_idx, has_init, num_seqs,
                          num_tokens, num_k_heads, num_v_heads, dk, dv, scale, qk_l2norm, dtype,
                          out, out_row_stride, dev_err, o);
  if (rc != CCONV_OK || num_seqs == 0) return rc;
  if (!cu_seqlens) return CCONV_ERR_INVALID;
  o.cu = cu_seqlens;
  o.num_acc = nullptr;
  o.q_len = 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // sequences of more than kStepMax tokens go chunk by chunk where there is a
  // kernel for it; a call of no more tokens than that has none
  const bool chunked = dtype == CCONV_DTYPE_BF16 && dk == 128 && dv == 128 &&
                       num_tokens > kStepMax;
  if (chunked) {
    o.max_len = kStepMax;
    if (gdn_launch_chunk(o, states.dtype, st) != cudaSuccess) return CCONV_ERR_LAUNCH;
  }
  return gdn_launch_step(o, dtype, states.dtype, dk, dv, st) == cudaSuccess ? CCONV_OK
                                                                           : CCONV_ERR_LAUNCH;
}

extern "C" int gdn_update(const void* q, int64_t q_row_stride, const void* k,
                          int64_t k_row_stride, const void* v, int64_t v_row_stride,
                          const void* a, int64_t a_row_stride, const void* b,
                          int64_t b_row_stride, const float* A_log, const float* dt_bias,
                          gdn_state_t states, const int32_t* state_idx, int32_t num_seqs,
                          int32_t n_spec, const int32_t* num_accepted, const uint8_t* has_init,
                          int32_t num_k_heads, int32_t num_v_heads, int32_t dk, int32_t dv,
                          float scale, int32_t qk_l2norm, int32_t dtype, void* out,
                          int64_t out_row_stride, int32_t* dev_err, cconv_stream_t stream) {
  if (n_spec < 0) return CCONV_ERR_INVALID;
  if (n_spec > kMaxSpec) return CCONV_ERR_UNSUPPORTED;
  GdnArgs o;
  const int rc = gdn_args(q, q_row_stride, k, k_row_stride, v, v_row_stride, a, a_row_stride, b,
                          b_row_stride, A_log, dt_bias, states, state_idx, has_init, num_seqs,
                          (int64_t)num_seqs * (1 + n_spec), num_k_heads, num_v_heads, dk, dv,
                          scale, qk_l2norm, dtype, out, out_row_stride, dev_err, o);
  if (rc != CCONV_OK || num_seqs == 0) return rc;
  if (n_spec > 0 && !num_accepted) return CCONV_ERR_INVALID;
  o.cu = nullptr;
  o.num_acc = num_accepted;
  o.q_len = 1 + n_spec;
  const cudaError_t e = gdn_launch_step(o, dtype, states.dtype, dk, dv,
                                        reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}
