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
// 32 heads is 128 items. Blocks, eight an SM, take one item after the other, and
// request the next item's state (cp.async, each thread into its own place in
// shared memory, so that no barrier is needed) before they work on this one:
// 128 KB are on their way to an SM at any time. Without that, one block an item
// and as many a SM, a decode step of 64 requests took 57.8 us (4.7 TB/s).
//
// Per token one reduction over the rows gives both products with the old
// state, x = S^T k and y = S^T q, and the rest follows from them:
//   r = beta (v - alpha x),  S' = alpha S + k r^T,  o = alpha y + (q.k) r
// The norms of q and k enter as factors, so that raw q and k are staged.
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

namespace {

constexpr int kCols = 32;      // state columns of a block
constexpr int kTok = 4;        // tokens staged at a time
constexpr int kStepBlocks = 8; // of an SM
constexpr int kStepThreads = 128;
constexpr int kStepMax = 8;    // longest sequence of this kernel where the chunked one serves

struct StepItem {
  int s, h, blk, row0, len, slot_in, slot_out;
  bool skip, init;
};
// Item i: its sequence, head and columns, and the slots to start from and (not
// for gdn_update, which has one for each token) to end in. Reports bad indices.
__device__ __forceinline__ void step_item(const GdnArgs& a, int i, int nblk, StepItem& t) {
  t.blk = i % nblk;
  t.h = i / nblk % a.Hv;
  t.s = i / nblk / a.Hv;
  t.skip = true;
  t.init = false;
  const bool first = t.blk == 0 && t.h == 0 && threadIdx.x == 0;
  if (!gdn_bounds(a, t.s, t.row0, t.len)) {
    if (first) flag_error(a.dev_err, CCONV_DERR_CU_SEQLENS);
    return;
  }
  if (a.max_len > 0 && t.len > a.max_len) return;
  bool bad = false;
  if (a.cu) {
    t.slot_in = t.slot_out = a.state_idx[t.s];
    bad = t.slot_in >= a.num_slots;
  } else {
    const int32_t* idx = a.state_idx + (int64_t)t.s * a.q_len;
    int acc = 1;
    if (a.q_len > 1) {
      acc = a.num_acc[t.s];
      if (acc < 1 || acc > a.q_len) {
        if (first) flag_error(a.dev_err, CCONV_DERR_NUM_ACCEPTED);
        return;
      }
    }
    for (int k = 0; k < a.q_len; ++k) bad |= idx[k] >= a.num_slots;
    t.slot_in = idx[acc - 1];
    t.slot_out = -1;
  }
  if (bad) {
    if (first) flag_error(a.dev_err, CCONV_DERR_SLOT_RANGE);
    return;
  }
  t.init = t.slot_in >= 0 && (!a.has_init || a.has_init[t.s]);
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
gdn_step_kernel(const GdnArgs a, const int dv, const int items) {
  constexpr int R = DK / 16;                     // rows of a thread
  constexpr int kUnit = 4 * sizeof(ST);          // bytes of its 4 columns of a row
  __shared__ __align__(16) unsigned char stage[R][kStepThreads][kUnit];
  __shared__ float sk[kTok][DK], sq[kTok][DK];   // raw k and q of the staged tokens
  __shared__ float sv[kTok][kCols];
  __shared__ float spart[2][3][4][kTok];          // sums of squares and q.k by warp
  __shared__ float sgate[kTok][2];
  __shared__ float4 sred[2][2][4][8];            // [token parity][x, y][warp][column quad]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nblk = dv / kCols;
  const int cq = (lane & 7) * 4;                     // the thread's 4 columns of the item
  const int rg = warp * 4 + (lane >> 3);             // rows rg + 16 i
  auto state_of = [&](const StepItem& t, int slot) {
    return reinterpret_cast<ST*>(a.st) + (int64_t)slot * a.st_slot + (int64_t)t.h * a.st_head +
           t.blk * kCols + cq + (int64_t)rg * dv;
  };
  auto request = [&](const StepItem& t) {
    if (t.skip || !t.init) return;
    const ST* p = state_of(t, t.slot_in);
#pragma unroll
    for (int i = 0; i < R; ++i) cp_async_small<kUnit>(smem_addr(stage[i][tid]), p + 16 * i * dv);
  };
  StepItem it, nx;
  step_item(a, blockIdx.x, nblk, nx);
  request(nx);
  int pb = 0;
#pragma unroll 1
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    it = nx;
    cp_async_commit();
    cp_async_wait<0>();
    float S[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (it.init)
        load4<ST>(reinterpret_cast<const ST*>(stage[r][tid]), S[r]);
      else
        S[r][0] = S[r][1] = S[r][2] = S[r][3] = 0.0f;
    }
    if (i + (int)gridDim.x < items) {
      step_item(a, i + gridDim.x, nblk, nx);
      request(nx);
    }
    if (it.skip) continue;
    const int hk = it.h / (a.Hv / a.Hk);
    const T* const qp = reinterpret_cast<const T*>(a.q) + (int64_t)hk * DK;
    const T* const kp = reinterpret_cast<const T*>(a.k) + (int64_t)hk * DK;
    const T* const vp = reinterpret_cast<const T*>(a.v) + (int64_t)it.h * dv + it.blk * kCols;
#pragma unroll 1
    for (int t0 = 0; t0 < it.len; t0 += kTok) {
      const int n = min(kTok, it.len - t0);
      pb ^= 1;
      __syncthreads();   // the last tokens' reads are done
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        const int64_t row = (int64_t)it.row0 + t0 + t;
        float kk = 0.0f, qq = 0.0f, qk = 0.0f;
        if (DK == kStepThreads || tid < DK) {
          const float kv = elem<T>(kp, row * a.k_rs + tid), qv = elem<T>(qp, row * a.q_rs + tid);
          sk[t][tid] = kv;
          sq[t][tid] = qv;
          kk = kv * kv;
          qq = qv * qv;
          qk = qv * kv;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          kk += __shfl_xor_sync(0xffffffffu, kk, d);
          qq += __shfl_xor_sync(0xffffffffu, qq, d);
          qk += __shfl_xor_sync(0xffffffffu, qk, d);
        }
        if (lane == 0) {
          spart[pb][0][warp][t] = kk;
          spart[pb][1][warp][t] = qq;
          spart[pb][2][warp][t] = qk;
        }
      }
      if (tid < n * kCols)
        sv[tid / kCols][tid % kCols] =
            elem<T>(vp, ((int64_t)it.row0 + t0 + tid / kCols) * a.v_rs + tid % kCols);
      if (tid < n) {
        const int64_t row = (int64_t)it.row0 + t0 + tid;
        sgate[tid][0] = expf(gdn_log_decay(
            elem<T>(reinterpret_cast<const T*>(a.a), row * a.a_rs + it.h), a.A_log[it.h],
            a.dt_bias[it.h]));
        sgate[tid][1] = gdn_beta(elem<T>(reinterpret_cast<const T*>(a.b), row * a.b_rs + it.h));
      }
      __syncthreads();
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f}, kr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          kr[r] = sk[t][rg + 16 * r];
          const float qv = sq[t][rg + 16 * r];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            x[c] = fmaf(kr[r], S[r][c], x[c]);
            y[c] = fmaf(qv, S[r][c], y[c]);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] += __shfl_xor_sync(0xffffffffu, x[c], 8);
          y[c] += __shfl_xor_sync(0xffffffffu, y[c], 8);
          x[c] += __shfl_xor_sync(0xffffffffu, x[c], 16);
          y[c] += __shfl_xor_sync(0xffffffffu, y[c], 16);
        }
        // two copies of the exchange by token parity: one barrier a token
        if (lane < 8) {
          sred[t & 1][0][warp][lane] = make_float4(x[0], x[1], x[2], x[3]);
          sred[t & 1][1][warp][lane] = make_float4(y[0], y[1], y[2], y[3]);
        }
        __syncthreads();
        float4 X = make_float4(0.f, 0.f, 0.f, 0.f), Y = X;
        float kk = 0.0f, qq = 0.0f, qk = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 u = sred[t & 1][0][w][lane & 7], z = sred[t & 1][1][w][lane & 7];
          X.x += u.x, X.y += u.y, X.z += u.z, X.w += u.w;
          Y.x += z.x, Y.y += z.y, Y.z += z.z, Y.w += z.w;
          kk += spart[pb][0][w][t];
          qq += spart[pb][1][w][t];
          qk += spart[pb][2][w][t];
        }
        const float rk = a.l2norm ? 1.0f / sqrtf(kk + kGdnNormEps) : 1.0f;
        const float rq = (a.l2norm ? 1.0f / sqrtf(qq + kGdnNormEps) : 1.0f) * a.scale;
        const float al = sgate[t][0], be = sgate[t][1];
        const float ark = al * rk, arq = al * rq, kq = rq * rk * qk;
        const float* vt = &sv[t][cq];
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
        const int so = a.cu ? (t0 + t + 1 == it.len ? it.slot_out : -1)
                            : a.state_idx[(int64_t)it.s * a.q_len + t0 + t];
        if (so >= 0) {
          ST* p = state_of(it, so);
#pragma unroll
          for (int r = 0; r < R; ++r) store4<ST>(p + 16 * r * dv, S[r]);
        }
      }
    }
    if (it.len == 0) {      // cleared
      ST* p = state_of(it, it.slot_out);
#pragma unroll
      for (int r = 0; r < R; ++r) store4<ST>(p + 16 * r * dv, S[r]);
    }
  }
}

template <typename T, typename ST>
cudaError_t launch_step_t(const GdnArgs& a, int dk, int dv, cudaStream_t st) {
  const int sms = mix_sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  const int items = a.B * a.Hv * (dv / kCols);     // (at most 2^31 - 1: a host check)
  const int grid = std::min(items, sms * kStepBlocks);
  if (dk == 64)
    gdn_step_kernel<T, ST, 64><<<grid, kStepThreads, 0, st>>>(a, dv, items);
  else
    gdn_step_kernel<T, ST, 128><<<grid, kStepThreads, 0, st>>>(a, dv, items);
  return cudaGetLastError();
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
