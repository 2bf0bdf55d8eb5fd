// Entry point attn_decode: host side, the plain-arithmetic kernel and the join
// of split results. The split is described in attn_decode.cuh.
//
// attn_kernel keeps one softmax pass over the tiles: K and V of 32 positions go
// to shared memory, each warp scores two of up to kRows query rows (lane =
// position), and the threads hold kRows weighted sums of their columns of V.
// All rows of a kv head read its K and V once.
#include "attn_decode.cuh"

#include <math.h>

namespace cconv {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;
constexpr int kRows = 8;          // query rows of a block

template <typename T, int D>
struct AttnSmem {
  float k[kTile][D + 4];
  float v[kTile][D];
  float q[kRows][D];
  float p[kRows][kTile];
  float corr[kRows];
  int64_t scan[kThreads + 4];
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_kernel(const AttnArgs a) {
  constexpr int V = Elem<T>::V, E = Elem<T>::bytes;
  constexpr int CD = (D + kThreads - 1) / kThreads;   // columns of a thread
  extern __shared__ uint4 attn_dyn[];
  AttnSmem<T, D>& sm = *reinterpret_cast<AttnSmem<T, D>*>(attn_dyn);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  AttnRun run;
  if (!attn_split<kThreads>(a, kTile, sm.scan, run)) return;
  const int rows_all = a.G * a.q_len;
  while (run.p < run.end) {
    const AttnSeg sg = attn_segment(a, kTile, run);
    if (tid == 0) attn_note(a, sg, run);
    attn_advance(a, sg, run);
    if (sg.len < 0) {
      if (tid == 0) flag_error(a.dev_err, CCONV_DERR_SEQ_LEN);
      continue;
    }
    const int hkv = sg.unit / a.rblocks, r0 = sg.unit % a.rblocks * kRows;
    const int nr = min(kRows, rows_all - r0);
    // row r is token (r0 + r) / G of the request, head hkv * G + (r0 + r) % G
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kThreads) {
      const int r = i / D, c = i % D, rr = r0 + r;
      float x = 0.0f;
      if (r < nr)
        x = a.scale * load_f32<T>(a.q, ((int64_t)sg.b * a.q_len + rr / a.G) * a.q_rs +
                                           (int64_t)(hkv * a.G + rr % a.G) * D + c);
      sm.q[r][c] = x;
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, acc[CD][kRows];
#pragma unroll
    for (int c = 0; c < CD; ++c)
#pragma unroll
      for (int r = 0; r < kRows; ++r) acc[c][r] = 0.0f;
    for (int j = sg.j0; j < sg.j1; ++j) {
      const int t0 = j * kTile;
      __syncthreads();
      constexpr int UPR = D / V;                       // 16-byte units a row
      for (int i = tid; i < kTile * UPR; i += kThreads) {
        const int t = i / UPR, u = i % UPR, pos = t0 + t;
        int page = -1;
        if (pos < sg.len) {
          page = a.table[(int64_t)sg.b * a.table_rs + pos / a.page_size];
          if (page < 0 || page >= a.num_pages) {
            flag_error(a.dev_err, CCONV_DERR_PAGE);
            page = -1;
          }
        }
        float fk[V], fv[V];
        if (page >= 0) {
          const int64_t off = ((int64_t)page * a.s_page + (pos % a.page_size) * a.s_tok +
                               (int64_t)hkv * a.s_head + u * V) * E;
          unpack16<T>(ldg16(a.kc + off), fk);
          unpack16<T>(ldg16(a.vc + off), fv);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) fk[e] = fv[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sm.k[t][u * V + e] = fk[e];
          sm.v[t][u * V + e] = fv[e];
        }
      }
      __syncthreads();
      // scores: this lane's position, the warp's two rows
      float s[2] = {0.0f, 0.0f};
#pragma unroll 8
      for (int c = 0; c < D; c += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[lane][c]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[warp * 2 + i][c]);
          s[i] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[i]))));
        }
      }
      const int pos = t0 + lane;
      bool there = pos < sg.len;
      if (there) {
        const int page = a.table[(int64_t)sg.b * a.table_rs + pos / a.page_size];
        there = page >= 0 && page < a.num_pages;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = warp * 2 + i;
        const int seen = sg.len - a.q_len + 1 + (r0 + r) / a.G;   // positions this row sees
        const float x = (there && r < nr && pos < seen) ? s[i] : -INFINITY;
        float mx = x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx);
        const float p = mn == -INFINITY ? 0.0f : expf(x - mn);
        const float corr = mn == -INFINITY ? 1.0f : expf(m[i] - mn);
        float ps = p;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, d);
        l[i] = l[i] * corr + ps;
        m[i] = mn;
        sm.p[r][lane] = p;
        if (lane == 0) sm.corr[r] = corr;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float corr = sm.corr[r];
#pragma unroll
        for (int c = 0; c < CD; ++c) acc[c][r] *= corr;
      }
      if (tid < D)
#pragma unroll 4
        for (int t = 0; t < kTile; ++t)
#pragma unroll
          for (int c = 0; c < CD; ++c) {
            const float v = sm.v[t][tid + c * kThreads];
#pragma unroll
            for (int r = 0; r < kRows; ++r) acc[c][r] = fmaf(sm.p[r][t], v, acc[c][r]);
          }
    }
    if (sg.whole) {
      __syncthreads();
      if (lane == 0) {
        sm.corr[warp * 2] = l[0];
        sm.corr[warp * 2 + 1] = l[1];
      }
      __syncthreads();
      if (tid < D)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r < nr) {
            const int rr = r0 + r;
            const float inv = sm.corr[r] > 0.0f ? 1.0f / sm.corr[r] : 0.0f;
            T* o = reinterpret_cast<T*>(a.out) + ((int64_t)sg.b * a.q_len + rr / a.G) * a.out_rs +
                   (int64_t)(hkv * a.G + rr % a.G) * D;
#pragma unroll
            for (int c = 0; c < CD; ++c) {
              const auto raw = f32_to_raw<T>(acc[c][r] * inv);
              *reinterpret_cast<std::remove_const_t<decltype(raw)>*>(o + tid + c * kThreads) = raw;
            }
          }
      if (a.lse && lane < 2) {
        const int r = warp * 2 + lane, rr = r0 + r;
        if (r < nr)
          a.lse[((int64_t)sg.b * a.q_len + rr / a.G) * a.Hq + hkv * a.G + rr % a.G] =
              l[lane] > 0.0f ? m[lane] + logf(l[lane]) : -INFINITY;
      }
    } else {
      float* part = attn_part(a, sg, D);
      if (tid < D)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int c = 0; c < CD; ++c) part[r * (D + 2) + tid + c * kThreads] = acc[c][r];
      if (lane < 2) {
        part[(warp * 2 + lane) * (D + 2) + D] = m[lane];
        part[(warp * 2 + lane) * (D + 2) + D + 1] = l[lane];
      }
    }
  }
}

// Joins the parts of a cut unit, one block a unit: a thread a column, rows in
// turn. Part i (block c0 + i) is slot 1 of block c0 and slot 0 of the others.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const AttnArgs a, const int D) {
  const int u = blockIdx.x % (a.Hkv * a.rblocks), b = blockIdx.x / (a.Hkv * a.rblocks);
  const int c0 = a.meta[(int64_t)blockIdx.x * 2], c1 = a.meta[(int64_t)blockIdx.x * 2 + 1];
  if (c0 < 0) return;
  const int hkv = u / a.rblocks, r0 = u % a.rblocks * a.rows;
  const int nr = min(a.rows, a.G * a.q_len - r0);
  const int64_t one = (int64_t)a.rows * (D + 2);
  auto slot = [&](int c) { return a.part + ((int64_t)c * 2 + (c == c0)) * one; };
  for (int r = blockIdx.y; r < nr; r += gridDim.y) {
    float m = -INFINITY;
    for (int c = c0; c <= c1; ++c) m = fmaxf(m, slot(c)[r * (D + 2) + D]);
    float l = 0.0f, acc[2] = {0.0f, 0.0f};
    if (m > -INFINITY)
      for (int c = c0; c <= c1; ++c) {
        const float* p = slot(c) + r * (D + 2);
        const float w = expf(p[D] - m);
        l = fmaf(w, p[D + 1], l);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if ((int)threadIdx.x + i * kThreads < D)
            acc[i] = fmaf(w, p[threadIdx.x + i * kThreads], acc[i]);
      }
    const int rr = r0 + r;
    const int64_t row = (int64_t)b * a.q_len + rr / a.G;
    const int h = hkv * a.G + rr % a.G;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if ((int)threadIdx.x + i * kThreads < D) {
        const auto raw = f32_to_raw<T>(acc[i] * inv);
        *reinterpret_cast<std::remove_const_t<decltype(raw)>*>(
            reinterpret_cast<T*>(a.out) + row * a.out_rs + (int64_t)h * D + threadIdx.x +
            i * kThreads) = raw;
      }
    if (a.lse && threadIdx.x == 0)
      a.lse[row * a.Hq + h] = l > 0.0f ? m + logf(l) : -INFINITY;
  }
}

template <typename T, int D>
cudaError_t launch_attn(const AttnArgs& a, int grid, cudaStream_t st) {
  const size_t smem = sizeof(AttnSmem<T, D>);
  const cudaError_t e = cudaFuncSetAttribute(
      attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  attn_kernel<T, D><<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

struct AttnPlan {
  int rblocks, rows, grid;
  int64_t meta_bytes, bytes;
};
AttnPlan plan(int dtype, int sms, int64_t B, int q_len, int G, int Hkv, int D) {
  AttnPlan p;
  const int rows = G * q_len;
  if (dtype == CCONV_DTYPE_F32) {
    p.rows = kRows;
    p.grid = sms * 2;
  } else {
    // row tiles whose sums fit in registers; blocks that an SM holds at once, by
    // their shared memory (70 to 218 KB) and registers
    p.rows = rows <= 16 || D == 256 ? 16 : 32;
    p.grid = sms * (D * p.rows >= 4096 ? 1 : D * p.rows >= 2048 ? 2 : 3);
  }
  p.rblocks = (rows + p.rows - 1) / p.rows;
  p.meta_bytes = (B * Hkv * p.rblocks * 8 + 15) / 16 * 16;
  p.bytes = p.meta_bytes + (int64_t)p.grid * 2 * p.rows * (D + 2) * 4;
  return p;
}

int check_sizes(int32_t num_seqs, int32_t n_spec, int32_t Hq, int32_t Hkv, int32_t D) {
  if (num_seqs < 0 || n_spec < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0)
    return CCONV_ERR_INVALID;
  if (n_spec > kMaxSpec || (int64_t)(Hq / Hkv) * (1 + n_spec) > 64 ||
      (D != 64 && D != 128 && D != 256))
    return CCONV_ERR_UNSUPPORTED;
  if ((int64_t)num_seqs * Hkv * 8 > INT32_MAX || (int64_t)num_seqs * (1 + n_spec) > INT32_MAX)
    return CCONV_ERR_INVALID;
  return CCONV_OK;
}

}  // namespace
}  // namespace cconv

using namespace cconv;

extern "C" int64_t attn_decode_workspace_bytes(int32_t num_seqs, int32_t n_spec,
                                               int32_t num_q_heads, int32_t num_kv_heads,
                                               int32_t head_dim) {
  const int rc = check_sizes(num_seqs, n_spec, num_q_heads, num_kv_heads, head_dim);
  if (rc != CCONV_OK) return rc;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  int64_t most = 0;
  for (const int dtype : {CCONV_DTYPE_F32, CCONV_DTYPE_BF16})
    most = std::max(most, plan(dtype, sms, num_seqs, 1 + n_spec, num_q_heads / num_kv_heads,
                               num_kv_heads, head_dim).bytes);
  return most;
}

extern "C" int attn_decode(const void* q, int64_t q_row_stride, kv_cache_t cache,
                           const int32_t* block_table, int64_t block_table_row_stride,
                           int32_t table_width, const int32_t* seq_lens, int32_t num_seqs,
                           int32_t n_spec, int32_t num_q_heads, float scale, int32_t dtype,
                           void* out, int64_t out_row_stride, float* lse, void* workspace,
                           int64_t workspace_bytes, int32_t* dev_err, cconv_stream_t stream) {
  const int e = mix_dtype_bytes(dtype);
  if (e == 0) return CCONV_ERR_INVALID;
  int rc = mix_check_cache(cache, dtype);
  if (rc != CCONV_OK) return rc;
  rc = check_sizes(num_seqs, n_spec, num_q_heads, cache.num_kv_heads, cache.head_dim);
  if (rc != CCONV_OK) return rc;
  if (num_seqs == 0) return CCONV_OK;
  const int V = 16 / e, D = cache.head_dim;
  if (!mix_rows_ok(q, q_row_stride, (int64_t)num_q_heads * D, V) ||
      !mix_rows_ok(out, out_row_stride, (int64_t)num_q_heads * D, V) || !seq_lens ||
      table_width < 0 || (table_width > 0 && !block_table) ||
      block_table_row_stride < table_width ||
      (int64_t)table_width * cache.page_size > INT32_MAX - 1024)
    return CCONV_ERR_INVALID;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  const AttnPlan p = plan(dtype, sms, num_seqs, 1 + n_spec, num_q_heads / cache.num_kv_heads,
                          cache.num_kv_heads, D);
  if (!workspace || !mix_aligned16(workspace) || workspace_bytes < p.bytes)
    return CCONV_ERR_INVALID;
  AttnArgs a;
  a.q = static_cast<const char*>(q);
  a.q_rs = q_row_stride;
  a.kc = static_cast<const char*>(cache.k);
  a.vc = static_cast<const char*>(cache.v);
  a.s_page = cache.s_page, a.s_tok = cache.s_token, a.s_head = cache.s_head;
  a.num_pages = cache.num_pages, a.page_size = cache.page_size;
  a.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (cache.page_size == 1 << s) a.page_shift = s;
  a.table = block_table;
  a.table_rs = block_table_row_stride;
  a.table_width = table_width;
  a.seq_lens = seq_lens;
  a.B = num_seqs;
  a.q_len = 1 + n_spec;
  a.Hq = num_q_heads;
  a.Hkv = cache.num_kv_heads;
  a.G = num_q_heads / cache.num_kv_heads;
  a.scale = scale;
  a.out = static_cast<char*>(out);
  a.out_rs = out_row_stride;
  a.lse = lse;
  a.meta = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.meta_bytes);
  a.rblocks = p.rblocks;
  a.rows = p.rows;
  a.dev_err = dev_err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == CCONV_DTYPE_F32)
    err = D == 64 ? launch_attn<float, 64>(a, p.grid, st)
          : D == 128 ? launch_attn<float, 128>(a, p.grid, st)
                     : launch_attn<float, 256>(a, p.grid, st);
  else
    err = attn_launch_mma(a, D, p.grid, st);
  if (err != cudaSuccess) return CCONV_ERR_LAUNCH;
  const dim3 grid((unsigned)(num_seqs * cache.num_kv_heads * p.rblocks),
                  (unsigned)std::min(8, p.rows));
  if (dtype == CCONV_DTYPE_F32)
    attn_join_kernel<float><<<grid, kThreads, 0, st>>>(a, D);
  else
    attn_join_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, D);
  return cudaGetLastError() == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}
