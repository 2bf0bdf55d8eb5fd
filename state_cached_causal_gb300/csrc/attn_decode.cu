// Entry points attn_decode and attn_decode_q8: host side, the plain-arithmetic
// kernel and the join of split results. The split is described in attn_decode.cuh.
//
// attn_kernel keeps one softmax pass over the tiles: K and V of 32 positions go
// to shared memory, each warp scores two of up to kRows query rows (lane =
// position), and the threads hold kRows weighted sums of their columns of V.
// Up to kRows rows of a kv head read its K and V once; more rows are taken in
// blocks, each of which reads them again (32 heads on 8 of 128 with 4 tokens, 16
// rows: 3 requests of up to 3616 positions 69 us). A block loads and computes in
// turn, so it is the other blocks of the SM that keep the memory busy: 60 requests
// of up to 8192 positions, 2 kv heads of 64: 123 us with seven (2.1 TB/s), 274
// with two.
#include "attn_decode.cuh"
#include "q8.cuh"

#include <math.h>

namespace cconv {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;
constexpr int kRows = kAttnPlainRows;
constexpr int kMaxGrid = kAttnMaxGrid;

template <typename T, int D>
struct AttnSmem {
  float k[kTile][D + 4];
  float v[kTile][D];
  float q[kRows][D];
  float p[kRows][kTile];
  float corr[kRows];
  int64_t scan[kThreads + 4];
};

template <typename T, int D, bool Q8>
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
        if (Q8 && page >= 0) {
          const int64_t off = page * a.s_page + (pos % a.page_size) * a.s_tok +
                              (int64_t)hkv * a.s_head + u * V;
          const int64_t to = page * a.c_page + (pos % a.page_size) * a.c_tok + hkv * a.c_head;
          const float ks = q8_scale(a.ksc[to]), vs = q8_scale(a.vsc[to]);
#pragma unroll
          for (int e = 0; e < V; e += 4) {
            float yk[4], yv[4];
            unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(a.kc + off + e), yk);
            unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(a.vc + off + e), yv);
#pragma unroll
            for (int k = 0; k < 4; ++k) fk[e + k] = yk[k] * ks, fv[e + k] = yv[k] * vs;
          }
        } else if (page >= 0) {
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
        const float base = mn == -INFINITY ? 0.0f : mn;   // (a NaN score stays one)
        const float p = expf(x - base), corr = expf(m[i] - base);
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
      // (a weight of zero does not hide an infinity or NaN among the values of
      // a draft token from the rows before it: there the rows choose)
      const int drafts = sg.len - a.q_len + 1 - t0;   // positions that all rows see
      if (tid < D && drafts >= kTile) {
#pragma unroll 4
        for (int t = 0; t < kTile; ++t)
#pragma unroll
          for (int c = 0; c < CD; ++c) {
            const float v = sm.v[t][tid + c * kThreads];
#pragma unroll
            for (int r = 0; r < kRows; ++r) acc[c][r] = fmaf(sm.p[r][t], v, acc[c][r]);
          }
      } else if (tid < D) {
#pragma unroll 1
        for (int t = 0; t < kTile; ++t)
#pragma unroll
          for (int c = 0; c < CD; ++c) {
            const float v = sm.v[t][tid + c * kThreads];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
              if (t < drafts + (r0 + r) / a.G) acc[c][r] = fmaf(sm.p[r][t], v, acc[c][r]);
          }
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
            const float inv = sm.corr[r] != 0.0f ? 1.0f / sm.corr[r] : 0.0f;
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
              l[lane] != 0.0f ? m[lane] + logf(l[lane]) : -INFINITY;
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

// The joins of the parts of cut units. Part i (block c0 + i) is slot 1 of block
// c0 and slot 0 of the others. (Both kernels are launched to overlap the end of
// the kernel before, whose results they wait for.)
//
// A few rows have many parts each -- one long context has one of every block:
// a block a row and CC of its columns. A thread takes a column and every
// kGroups-th part; it requests its first kPre values, then the threads turn the
// parts' maxima and sums into weights: two round trips to the L2 in all.
template <typename T, int D>
__global__ void __launch_bounds__(512) attn_join_kernel(const AttnArgs a) {
  constexpr int kJoinThreads = 512, CC = 16, kGroups = kJoinThreads / CC;
  constexpr int kPre = 10;
  __shared__ float wt[kMaxGrid], lt[kMaxGrid];
  __shared__ float red[2][kJoinThreads / 32];
  __shared__ float sums[kGroups][CC];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rows = a.hw * a.rows, used = min(a.rows, a.G * a.q_len);
  const int64_t bu = blockIdx.x;                    // request and unit
  const int row = blockIdx.y / used * a.rows + blockIdx.y % used;
  const int c0 = a.meta[bu * 2], c1 = a.meta[bu * 2 + 1];
  if (!attn_joins(c0, c1, a.grid)) return;
  const int b = (int)(bu / a.units), u = (int)(bu % a.units);
  const int hkv = u / a.rblocks * a.hw + row / a.rows;
  const int rr = u % a.rblocks * a.rows + row % a.rows;
  if (rr >= a.G * a.q_len) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, parts = c1 - c0 + 1;
  const int64_t one = (int64_t)rows * (D + 2);
  auto part = [&](int i) {
    return a.part + ((int64_t)(c0 + i) * 2 + (i == 0)) * one + row * (D + 2);
  };
  const int cl = tid % CC, g = tid / CC, c = blockIdx.z * CC + cl;
  float x[kPre];
#pragma unroll
  for (int k = 0; k < kPre; ++k)
    x[k] = g + k * kGroups < parts ? part(g + k * kGroups)[c] : 0.0f;
  float m = -INFINITY;
  for (int i = tid; i < parts; i += kJoinThreads) {
    const float2 ml = *reinterpret_cast<const float2*>(part(i) + D);
    wt[i] = ml.x;
    lt[i] = ml.y;
    m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, red[0][w]);
  float l = 0.0f;
  for (int i = tid; i < parts; i += kJoinThreads) {
    const float w = m == -INFINITY ? 0.0f : expf(wt[i] - m);
    wt[i] = w;
    l = fmaf(w, lt[i], l);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) l += red[1][w];
  float acc = 0.0f;
#pragma unroll
  for (int k = 0; k < kPre; ++k)
    if (g + k * kGroups < parts) acc = fmaf(wt[g + k * kGroups], x[k], acc);
  for (int i = g + kPre * kGroups; i < parts; i += kGroups) acc = fmaf(wt[i], part(i)[c], acc);
  sums[g][cl] = acc;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) acc += sums[k][cl];
  const int64_t orow = (int64_t)b * a.q_len + rr / a.G;
  const int h = hkv * a.G + rr % a.G;
  const auto raw = f32_to_raw<T>(l != 0.0f ? acc / l : 0.0f);
  T* const o = reinterpret_cast<T*>(a.out) + orow * a.out_rs + (int64_t)h * D + c;
  *reinterpret_cast<std::remove_const_t<decltype(raw)>*>(o) = raw;
  if (a.lse && c == 0) a.lse[orow * a.Hq + h] = l != 0.0f ? m + logf(l) : -INFINITY;
}

// Many rows have few parts each: a warp a row. (A block a row took 4096 blocks,
// four rounds of them, for 64 requests of 64 rows: 66 us in all, 56 so.)
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_rows_kernel(const AttnArgs a, const int64_t n) {
  constexpr int kPairs = D / 64, kAhead = 4;
  const int lane = threadIdx.x & 31;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (at >= n) return;
  const int rows = a.hw * a.rows, used = min(a.rows, a.G * a.q_len), y = a.hw * used;
  const int64_t bu = at / y;                        // request and unit
  const int row = (int)(at % y) / used * a.rows + (int)(at % y) % used;
  const int c0 = a.meta[bu * 2], c1 = a.meta[bu * 2 + 1];
  if (!attn_joins(c0, c1, a.grid)) return;
  const int b = (int)(bu / a.units), u = (int)(bu % a.units);
  const int hkv = u / a.rblocks * a.hw + row / a.rows;
  const int rr = u % a.rblocks * a.rows + row % a.rows;
  if (rr >= a.G * a.q_len) return;
  const int parts = c1 - c0 + 1;
  const int64_t one = (int64_t)rows * (D + 2);
  auto part = [&](int i) {
    return a.part + ((int64_t)(c0 + i) * 2 + (i == 0)) * one + row * (D + 2);
  };
  auto stats = [&](int i) {
    return i < parts ? *reinterpret_cast<const float2*>(part(i) + D)
                     : make_float2(-INFINITY, 0.0f);
  };
  const float2 first = stats(lane);
  float m = first.x;
  for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, stats(i).x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float l = 0.0f, acc[kPairs][2] = {};
  for (int i0 = 0; i0 < parts; i0 += 32) {
    const float2 ml = i0 == 0 ? first : stats(i0 + lane);
    const float w = ml.x == -INFINITY ? 0.0f : expf(ml.x - m);
    l = fmaf(w, ml.y, l);
    const int end = min(32, parts - i0);
    for (int k0 = 0; k0 < end; k0 += kAhead) {
      float2 x[kAhead][kPairs];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
          x[k][j] = k0 + k < end ? *reinterpret_cast<const float2*>(part(i0 + k0 + k) + j * 64 +
                                                                    lane * 2)
                                 : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k0 + k);   // (0 behind the last part)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          acc[j][0] = fmaf(wk, x[k][j].x, acc[j][0]);
          acc[j][1] = fmaf(wk, x[k][j].y, acc[j][1]);
        }
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const int64_t orow = (int64_t)b * a.q_len + rr / a.G;
  const int h = hkv * a.G + rr % a.G;
  T* const o = reinterpret_cast<T*>(a.out) + orow * a.out_rs + (int64_t)h * D + lane * 2;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const float v0 = acc[j][0] * inv, v1 = acc[j][1] * inv;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(o + j * 64) = make_float2(v0, v1);
    else
      *reinterpret_cast<uint32_t*>(o + j * 64) = pack_bf16x2(v0, v1);
  }
  if (a.lse && lane == 0) a.lse[orow * a.Hq + h] = l != 0.0f ? m + logf(l) : -INFINITY;
}

template <typename T, int D>
cudaError_t launch_join(const AttnArgs& a, cudaStream_t st) {
  const int y = a.hw * std::min(a.rows, a.G * a.q_len);
  const int64_t units = (int64_t)a.B * a.units, n = units * y;
  const bool few = n <= 512;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = few ? dim3((unsigned)units, (unsigned)y, D / 16) : dim3((unsigned)((n + 7) / 8));
  cfg.blockDim = dim3(few ? 512 : 256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, attn_join_kernel<T, D>, a)
             : cudaLaunchKernelEx(&cfg, attn_join_rows_kernel<T, D>, a, n);
}

template <typename T, int D, bool Q8>
cudaError_t launch_attn(const AttnArgs& a, int grid, cudaStream_t st) {
  const size_t smem = sizeof(AttnSmem<T, D>);
  static std::atomic<uint64_t> full;
  const cudaError_t e = mix_full_smem(reinterpret_cast<const void*>(attn_kernel<T, D, Q8>), full);
  if (e != cudaSuccess) return e;
  attn_kernel<T, D, Q8><<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename T, bool Q8>
cudaError_t launch_attn_d(const AttnArgs& a, int D, int grid, cudaStream_t st) {
  return D == 64    ? launch_attn<T, 64, Q8>(a, grid, st)
         : D == 128 ? launch_attn<T, 128, Q8>(a, grid, st)
                    : launch_attn<T, 256, Q8>(a, grid, st);
}

// What both entry points check and do; a's cache is set.
int decode(AttnArgs& a, int D, bool q8, const void* q, int64_t q_row_stride,
           const int32_t* block_table, int64_t block_table_row_stride, int32_t table_width,
           const int32_t* seq_lens, int32_t num_seqs, int32_t n_spec, int32_t num_q_heads,
           float scale, int32_t dtype, void* out, int64_t out_row_stride, float* lse,
           void* workspace, int64_t workspace_bytes, int32_t* dev_err, cconv_stream_t stream) {
  const int rc = attn_check_sizes(num_seqs, n_spec, num_q_heads, a.Hkv, D);
  if (rc != CCONV_OK) return rc;
  if (num_seqs == 0) return CCONV_OK;
  if (!attn_rows_ok(a, D, dtype, q, q_row_stride, out, out_row_stride, num_q_heads, block_table,
                    block_table_row_stride, table_width, seq_lens))
    return CCONV_ERR_INVALID;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  const AttnPlan p = attn_plan(dtype, q8, sms, num_seqs, 1 + n_spec, num_q_heads / a.Hkv, a.Hkv, D);
  if (!workspace || !mix_aligned16(workspace) || workspace_bytes < p.bytes)
    return CCONV_ERR_INVALID;
  attn_fill(a, p, D, q8 ? 1 : 2, q, q_row_stride, block_table, block_table_row_stride, table_width,
            seq_lens, num_seqs, n_spec, num_q_heads, scale, out, out_row_stride, lse, dev_err);
  a.meta = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.meta_bytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == CCONV_DTYPE_F32)
    err = q8 ? launch_attn_d<float, true>(a, D, p.grid, st)
             : launch_attn_d<float, false>(a, D, p.grid, st);
  else
    err = q8 ? attn_launch_mma_q8(a, D, p.grid, false, st)
             : attn_launch_mma(a, D, p.grid, false, st);
  if (err != cudaSuccess) return CCONV_ERR_LAUNCH;
  if (dtype == CCONV_DTYPE_F32)
    err = D == 64 ? launch_join<float, 64>(a, st) : D == 128 ? launch_join<float, 128>(a, st)
                                                             : launch_join<float, 256>(a, st);
  else
    err = D == 64 ? launch_join<__nv_bfloat16, 64>(a, st)
          : D == 128 ? launch_join<__nv_bfloat16, 128>(a, st)
                     : launch_join<__nv_bfloat16, 256>(a, st);
  return err == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}

}  // namespace
}  // namespace cconv

using namespace cconv;

extern "C" int64_t attn_decode_workspace_bytes(int32_t num_seqs, int32_t n_spec,
                                               int32_t num_q_heads, int32_t num_kv_heads,
                                               int32_t head_dim) {
  const int rc = attn_check_sizes(num_seqs, n_spec, num_q_heads, num_kv_heads, head_dim);
  if (rc != CCONV_OK) return rc;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  int64_t most = 0;
  for (const int dtype : {CCONV_DTYPE_F32, CCONV_DTYPE_BF16})
    for (const bool q8 : {false, true})
      most = std::max(most, attn_plan(dtype, q8, sms, num_seqs, 1 + n_spec,
                                      num_q_heads / num_kv_heads, num_kv_heads, head_dim).bytes);
  return most;
}

extern "C" int attn_decode(const void* q, int64_t q_row_stride, kv_cache_t cache,
                           const int32_t* block_table, int64_t block_table_row_stride,
                           int32_t table_width, const int32_t* seq_lens, int32_t num_seqs,
                           int32_t n_spec, int32_t num_q_heads, float scale, int32_t dtype,
                           void* out, int64_t out_row_stride, float* lse, void* workspace,
                           int64_t workspace_bytes, int32_t* dev_err, cconv_stream_t stream) {
  if (mix_dtype_bytes(dtype) == 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache(cache, dtype);
  if (rc != CCONV_OK) return rc;
  AttnArgs a = attn_cache_args(cache);
  return decode(a, cache.head_dim, false, q, q_row_stride, block_table, block_table_row_stride,
                table_width, seq_lens, num_seqs, n_spec, num_q_heads, scale, dtype, out,
                out_row_stride, lse, workspace, workspace_bytes, dev_err, stream);
}

extern "C" int attn_decode_q8(const void* q, int64_t q_row_stride, kv_cache_q8_t cache,
                              const int32_t* block_table, int64_t block_table_row_stride,
                              int32_t table_width, const int32_t* seq_lens, int32_t num_seqs,
                              int32_t n_spec, int32_t num_q_heads, float scale, int32_t dtype,
                              void* out, int64_t out_row_stride, float* lse, void* workspace,
                              int64_t workspace_bytes, int32_t* dev_err, cconv_stream_t stream) {
  if (mix_dtype_bytes(dtype) == 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache_q8(cache);
  if (rc != CCONV_OK) return rc;
  AttnArgs a = attn_cache_args(cache);
  a.ksc = cache.k_scale;
  a.vsc = cache.v_scale;
  a.c_page = cache.c_page, a.c_tok = cache.c_token, a.c_head = cache.c_head;
  return decode(a, cache.head_dim, true, q, q_row_stride, block_table, block_table_row_stride,
                table_width, seq_lens, num_seqs, n_spec, num_q_heads, scale, dtype, out,
                out_row_stride, lse, workspace, workspace_bytes, dev_err, stream);
}
