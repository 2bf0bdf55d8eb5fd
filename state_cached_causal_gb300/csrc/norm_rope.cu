// Entry point attn_norm_rope_cache: per-head RMS norm of q and k, rotation by
// position, and the write of k and v into the paged cache, in one pass.
//
// The pass reads every row once and writes every row once, with about 10
// flops a value: it is bound by HBM. A head is a run of 16-byte units, one per
// lane (LPH lanes a head, 32/LPH heads a warp at a time). A warp keeps one
// token: its lanes hold the same columns of every head, so the token's cosines
// and sines and the norm weights are loaded once into registers and serve all
// its heads; heads go in groups of kUnroll whose loads are in flight together.
// When there are few tokens a token's heads are spread over several warps.
#include "mixer.cuh"

namespace cconv {
namespace {

constexpr int kNrThreads = 128;
constexpr int kUnroll = 4;

struct NrArgs {
  const char *q, *k, *v;
  int64_t q_rs, k_rs, v_rs, qo_rs;
  const char *qw, *kw;
  float eps;
  const float* cs;
  int32_t max_pos, rot;
  const int32_t* pos;
  char *kc, *vc;
  int64_t s_page, s_tok, s_head;
  int32_t page_size;
  int64_t num_slots;
  const int32_t* slots;
  int32_t T, Hq, Hkv;
  int32_t parts;      // warps a token
  char* qo;
  int32_t* dev_err;
};

// U units of a head per lane (2 when a head has more than 32 units).
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NrArgs a) {
  constexpr int V = Elem<T>::V, E = Elem<T>::bytes;
  constexpr int UNITS = D / V;
  constexpr int U = UNITS > 32 ? UNITS / 32 : 1;
  constexpr int LPH = UNITS / U;              // lanes a head
  constexpr int HPW = 32 / LPH;               // heads a warp at a time
  const int lane = threadIdx.x & 31;
  const int64_t wid = (int64_t)blockIdx.x * (kNrThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = wid / a.parts;
  const int part = (int)(wid % a.parts);
  if (t >= a.T) return;
  const int pos = a.pos[t];
  const int slot = a.slots[t];
  if (pos < 0 || pos >= a.max_pos || slot >= a.num_slots) {
    if (part == 0 && lane == 0) flag_error(a.dev_err, CCONV_DERR_POSITION);
    return;
  }
  const int sub = lane / LPH, hl = lane % LPH;   // head of the group, lane of the head
  // the lane's unit u holds columns u * LPH * V + hl * V + [0, V)
  float c[U][V], s[U][V];
  const int half = a.rot / 2;
  const float* cs = a.cs + (int64_t)pos * a.rot;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int col = (u * LPH + hl) * V + e;
      c[u][e] = 1.0f;
      s[u][e] = 0.0f;
      if (col < a.rot) {
        const int i = PAIRS ? col >> 1 : (col < half ? col : col - half);
        const bool lo = PAIRS ? (col & 1) == 0 : col < half;
        c[u][e] = __ldg(cs + i);
        s[u][e] = lo ? -__ldg(cs + half + i) : __ldg(cs + half + i);
      }
    }
  char *kdst = nullptr, *vdst = nullptr;
  if (slot >= 0) {
    const int64_t page = slot / a.page_size, tok = slot % a.page_size;
    const int64_t off = (page * a.s_page + tok * a.s_tok) * E;
    kdst = a.kc + off;
    vdst = a.vc + off;
  }
  // heads [0, Hq) of q, then Hkv of k (both normalised and rotated)
  auto rotate_heads = [&](int h_begin, int h_end, const char* src, const char* w, char* dst,
                          int64_t dst_head) {
    float wt[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e)
        wt[u][e] = w ? load_f32<T>(w, (u * LPH + hl) * V + e) : 1.0f;
    for (int h0 = h_begin; h0 < h_end; h0 += HPW * kUnroll) {
      uint4 raw[kUnroll][U];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int h = h0 + j * HPW + sub;
        if (h < h_end)
#pragma unroll
          for (int u = 0; u < U; ++u)
            raw[j][u] = *reinterpret_cast<const uint4*>(
                src + ((int64_t)h * D + (u * LPH + hl) * V) * E);
        else
#pragma unroll
          for (int u = 0; u < U; ++u) raw[j][u] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        if (h0 + j * HPW >= h_end) break;            // warp-uniform
        const int h = h0 + j * HPW + sub;
        float x[U][V], sum = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          unpack16<T>(raw[j][u], x[u]);
#pragma unroll
          for (int e = 0; e < V; ++e) sum = fmaf(x[u][e], x[u][e], sum);
        }
        if (w) {
#pragma unroll
          for (int d = LPH / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          const float r = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) x[u][e] *= r * wt[u][e];
        }
        float y[U][V];
        if constexpr (PAIRS) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) y[u][e] = fmaf(x[u][e ^ 1], s[u][e], x[u][e] * c[u][e]);
        } else {
          // the partner column is half columns away: half is a whole number of
          // units, so the same element of another lane's unit
          const int hu = half / V;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int unit = u * LPH + hl;
            int pu = unit;
            if (unit < 2 * hu) pu = unit < hu ? unit + hu : unit - hu;
            const int pl = (lane - hl) + pu % LPH;
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float other = __shfl_sync(0xffffffffu, x[0][e], pl);
              if constexpr (U == 2) {
                const float hi = __shfl_sync(0xffffffffu, x[1][e], pl);
                if (pu >= LPH) other = hi;
              }
              y[u][e] = fmaf(other, s[u][e], x[u][e] * c[u][e]);
            }
          }
        }
        if (h < h_end && dst) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            stg16(dst + ((int64_t)h * dst_head + (u * LPH + hl) * V) * E, pack16<T>(y[u]));
        }
      }
    }
  };
  // this warp's share of the heads, in whole groups of HPW
  const int gq = (a.Hq + HPW - 1) / HPW, gk = (a.Hkv + HPW - 1) / HPW;
  auto share = [&](int groups, int heads, int& b, int& e) {
    b = min(heads, (int)((int64_t)groups * part / a.parts) * HPW);
    e = min(heads, (int)((int64_t)groups * (part + 1) / a.parts) * HPW);
  };
  int hb, he;
  share(gq, a.Hq, hb, he);
  if (hb < he)
    rotate_heads(hb, he, a.q + t * a.q_rs * E, a.qw, a.qo + t * a.qo_rs * E, D);
  if (!kdst) return;
  share(gk, a.Hkv, hb, he);
  if (hb < he) {
    // the values first: their loads run while the keys are worked on
    const char* vs = a.v + t * a.v_rs * E;
    for (int h0 = hb; h0 < he; h0 += HPW) {
      const int h = h0 + sub;
      if (h < he)
#pragma unroll
        for (int u = 0; u < U; ++u)
          stg16(vdst + ((int64_t)h * a.s_head + (u * LPH + hl) * V) * E,
                *reinterpret_cast<const uint4*>(vs + ((int64_t)h * D + (u * LPH + hl) * V) * E));
    }
    rotate_heads(hb, he, a.k + t * a.k_rs * E, a.kw, kdst, a.s_head);
  }
}

template <typename T, int D>
cudaError_t launch_nr(const NrArgs& a, bool pairs, cudaStream_t st) {
  const int64_t warps = (int64_t)a.T * a.parts;
  const unsigned grid = (unsigned)((warps + kNrThreads / 32 - 1) / (kNrThreads / 32));
  if (pairs)
    norm_rope_kernel<T, D, true><<<grid, kNrThreads, 0, st>>>(a);
  else
    norm_rope_kernel<T, D, false><<<grid, kNrThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_nr_d(const NrArgs& a, int D, bool pairs, cudaStream_t st) {
  if (D == 64) return launch_nr<T, 64>(a, pairs, st);
  if (D == 128) return launch_nr<T, 128>(a, pairs, st);
  return launch_nr<T, 256>(a, pairs, st);
}

}  // namespace
}  // namespace cconv

using namespace cconv;

extern "C" int attn_norm_rope_cache(const void* q, int64_t q_row_stride, const void* k,
                                    int64_t k_row_stride, const void* v, int64_t v_row_stride,
                                    const void* q_weight, const void* k_weight, float eps,
                                    const float* cos_sin, int32_t max_position, int32_t rot_dim,
                                    int32_t interleaved, const int32_t* positions,
                                    kv_cache_t cache, const int32_t* slot_mapping,
                                    int32_t num_tokens, int32_t num_q_heads, int32_t dtype,
                                    void* q_out, int64_t q_out_row_stride, int32_t* dev_err,
                                    cconv_stream_t stream) {
  const int e = mix_dtype_bytes(dtype);
  if (e == 0 || num_tokens < 0 || num_q_heads <= 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache(cache, dtype);
  if (rc != CCONV_OK) return rc;
  const int V = 16 / e, D = cache.head_dim;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 || (!interleaved && rot_dim % (2 * V)) ||
      max_position <= 0 || (rot_dim > 0 && !cos_sin) || !(eps >= 0.0f))
    return CCONV_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(q_weight) % e || reinterpret_cast<uintptr_t>(k_weight) % e)
    return CCONV_ERR_INVALID;
  if (num_tokens == 0) return CCONV_OK;
  if (!mix_rows_ok(q, q_row_stride, (int64_t)num_q_heads * D, V) ||
      !mix_rows_ok(k, k_row_stride, (int64_t)cache.num_kv_heads * D, V) ||
      !mix_rows_ok(v, v_row_stride, (int64_t)cache.num_kv_heads * D, V) ||
      !mix_rows_ok(q_out, q_out_row_stride, (int64_t)num_q_heads * D, V) || !positions ||
      !slot_mapping)
    return CCONV_ERR_INVALID;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  NrArgs a;
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.q_rs = q_row_stride, a.k_rs = k_row_stride, a.v_rs = v_row_stride;
  a.qo_rs = q_out_row_stride;
  a.qw = static_cast<const char*>(q_weight);
  a.kw = static_cast<const char*>(k_weight);
  a.eps = eps;
  a.cs = cos_sin;
  a.max_pos = max_position;
  a.rot = rot_dim;
  a.pos = positions;
  a.kc = static_cast<char*>(cache.k);
  a.vc = static_cast<char*>(cache.v);
  a.s_page = cache.s_page, a.s_tok = cache.s_token, a.s_head = cache.s_head;
  a.page_size = cache.page_size;
  a.num_slots = (int64_t)cache.num_pages * cache.page_size;
  a.slots = slot_mapping;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.Hkv = cache.num_kv_heads;
  a.qo = static_cast<char*>(q_out);
  a.dev_err = dev_err;
  // several warps a token while there are fewer than 16 warps an SM
  a.parts = (int32_t)std::max<int64_t>(
      1, std::min<int64_t>(8, (int64_t)sms * 16 / std::max(1, num_tokens)));
  if (((int64_t)num_tokens * a.parts) / (kNrThreads / 32) + 1 > INT32_MAX)
    return CCONV_ERR_INVALID;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == CCONV_DTYPE_F32
                              ? launch_nr_d<float>(a, D, interleaved != 0, st)
                              : launch_nr_d<__nv_bfloat16>(a, D, interleaved != 0, st);
  return err == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}
