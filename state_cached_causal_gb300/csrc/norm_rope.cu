// Entry point attn_norm_rope_cache: per-head RMS norm of q and k, rotation by
// position, and the write of k and v into the paged cache, in one pass.
//
// The pass reads every row once and writes every row once, with about 10
// flops a value: it is bound by HBM as long as the instructions around those
// flops stay few. A lane holds two 16-byte units of a head, in the half-split
// rotation unit u of the first half and unit u of the second, so that both
// values of every rotated pair are in one lane (with one unit a lane the partner
// came by shuffles, 8 for 8 values). A warp takes one token after the other: its
// lanes hold the same columns of every head, so a token's cosines and sines, and
// for all tokens the norm weights, are in registers and serve all heads. When
// there are few tokens a token's heads are spread over several warps.
//
// Four groups of query heads have their loads in flight together, beside the
// first group of keys and values, and four blocks an SM take the tokens one after
// the other, the next token's position and slot read ahead. 33024 tokens of
// 16 + 4 + 4 heads of 128 in bf16: 75.9 us for 422 MB, 5.6 TB/s (keys after the
// queries, values after the keys: 78.7 us; three blocks, whose 168 registers
// spill nothing: 78.1 us; one unit a lane: 98.7 us). 61 tokens: 3.0 us, the
// latency of a few dependent loads.
#include "mixer.cuh"

namespace cconv {
namespace {

constexpr int kNrThreads = 128;
constexpr int kNrBlocks = 4;    // of an SM
constexpr int kUnroll = 4;      // groups of heads whose loads are in flight together

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

template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kNrThreads, kNrBlocks) norm_rope_kernel(const NrArgs a) {
  constexpr int V = Elem<T>::V, E = Elem<T>::bytes;
  constexpr int LPH = D / V / 2;              // lanes a head, two units each
  constexpr int HPW = 32 / LPH;               // heads a warp at a time
  const int lane = threadIdx.x & 31;
  const int wid = blockIdx.x * (kNrThreads / 32) + (threadIdx.x >> 5);
  const int part = wid % a.parts;
  const int step = gridDim.x * (kNrThreads / 32) / a.parts;   // tokens at a time
  const int sub = lane / LPH, l = lane % LPH;    // head of the group, lane of the head
  // columns [c0, c0 + V) and [c1, c1 + V): partners half a rotation apart, or
  // neighbours where nothing is rotated (and in the interleaved rotation)
  const int half = a.rot / 2, hu = PAIRS ? 0 : half / V;
  // unit at column c of a weight vector (of any alignment)
  auto load_w = [](const char* w, int c) {
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = load_f32<T>(w, c + e);
    return pack16<T>(f);
  };
  const int c0 = (l < hu ? l : 2 * l) * V, c1 = (l < hu ? l + hu : 2 * l + 1) * V;
  uint4 wq[2] = {}, wk[2] = {};   // the lane's norm weights
  if (a.qw) wq[0] = load_w(a.qw, c0), wq[1] = load_w(a.qw, c1);
  if (a.kw) wk[0] = load_w(a.kw, c0), wk[1] = load_w(a.kw, c1);
  int t = wid / a.parts;
  if (t >= step) return;        // (a last, incomplete row of warps)
  int pos = t < a.T ? a.pos[t] : 0, slot = t < a.T ? a.slots[t] : 0;
#pragma unroll 1
  while (t < a.T) {
    const int p = pos, sl = slot, tok = t;
    t += step;
    if (t < a.T) {                // the next token's, while this one is worked on
      pos = a.pos[t];
      slot = a.slots[t];
    }
    if (p < 0 || p >= a.max_pos || sl >= a.num_slots) {
      if (part == 0 && lane == 0) flag_error(a.dev_err, CCONV_DERR_POSITION);
      continue;
    }
    // factors of the lane's V pairs: (x0[e], x1[e]), or (x0[2i], x0[2i+1]) then
    // (x1[2i], x1[2i+1])
    float c[V], s[V];
    const float* cs = a.cs + (int64_t)p * a.rot;
    if constexpr (PAIRS) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int i = e < V / 2 ? c0 / 2 + e : c1 / 2 + e - V / 2;
        const bool in = 2 * i < a.rot;
        c[e] = in ? __ldg(cs + i) : 1.0f;
        s[e] = in ? __ldg(cs + half + i) : 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 x = l < hu ? __ldg(reinterpret_cast<const float4*>(cs + c0 + e)) : one;
        const float4 y = l < hu ? __ldg(reinterpret_cast<const float4*>(cs + half + c0 + e)) : zero;
        c[e] = x.x, c[e + 1] = x.y, c[e + 2] = x.z, c[e + 3] = x.w;
        s[e] = y.x, s[e + 1] = y.y, s[e + 2] = y.z, s[e + 3] = y.w;
      }
    }
    char *kdst = nullptr, *vdst = nullptr;
    if (sl >= 0) {
      const int page = sl / a.page_size;
      const int64_t off = (page * a.s_page + (int64_t)(sl - page * a.page_size) * a.s_tok) * E;
      kdst = a.kc + off;
      vdst = a.vc + off;
    }
    // one group of heads: norm, rotation, store (`in`: the lane's head exists)
    auto rotate = [&](const uint4& u0, const uint4& u1, const float (&w0)[V], const float (&w1)[V],
                      bool norm, char* dst, bool in) {
      float x0[V], x1[V];
      unpack16<T>(u0, x0);
      unpack16<T>(u1, x1);
      if (norm) {
        float q0 = 0.0f, q1 = 0.0f, q2 = 0.0f, q3 = 0.0f;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          fma_x2(q0, q1, x0[e], x0[e + 1], x0[e], x0[e + 1], q0, q1);
          fma_x2(q2, q3, x1[e], x1[e + 1], x1[e], x1[e + 1], q2, q3);
        }
        float sum = (q0 + q1) + (q2 + q3);
#pragma unroll
        for (int d = LPH / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float r = rsqrtf(fmaf(sum, 1.0f / D, a.eps));
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          mul_x2(x0[e], x0[e + 1], x0[e], x0[e + 1], r * w0[e], r * w0[e + 1]);
          mul_x2(x1[e], x1[e + 1], x1[e], x1[e + 1], r * w1[e], r * w1[e + 1]);
        }
      }
      float y0[V], y1[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (PAIRS) {
          float* y = e < V / 2 ? y0 + 2 * e : y1 + 2 * e - V;
          const float* x = e < V / 2 ? x0 + 2 * e : x1 + 2 * e - V;
          y[0] = fmaf(-x[1], s[e], x[0] * c[e]);
          y[1] = fmaf(x[0], s[e], x[1] * c[e]);
        } else {
          y0[e] = fmaf(-x1[e], s[e], x0[e] * c[e]);
          y1[e] = fmaf(x0[e], s[e], x1[e] * c[e]);
        }
      }
      if (in) {
        stg16(dst + c0 * E, pack16<T>(y0));
        stg16(dst + c1 * E, pack16<T>(y1));
      }
    };
    auto load = [&](const char* p, bool in, uint4& u0, uint4& u1, int b0, int b1) {
      u0 = u1 = make_uint4(0u, 0u, 0u, 0u);
      if (in) {
        u0 = *reinterpret_cast<const uint4*>(p + b0);
        u1 = *reinterpret_cast<const uint4*>(p + b1);
      }
    };
    // this warp's share of the heads, in whole groups of HPW
    auto share = [&](int heads, int& b, int& e) {
      const int groups = (heads + HPW - 1) / HPW;
      b = min(heads, groups * part / a.parts * HPW);
      e = min(heads, groups * (part + 1) / a.parts * HPW);
    };
    int qb, qe, kb, ke;
    share(a.Hq, qb, qe);
    share(a.Hkv, kb, ke);
    if (!kdst) ke = kb;
    const char* const qs = a.q + tok * a.q_rs * E;
    const char* const ks = a.k + tok * a.k_rs * E;
    const char* const vs = a.v + tok * a.v_rs * E;
    char* const qd = a.qo + tok * a.qo_rs * E;
    // values pass as they are: two units a lane, side by side over the lanes
    const int v0 = l * 16, v1 = (LPH + l) * 16;
    // the first group of keys and values comes while the queries are worked on
    uint4 ku0, ku1, vu0, vu1;
    const int64_t at0 = (int64_t)(kb + sub) * (D * E);
    load(ks + at0, kb + sub < ke, ku0, ku1, c0 * E, c1 * E);
    load(vs + at0, kb + sub < ke, vu0, vu1, v0, v1);
    float w0[V], w1[V];
    unpack16<T>(wq[0], w0);
    unpack16<T>(wq[1], w1);
#pragma unroll 1
    for (int h0 = qb; h0 < qe; h0 += HPW * kUnroll) {
      uint4 u0[kUnroll], u1[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int h = h0 + j * HPW + sub;
        load(qs + (int64_t)h * (D * E), h < qe, u0[j], u1[j], c0 * E, c1 * E);
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        if (h0 + j * HPW >= qe) break;              // warp-uniform
        const int h = h0 + j * HPW + sub;
        rotate(u0[j], u1[j], w0, w1, a.qw != nullptr, qd + (int64_t)h * (D * E), h < qe);
      }
    }
    unpack16<T>(wk[0], w0);
    unpack16<T>(wk[1], w1);
#pragma unroll 1
    for (int h0 = kb; h0 < ke; h0 += HPW) {
      const int h = h0 + sub;
      const int64_t to = (int64_t)h * a.s_head * E;
      if (h < ke) {
        stg16(vdst + to + v0, vu0);
        stg16(vdst + to + v1, vu1);
      }
      const uint4 k0 = ku0, k1 = ku1;
      const int64_t next = (int64_t)(h + HPW) * (D * E);
      load(ks + next, h + HPW < ke, ku0, ku1, c0 * E, c1 * E);
      load(vs + next, h + HPW < ke, vu0, vu1, v0, v1);
      rotate(k0, k1, w0, w1, a.kw != nullptr, kdst + to, h < ke);
    }
  }
}

template <typename T, int D>
cudaError_t launch_nr(const NrArgs& a, bool pairs, int sms, cudaStream_t st) {
  const int64_t warps = (int64_t)a.T * a.parts, per = kNrThreads / 32;
  const unsigned grid =
      (unsigned)std::min<int64_t>((warps + per - 1) / per, (int64_t)sms * kNrBlocks);
  if (pairs)
    norm_rope_kernel<T, D, true><<<grid, kNrThreads, 0, st>>>(a);
  else
    norm_rope_kernel<T, D, false><<<grid, kNrThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_nr_d(const NrArgs& a, int D, bool pairs, int sms, cudaStream_t st) {
  if (D == 64) return launch_nr<T, 64>(a, pairs, sms, st);
  if (D == 128) return launch_nr<T, 128>(a, pairs, sms, st);
  return launch_nr<T, 256>(a, pairs, sms, st);
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
      max_position <= 0 || (rot_dim > 0 && (!cos_sin || !mix_aligned16(cos_sin))) || !(eps >= 0.0f))
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
  // several warps a token while there are fewer than 16 warps an SM: 1, 2, 4 or 8,
  // so that a block's four warps, and the grid's, fall into whole tokens
  a.parts = 1;
  while (a.parts < 8 && (int64_t)num_tokens * a.parts * 2 <= (int64_t)sms * 16) a.parts *= 2;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == CCONV_DTYPE_F32
                              ? launch_nr_d<float>(a, D, interleaved != 0, sms, st)
                              : launch_nr_d<__nv_bfloat16>(a, D, interleaved != 0, sms, st);
  return err == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}
