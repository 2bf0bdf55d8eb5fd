// Entry points attn_norm_rope_cache and attn_norm_rope_cache_q8: per-head RMS norm
// of q and k, rotation by position, and the write of k and v into the paged cache,
// in one pass.
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
// first group of keys and values, and the blocks' warps take the tokens one after the
// other, the next token's position and slot read ahead. 33024 tokens of 16 + 4 + 4
// heads of 128 in bf16: 73.0 us for 422 MB, 5.8 TB/s (keys after the queries, values
// after the keys: 5 % more; one unit a lane: 30 % more). 61 tokens: 3.0 us, the latency
// of a few dependent loads.
//
// An SM holds three blocks or four (`blocks_of`). Three spill nothing in bf16 and are 3
// to 15 % faster for as many steps; four have fewer steps in turn for some numbers of
// tokens, and then are faster: 2100 tokens of the heads above 8.6 us where three take
// 10.0, in fp32 11.4 and 14.3; 16000 in fp32 62.9 and 66.6.
//
// Into a cache in 8 bits a row's largest magnitude is reduced over the head's lanes
// as its sum of squares is, and a unit of 16 bytes becomes one of 8 (4 from fp32). The
// same tokens: 75.1 us for 389 MB, 5.2 TB/s (the 8 bytes in one store instead of two: the
// same): the second reduction, the conversions and the narrower stores cost the
// instructions what the bytes save.
#include "q8.cuh"

namespace cconv {
namespace {

constexpr int kNrThreads = 128;
constexpr int kUnroll = 4;      // groups of heads whose loads are in flight together
constexpr int kBatch = 32 * 2 * 16 * kUnroll;   // bytes of queries that a warp loads together

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
  bool ahead;         // the next token's queries are asked into the L2
  char* qo;
  int32_t* dev_err;
  uint8_t *ksc, *vsc;   // of a cache in 8 bits
  int64_t c_page, c_tok, c_head;
};

template <typename T, int D, bool PAIRS, bool Q8, int BLOCKS>
__global__ void __launch_bounds__(kNrThreads, BLOCKS) norm_rope_kernel(const NrArgs a) {
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
      if (BLOCKS == 3 && a.ahead) // its queries to the L2, whose latency it then waits for
        for (int at = lane * 128; at < a.Hq * (D * E); at += 32 * 128)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + t * a.q_rs * E + at));
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
    uint8_t *kscale = nullptr, *vscale = nullptr;
    constexpr int CE = Q8 ? 1 : E;              // bytes of a cached value
    if (sl >= 0) {
      const int page = sl / a.page_size;
      const int64_t off = (page * a.s_page + (int64_t)(sl - page * a.page_size) * a.s_tok) * CE;
      kdst = a.kc + off;
      vdst = a.vc + off;
      if constexpr (Q8) {
        const int64_t to = page * a.c_page + (int64_t)(sl - page * a.page_size) * a.c_tok;
        kscale = a.ksc + to;
        vscale = a.vsc + to;
      }
    }
    // a head's row to 8 bits, of which the lane has columns from b0 and b1 on
    auto store_q8 = [&](float (&x0)[V], float (&x1)[V], char* dst, int b0, int b1, uint8_t* scale,
                        bool in) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x0[e] = q8_in(x0[e]);
        x1[e] = q8_in(x1[e]);
        m = fmaxf(m, fmaxf(fabsf(x0[e]), fabsf(x1[e])));
      }
#pragma unroll
      for (int d = LPH / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      const uint32_t byte = q8_byte(m);
      const float f = q8_factor(byte);
      if (!in) return;
      if (byte >= kQ8Top)
#pragma unroll
        for (int e = 0; e < V; ++e) x0[e] = q8_top(x0[e]), x1[e] = q8_top(x1[e]);
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        *reinterpret_cast<uint32_t*>(dst + b0 + e) =
            pack_e4m3x4(x0[e] * f, x0[e + 1] * f, x0[e + 2] * f, x0[e + 3] * f);
        *reinterpret_cast<uint32_t*>(dst + b1 + e) =
            pack_e4m3x4(x1[e] * f, x1[e + 1] * f, x1[e + 2] * f, x1[e + 3] * f);
      }
      if (l == 0) *scale = (uint8_t)byte;
    };
    // one group of heads: norm and rotation
    auto rotate = [&](const uint4& u0, const uint4& u1, const float (&w0)[V], const float (&w1)[V],
                      bool norm, float (&y0)[V], float (&y1)[V]) {
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
    };
    // (`in`: the lane's head exists)
    auto store = [&](const float (&y0)[V], const float (&y1)[V], char* dst, bool in) {
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
        float y0[V], y1[V];
        rotate(u0[j], u1[j], w0, w1, a.qw != nullptr, y0, y1);
        store(y0, y1, qd + (int64_t)h * (D * E), h < qe);
      }
    }
    unpack16<T>(wk[0], w0);
    unpack16<T>(wk[1], w1);
#pragma unroll 1
    for (int h0 = kb; h0 < ke; h0 += HPW) {
      const int h = h0 + sub;
      const int64_t to = (int64_t)h * a.s_head * CE, sc = Q8 ? h * a.c_head : 0;
      if constexpr (Q8) {
        float x0[V], x1[V];
        unpack16<T>(vu0, x0);
        unpack16<T>(vu1, x1);
        store_q8(x0, x1, vdst + to, l * V, (LPH + l) * V, vscale + sc, h < ke);
      } else if (h < ke) {
        stg16(vdst + to + v0, vu0);
        stg16(vdst + to + v1, vu1);
      }
      const uint4 k0 = ku0, k1 = ku1;
      const int64_t next = (int64_t)(h + HPW) * (D * E);
      load(ks + next, h + HPW < ke, ku0, ku1, c0 * E, c1 * E);
      load(vs + next, h + HPW < ke, vu0, vu1, v0, v1);
      float y0[V], y1[V];
      rotate(k0, k1, w0, w1, a.kw != nullptr, y0, y1);
      if constexpr (Q8)
        store_q8(y0, y1, kdst + to, c0, c1, kscale + sc, h < ke);
      else
        store(y0, y1, kdst + to, h < ke);
    }
  }
}

// Warps of a token, for `slots` of them at work at once: several while that leaves all of
// them at work at once, 1, 2, 4 or 8, so that a block's four warps, and the grid's, fall
// into whole tokens.
int parts_of(int64_t tokens, int64_t slots) {
  int p = 1;
  while (p < 8 && tokens * p * 2 <= slots) p *= 2;
  return p;
}
// The blocks of an SM: four where a warp then has fewer steps in turn, tokens one after
// the other and batches of its share of a token's queries. (With three: 1000 tokens in
// fp32, whose 8 KB of queries are two batches, 8.4 us where four blocks, with twice the
// warps a token, take 7.2.) `ahead`: tokens in turn ask for the next one's queries, in bf16
// where those are a batch at most, and queries, keys and values three quarters of one. With four
// turns or more that is worth three blocks: 16000 tokens 37.1 us (four blocks 38.7, three
// without 39.2), into 8 bits 38.8 (41.7, 40.6), of 16 + 4 heads of 64 (3 KB) 26.4 (27.7,
// 28.1). Queries of several batches, shorter rows, and fp32 are slower with it: 14000 tokens
// of 32 + 8 heads of 128 65.2 us, four blocks 59.9; 33024 of 8 + 1 49.1, four blocks 48.1.
// For as many steps three are faster in bf16, and in fp32, which spills with neither, for
// rows of several batches or where four would take more warps a token (else 2 to 7 % slower).
int blocks_of(const NrArgs& a, int D, int e, int sms, bool& ahead) {
  const int64_t row = (int64_t)a.Hq * D * e, batches = (row + kBatch - 1) / kBatch;
  int64_t turns = 0;
  int p = 0;
  auto steps = [&](int blocks) {
    const int64_t slots = (int64_t)sms * blocks * (kNrThreads / 32);
    p = parts_of(a.T, slots);
    turns = (a.T * (int64_t)p + slots - 1) / slots;
    return turns * ((batches + p - 1) / p);
  };
  const int64_t four = steps(4);
  const int p4 = p;
  const int64_t three = steps(3);
  ahead = e == 2 && row <= kBatch && row + 2LL * a.Hkv * D * e >= kBatch * 3 / 4 && turns > 1;
  if (e == 4 && four == three && p == p4 && (turns == 1 || batches == 1)) return 4;
  return four < three && !(ahead && turns >= 4) ? 4 : 3;
}

template <typename T, int D, bool Q8, int BLOCKS>
cudaError_t launch_nr(NrArgs& a, bool pairs, int sms, cudaStream_t st) {
  const int64_t per = kNrThreads / 32;
  a.parts = parts_of(a.T, sms * BLOCKS * per);
  const unsigned grid =
      (unsigned)std::min<int64_t>(((int64_t)a.T * a.parts + per - 1) / per, (int64_t)sms * BLOCKS);
  if (pairs)
    norm_rope_kernel<T, D, true, Q8, BLOCKS><<<grid, kNrThreads, 0, st>>>(a);
  else
    norm_rope_kernel<T, D, false, Q8, BLOCKS><<<grid, kNrThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, bool Q8, int BLOCKS>
cudaError_t launch_nr_d(NrArgs& a, int D, bool pairs, int sms, cudaStream_t st) {
  if (D == 64) return launch_nr<T, 64, Q8, BLOCKS>(a, pairs, sms, st);
  if (D == 128) return launch_nr<T, 128, Q8, BLOCKS>(a, pairs, sms, st);
  return launch_nr<T, 256, Q8, BLOCKS>(a, pairs, sms, st);
}

template <typename T, bool Q8>
cudaError_t launch_nr_b(NrArgs& a, int D, bool pairs, int sms, cudaStream_t st) {
  return blocks_of(a, D, Elem<T>::bytes, sms, a.ahead) == 4
             ? launch_nr_d<T, Q8, 4>(a, D, pairs, sms, st)
             : launch_nr_d<T, Q8, 3>(a, D, pairs, sms, st);
}

// What both entry points check and fill in; a's cache, and D, are set.
int norm_rope(NrArgs& a, int D, bool q8, const void* q, int64_t q_row_stride, const void* k,
              int64_t k_row_stride, const void* v, int64_t v_row_stride, const void* q_weight,
              const void* k_weight, float eps, const float* cos_sin, int32_t max_position,
              int32_t rot_dim, int32_t interleaved, const int32_t* positions,
              const int32_t* slot_mapping, int32_t num_tokens, int32_t num_q_heads, int32_t dtype,
              void* q_out, int64_t q_out_row_stride, int32_t* dev_err, cconv_stream_t stream) {
  const int e = mix_dtype_bytes(dtype), V = 16 / e;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 || (!interleaved && rot_dim % (2 * V)) ||
      max_position <= 0 || (rot_dim > 0 && (!cos_sin || !mix_aligned16(cos_sin))) || !(eps >= 0.0f))
    return CCONV_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(q_weight) % e || reinterpret_cast<uintptr_t>(k_weight) % e)
    return CCONV_ERR_INVALID;
  if (num_tokens == 0) return CCONV_OK;
  if (!mix_rows_ok(q, q_row_stride, (int64_t)num_q_heads * D, V) ||
      !mix_rows_ok(k, k_row_stride, (int64_t)a.Hkv * D, V) ||
      !mix_rows_ok(v, v_row_stride, (int64_t)a.Hkv * D, V) ||
      !mix_rows_ok(q_out, q_out_row_stride, (int64_t)num_q_heads * D, V) || !positions ||
      !slot_mapping)
    return CCONV_ERR_INVALID;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
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
  a.slots = slot_mapping;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.qo = static_cast<char*>(q_out);
  a.dev_err = dev_err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool pairs = interleaved != 0;
  cudaError_t err;
  if (dtype == CCONV_DTYPE_F32)
    err = q8 ? launch_nr_b<float, true>(a, D, pairs, sms, st)
             : launch_nr_b<float, false>(a, D, pairs, sms, st);
  else
    err = q8 ? launch_nr_b<__nv_bfloat16, true>(a, D, pairs, sms, st)
             : launch_nr_b<__nv_bfloat16, false>(a, D, pairs, sms, st);
  return err == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}

template <typename C>
void nr_cache(NrArgs& a, const C& cache) {
  a.kc = static_cast<char*>(cache.k);
  a.vc = static_cast<char*>(cache.v);
  a.s_page = cache.s_page, a.s_tok = cache.s_token, a.s_head = cache.s_head;
  a.page_size = cache.page_size;
  a.num_slots = (int64_t)cache.num_pages * cache.page_size;
  a.Hkv = cache.num_kv_heads;
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
  if (mix_dtype_bytes(dtype) == 0 || num_tokens < 0 || num_q_heads <= 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache(cache, dtype);
  if (rc != CCONV_OK) return rc;
  NrArgs a = {};
  nr_cache(a, cache);
  return norm_rope(a, cache.head_dim, false, q, q_row_stride, k, k_row_stride, v, v_row_stride,
                   q_weight, k_weight, eps, cos_sin, max_position, rot_dim, interleaved, positions,
                   slot_mapping, num_tokens, num_q_heads, dtype, q_out, q_out_row_stride, dev_err,
                   stream);
}

extern "C" int attn_norm_rope_cache_q8(const void* q, int64_t q_row_stride, const void* k,
                                       int64_t k_row_stride, const void* v, int64_t v_row_stride,
                                       const void* q_weight, const void* k_weight, float eps,
                                       const float* cos_sin, int32_t max_position, int32_t rot_dim,
                                       int32_t interleaved, const int32_t* positions,
                                       kv_cache_q8_t cache, const int32_t* slot_mapping,
                                       int32_t num_tokens, int32_t num_q_heads, int32_t dtype,
                                       void* q_out, int64_t q_out_row_stride, int32_t* dev_err,
                                       cconv_stream_t stream) {
  if (mix_dtype_bytes(dtype) == 0 || num_tokens < 0 || num_q_heads <= 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache_q8(cache);
  if (rc != CCONV_OK) return rc;
  NrArgs a = {};
  nr_cache(a, cache);
  a.ksc = cache.k_scale;
  a.vsc = cache.v_scale;
  a.c_page = cache.c_page, a.c_tok = cache.c_token, a.c_head = cache.c_head;
  return norm_rope(a, cache.head_dim, true, q, q_row_stride, k, k_row_stride, v, v_row_stride,
                   q_weight, k_weight, eps, cos_sin, max_position, rot_dim, interleaved, positions,
                   slot_mapping, num_tokens, num_q_heads, dtype, q_out, q_out_row_stride, dev_err,
                   stream);
}
