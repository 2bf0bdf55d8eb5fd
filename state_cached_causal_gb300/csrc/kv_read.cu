// Entry point kv_cache_read_q8: rows of a cache in 8 bits as fp32 or bf16.
//
// A thread turns 8 bytes (4 for fp32) of a row into the 16 it stores, so that both
// sides of a warp are whole lines, and has four such units requested before the first
// is stored: slots, then bytes and scales, depend on one another. 65536 rows of 4 heads
// of 128 to bf16 (202 MB): 47 us, 4.3 TB/s, of which two thirds are
// stores (with one unit a thread 56 us).
#include "q8.cuh"

namespace cconv {
namespace {

constexpr int kReadThreads = 256;
constexpr int kUnits = 4;         // of a thread, requested together

struct ReadArgs {
  const char *kc, *vc;
  int64_t s_page, s_tok, s_head;
  const uint8_t *ksc, *vsc;
  int64_t c_page, c_tok, c_head;
  int32_t page_size, page_shift, Hkv;
  int64_t num_slots;
  const int32_t* slots;
  int32_t T;
  char *ko, *vo;
  int64_t ko_rs, vo_rs;
  int32_t* dev_err;
};

template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a) {
  constexpr int V = Elem<T>::V, E = Elem<T>::bytes, UPR = D / V;    // units a row
  const uint32_t per = 2 * a.Hkv * UPR;                             // units of a token
  // a block's tokens at a time: units of 16 bytes for kUnits a thread, or one token
  const int tokens = max(1u, kReadThreads * kUnits / per);
#pragma unroll 1
  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.T; t0 += (int64_t)gridDim.x * tokens) {
    const uint32_t n = (uint32_t)min((int64_t)tokens, a.T - t0) * per;
#pragma unroll 1
    for (uint32_t j0 = threadIdx.x; j0 < n; j0 += kReadThreads * kUnits) {
      // slots, then values and scales, of all units before the first is stored
      int slot[kUnits];
      uint32_t raw[kUnits][V / 4], byte[kUnits];
      char* dst[kUnits];
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const uint32_t j = j0 + k * kReadThreads;
        slot[k] = j < n ? a.slots[t0 + j / per] : -1;
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const uint32_t j = j0 + k * kReadThreads, t = j / per;
        uint32_t r = j - t * per;
        const bool isv = r >= per / 2;
        if (isv) r -= per / 2;
        const int h = r / UPR, u = r % UPR;
        if (slot[k] >= a.num_slots) {
          flag_error(a.dev_err, CCONV_DERR_POSITION);
          slot[k] = -1;
        }
        if (slot[k] < 0) continue;
        const int page = a.page_shift >= 0 ? slot[k] >> a.page_shift : slot[k] / a.page_size;
        const int tok = slot[k] - page * a.page_size;
        const char* const src = (isv ? a.vc : a.kc) + page * a.s_page + tok * a.s_tok +
                                h * a.s_head + u * V;
        if constexpr (V == 8) {
          const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src));
          raw[k][0] = w.x, raw[k][V / 4 - 1] = w.y;
        } else {
          raw[k][0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
        }
        byte[k] = (isv ? a.vsc : a.ksc)[page * a.c_page + tok * a.c_tok + h * a.c_head];
        dst[k] = (isv ? a.vo + (t0 + t) * a.vo_rs * E : a.ko + (t0 + t) * a.ko_rs * E) +
                 (int64_t)r * 16;
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        if (slot[k] < 0) continue;
        const float f = q8_scale(byte[k]);
        float x[V];
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          float y[4];
          unpack_e4m3x4(raw[k][e / 4], y);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[e + i] = y[i] * f;
        }
        stg16(dst[k], pack16<T>(x));
      }
    }
  }
}

template <typename T>
cudaError_t launch_read(const ReadArgs& a, int D, int sms, cudaStream_t st) {
  const int64_t n = (int64_t)a.T * 2 * a.Hkv * (D / Elem<T>::V), per = kReadThreads * kUnits;
  const unsigned grid = (unsigned)std::min<int64_t>((n + per - 1) / per, (int64_t)sms * 64);
  if (D == 64)
    kv_read_kernel<T, 64><<<grid, kReadThreads, 0, st>>>(a);
  else if (D == 128)
    kv_read_kernel<T, 128><<<grid, kReadThreads, 0, st>>>(a);
  else
    kv_read_kernel<T, 256><<<grid, kReadThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace cconv

using namespace cconv;

extern "C" int kv_cache_read_q8(kv_cache_q8_t cache, const int32_t* slot_mapping,
                                int32_t num_tokens, int32_t dtype, void* k_out,
                                int64_t k_out_row_stride, void* v_out, int64_t v_out_row_stride,
                                int32_t* dev_err, cconv_stream_t stream) {
  const int e = mix_dtype_bytes(dtype);
  if (e == 0 || num_tokens < 0) return CCONV_ERR_INVALID;
  const int rc = mix_check_cache_q8(cache);
  if (rc != CCONV_OK) return rc;
  if (num_tokens == 0) return CCONV_OK;
  const int64_t row = (int64_t)cache.num_kv_heads * cache.head_dim;
  if (!slot_mapping || !mix_rows_ok(k_out, k_out_row_stride, row, 16 / e) ||
      !mix_rows_ok(v_out, v_out_row_stride, row, 16 / e) || row > INT32_MAX / 4)
    return CCONV_ERR_INVALID;
  const int sms = mix_sm_count();
  if (sms <= 0) return CCONV_ERR_LAUNCH;
  ReadArgs a;
  a.kc = static_cast<const char*>(cache.k);
  a.vc = static_cast<const char*>(cache.v);
  a.s_page = cache.s_page, a.s_tok = cache.s_token, a.s_head = cache.s_head;
  a.ksc = cache.k_scale;
  a.vsc = cache.v_scale;
  a.c_page = cache.c_page, a.c_tok = cache.c_token, a.c_head = cache.c_head;
  a.page_size = cache.page_size;
  a.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (cache.page_size == 1 << s) a.page_shift = s;
  a.Hkv = cache.num_kv_heads;
  a.num_slots = (int64_t)cache.num_pages * cache.page_size;
  a.slots = slot_mapping;
  a.T = num_tokens;
  a.ko = static_cast<char*>(k_out);
  a.vo = static_cast<char*>(v_out);
  a.ko_rs = k_out_row_stride, a.vo_rs = v_out_row_stride;
  a.dev_err = dev_err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == CCONV_DTYPE_F32
                              ? launch_read<float>(a, cache.head_dim, sms, st)
                              : launch_read<__nv_bfloat16>(a, cache.head_dim, sms, st);
  return err == cudaSuccess ? CCONV_OK : CCONV_ERR_LAUNCH;
}
