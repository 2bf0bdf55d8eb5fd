// Entry point kv_cache_read_q8: rows of a cache in 8 bits as fp32 or bf16.
//
// A thread turns 8 bytes (4 for fp32) of a row into the 16 it stores, so that both
// sides of a warp are whole lines. It is bound by HBM.
#include "q8.cuh"

namespace cconv {
namespace {

constexpr int kReadThreads = 256;

struct ReadArgs {
  const char *kc, *vc;
  int64_t s_page, s_tok, s_head;
  const uint8_t *ksc, *vsc;
  int64_t c_page, c_tok, c_head;
  int32_t page_size, Hkv;
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
  const int64_t per = (int64_t)2 * a.Hkv * UPR, n = a.T * per;
  for (int64_t i = (int64_t)blockIdx.x * kReadThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kReadThreads) {
    const int64_t t = i / per;
    int r = (int)(i - t * per);
    const bool isv = r >= a.Hkv * UPR;
    if (isv) r -= a.Hkv * UPR;
    const int h = r / UPR, u = r % UPR, slot = a.slots[t];
    if (slot < 0 || slot >= a.num_slots) {
      if (slot >= 0) flag_error(a.dev_err, CCONV_DERR_POSITION);
      continue;
    }
    const int page = slot / a.page_size, tok = slot - page * a.page_size;
    const char* const src = (isv ? a.vc : a.kc) + page * a.s_page + tok * a.s_tok +
                            h * a.s_head + u * V;
    const float f = q8_scale((isv ? a.vsc : a.ksc)[page * a.c_page + tok * a.c_tok +
                                                   h * a.c_head]);
    float x[V];
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      float y[4];
      unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(src + e), y);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[e + j] = y[j] * f;
    }
    char* const dst = isv ? a.vo + t * a.vo_rs * E : a.ko + t * a.ko_rs * E;
    stg16(dst + (int64_t)r * 16, pack16<T>(x));
  }
}

template <typename T>
cudaError_t launch_read(const ReadArgs& a, int D, int sms, cudaStream_t st) {
  const int64_t n = (int64_t)a.T * 2 * a.Hkv * (D / Elem<T>::V);
  const unsigned grid =
      (unsigned)std::min<int64_t>((n + kReadThreads - 1) / kReadThreads, (int64_t)sms * 8);
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
