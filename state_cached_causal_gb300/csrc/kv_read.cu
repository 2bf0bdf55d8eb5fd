// Entry point kv_cache_read_q8: rows of a cache in 8 bits as fp32 or bf16.
//
// A thread turns 8 bytes (4 for fp32) of a row into the 16 it stores, so that both
// sides of a warp are whole lines. It takes the same unit of one token after the other,
// so that where that lies in a token is computed once, and has four tokens' bytes and
// scales requested before the first is stored, and their successors' slots. 65536 rows
// of 4 heads of 128 to bf16 (202 MB): 41 us, 4.9 TB/s, two thirds of it stores. The issue
// slots bound it, at 68 %, more than HBM, at 49 %: two conversions, two multiplications and
// a pack for two values. (Units dealt out in their order, with two divisions each: 47 us and
// 81 % of the issue slots; slots not read ahead: 50 us; two or eight tokens, twice the bytes
// a thread: 40 to 41.)
#include "q8.cuh"

namespace cconv {
namespace {

constexpr int kReadThreads = 256;
constexpr int kBlocks = 20;       // an SM (five: 45 us; 64: 45)
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
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a, const int cols,
                                                               const uint32_t wide) {
  constexpr int V = Elem<T>::V, E = Elem<T>::bytes, UPR = D / V;    // units a row
  const int per = 2 * a.Hkv * UPR;                                  // units of a token
  // the thread's unit of every token that it takes: K or V, head and place in that
  const int rows = blockDim.x / cols, row = threadIdx.x / cols;
  const uint32_t chunk = blockIdx.x / wide, block = blockIdx.x - chunk * wide;
  const int j = chunk * cols + threadIdx.x - row * cols;
  if (j >= per) return;
  const bool isv = j >= per / 2;
  const int r = isv ? j - per / 2 : j, h = r / UPR, u = r % UPR;
  const char* const src0 = (isv ? a.vc : a.kc) + h * a.s_head + u * V;
  const uint8_t* const scale0 = (isv ? a.vsc : a.ksc) + h * a.c_head;
  const int64_t rs = (isv ? a.vo_rs : a.ko_rs) * E;
  char* const dst0 = (isv ? a.vo : a.ko) + (int64_t)r * 16;
  const int64_t step = (int64_t)rows * kUnits;                      // tokens of a block at a time
  int32_t next[kUnits];             // slots, read a step ahead
  auto look = [&](int64_t t0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) next[k] = t0 + k * rows < a.T ? a.slots[t0 + k * rows] : -1;
  };
  int64_t t0 = block * step + row;
  look(t0);
#pragma unroll 1
  for (; t0 < a.T; t0 += wide * step) {
    // values and scales of all units before the first is stored
    int slot[kUnits];
    uint32_t raw[kUnits][V / 4], byte[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) slot[k] = next[k];
    look(t0 + wide * step);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (slot[k] >= a.num_slots) {
        flag_error(a.dev_err, CCONV_DERR_POSITION);
        slot[k] = -1;
      }
      if (slot[k] < 0) continue;
      const int page = a.page_shift >= 0 ? slot[k] >> a.page_shift : slot[k] / a.page_size;
      const int tok = slot[k] - page * a.page_size;
      const char* const src = src0 + page * a.s_page + tok * a.s_tok;
      if constexpr (V == 8) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src));
        raw[k][0] = w.x, raw[k][V / 4 - 1] = w.y;
      } else {
        raw[k][0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
      }
      byte[k] = scale0[page * a.c_page + tok * a.c_tok];
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
      stg16(dst0 + (t0 + k * rows) * rs, pack16<T>(x));
    }
  }
}

template <typename T>
cudaError_t launch_read(const ReadArgs& a, int D, int sms, cudaStream_t st) {
  const int per = 2 * a.Hkv * (D / Elem<T>::V);       // at most 2^28 (the caller checks)
  // a block takes all units of some tokens, or of one token as many as it has threads
  const int cols = std::min(per, kReadThreads), rows = kReadThreads / cols;
  const int chunks = (per + cols - 1) / cols;
  const int64_t most = ((int64_t)a.T + rows * kUnits - 1) / (rows * kUnits);
  const unsigned wide = (unsigned)std::min<int64_t>(most, std::max(sms * kBlocks / chunks, 1));
  const unsigned grid = wide * chunks;
  const int threads = cols * rows;
  if (D == 64)
    kv_read_kernel<T, 64><<<grid, threads, 0, st>>>(a, cols, wide);
  else if (D == 128)
    kv_read_kernel<T, 128><<<grid, threads, 0, st>>>(a, cols, wide);
  else
    kv_read_kernel<T, 256><<<grid, threads, 0, st>>>(a, cols, wide);
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
