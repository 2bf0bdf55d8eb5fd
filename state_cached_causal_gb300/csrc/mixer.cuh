// Host checks and small device helpers shared by the operators that follow the
// convolutions (gated delta rule, head norm and rotation, paged attention).
#pragma once

#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace cconv {

inline bool mix_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A [rows, cols] argument of 16-byte vectors: pointer, row stride and alignment.
inline bool mix_rows_ok(const void* p, int64_t stride, int64_t cols, int V) {
  return p && mix_aligned16(p) && stride >= cols && stride % V == 0;
}

inline int mix_dtype_bytes(int dtype) {
  return dtype == CCONV_DTYPE_F32 ? 4 : dtype == CCONV_DTYPE_BF16 ? 2 : 0;
}

inline int mix_check_cache(const kv_cache_t& c, int dtype) {
  if (mix_dtype_bytes(c.dtype) == 0) return CCONV_ERR_INVALID;
  const int V = 16 / mix_dtype_bytes(c.dtype);
  if (!c.k || !c.v || !mix_aligned16(c.k) || !mix_aligned16(c.v)) return CCONV_ERR_INVALID;
  if (c.num_pages <= 0 || c.page_size <= 0 || c.num_kv_heads <= 0 || c.head_dim <= 0)
    return CCONV_ERR_INVALID;
  if (c.s_page <= 0 || c.s_token <= 0 || c.s_head <= 0 || c.s_page % V || c.s_token % V ||
      c.s_head % V)
    return CCONV_ERR_INVALID;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return CCONV_ERR_UNSUPPORTED;
  if (c.dtype != dtype) return CCONV_ERR_UNSUPPORTED;
  return CCONV_OK;
}

// SMs of the current device (looked up once per device), 0 on an error.
int mix_sm_count();
// Lets kernel `f` take as much shared memory as a block can have, once per
// device; `done` is the kernel's own.
cudaError_t mix_full_smem(const void* f, std::atomic<uint64_t>& done);

// 4 consecutive elements of storage type T <-> fp32.
template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 r = *reinterpret_cast<const float4*>(p);
    f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(r.x << 16);
    f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16);
    f[3] = __uint_as_float(r.y & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&f)[4]) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
template <typename T>
__device__ __forceinline__ float elem(const T* p, int64_t i) {
  return load_f32<T>(reinterpret_cast<const char*>(p), i);
}

// The gates of one token and value head: log decay and write strength.
__device__ __forceinline__ float gdn_softplus(float x) {
  return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float gdn_log_decay(float a, float A_log, float dt_bias) {
  return -expf(A_log) * gdn_softplus(a + dt_bias);
}
__device__ __forceinline__ float gdn_beta(float b) { return 1.0f / (1.0f + expf(-b)); }

constexpr float kGdnNormEps = 1e-6f;

}  // namespace cconv
