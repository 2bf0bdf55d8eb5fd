// The gated delta rule: arguments and host checks shared by the recurrent
// kernel (gdn_step.cu) and the chunked one (gdn_chunk.cu).
#pragma once

#include "mixer.cuh"

namespace cconv {

struct GdnArgs {
  const char *q, *k, *v, *a, *b;
  int64_t q_rs, k_rs, v_rs, a_rs, b_rs, out_rs;   // elements
  const float* A_log;
  const float* dt_bias;
  char* out;
  char* st;
  int64_t st_slot, st_head;   // elements
  int32_t num_slots;
  int32_t st_bytes;           // of a state element (chunked kernel)
  const int32_t* state_idx;
  const int32_t* cu;          // NULL: rows [s*q_len, s*q_len + q_len)
  const int32_t* num_acc;
  const uint8_t* has_init;
  int32_t B, T, Hk, Hv, q_len;
  int32_t max_len;            // the recurrent kernel's longest sequence; longer ones are
                              // the chunked kernel's (0: no limit)
  float scale;
  int32_t l2norm;
  int32_t* dev_err;
};

// Bounds of sequence s, or false (with the error flagged by the caller's
// choice) for a bad cu_seqlens entry.
__device__ __forceinline__ bool gdn_bounds(const GdnArgs& a, int s, int& st, int& len) {
  st = a.cu[s];
  const int en = a.cu[s + 1];
  len = en - st;
  return st >= 0 && en >= st && en <= a.T;
}

// Recurrent kernel over all sequences; see gdn_step.cu.
cudaError_t gdn_launch_step(const GdnArgs& a, int dtype, int state_dtype, int dk, int dv,
                            cudaStream_t st);

// Chunked kernel (bf16, dk = dv = 128) over the sequences longer than
// a.max_len; see gdn_chunk.cu.
cudaError_t gdn_launch_chunk(const GdnArgs& a, int state_dtype, cudaStream_t st);

}  // namespace cconv
