// seq.h -- what the operators between a block's projections share: launchers
// (k_rope_append.hip, k_paged_attn*.hip, k_gdn*.hip) and small device helpers.
// Arguments are validated by seq_api.cpp before any launcher runs; what lies
// in device memory (offsets, pages, slots) is checked where it is read.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tq.h"

namespace tq {

hipError_t launch_rope_append(const tq_rope_append_args& a, hipStream_t s);

int64_t paged_attn_workspace_bytes(int64_t tokens, int64_t seqs, int heads, int kv_heads, int dim);
hipError_t launch_paged_attn(const tq_paged_attn_args& a, hipStream_t s);

int64_t gdn_workspace_bytes(int64_t tokens, int64_t seqs, int64_t max_len, int v_heads, int dk, int dv);
hipError_t launch_gdn(const tq_gdn_args& a, hipStream_t s);

inline int type_bytes(int t) { return t == TQ_F32 ? 4 : 2; }

#ifdef __HIPCC__
using bf16 = __bf16;
using f16 = _Float16;

// A range of the token axis, forced into [0, tokens].
struct SeqRange {
  int64_t t0;
  int n;
};

__device__ inline void raise_flag(int32_t* flag) {
  if (flag) *flag = 1;
}

__device__ inline SeqRange seq_range(const int32_t* cu, int64_t b, int64_t tokens, int32_t* flag) {
  if (!cu) return {b, 1};
  const int64_t lo = cu[b], hi = cu[b + 1];
  const int64_t t0 = lo < 0 ? 0 : lo > tokens ? tokens : lo;
  const int64_t t1 = hi < t0 ? t0 : hi > tokens ? tokens : hi;
  if (t0 != lo || t1 != hi) raise_flag(flag);
  return {t0, (int)(t1 - t0)};
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
#endif

}  // namespace tq
