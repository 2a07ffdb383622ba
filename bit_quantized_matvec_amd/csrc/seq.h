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
int paged_attn_tile_rows(int64_t tokens, int64_t seqs, int64_t max_len, int heads, int kv_heads, int dim);
hipError_t launch_paged_attn(const tq_paged_attn_args& a, hipStream_t s);

int64_t gdn_workspace_bytes(int64_t tokens, int64_t seqs, int64_t max_len, int v_heads, int dk, int dv);
hipError_t launch_gdn(const tq_gdn_args& a, hipStream_t s);
// k_gdn_chunk.hip: whether a call's longest sequence is worth chunks, and the call
bool gdn_chunked(int64_t tokens, int64_t seqs, int64_t max_len);
int64_t gdn_chunk_workspace_bytes(int64_t tokens, int64_t seqs, int64_t max_len, int v_heads, int dk, int dv);
hipError_t launch_gdn_chunk(const tq_gdn_args& a, hipStream_t s);

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

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

// Two fp32 values rounded to a 16-bit type, and back.
template <typename C>
__device__ inline unsigned pack2(float x, float y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef C c2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), c2));
}
template <typename C>
__device__ inline void unpack2(unsigned u, float* x, float* y) {
  if constexpr (__is_same(C, bf16)) {
    *x = __uint_as_float(u << 16), *y = __uint_as_float(u & 0xFFFF0000u);
  } else {
    typedef C c2 __attribute__((ext_vector_type(2)));
    const c2 v = __builtin_bit_cast(c2, u);
    *x = (float)v[0], *y = (float)v[1];
  }
}

// N fp32 values (a multiple of 2) as TERMS vectors of a 16-bit type whose sum holds as many bits as the terms have together.
template <int TERMS, typename VEC>
__device__ inline void split_terms(const float* p, VEC* out) {
  typedef __typeof__(VEC{}[0]) C;
  constexpr int N = sizeof(VEC) / 4;
  typedef unsigned words __attribute__((ext_vector_type(N)));
  words w[TERMS];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x = p[2 * i], y = p[2 * i + 1];
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      w[t][i] = pack2<C>(x, y);
      if (t + 1 < TERMS) {
        float u, v;
        unpack2<C>(w[t][i], &u, &v);
        x -= u, y -= v;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TERMS; ++t) out[t] = __builtin_bit_cast(VEC, w[t]);
}

// Tiles of `rows` rows over the sequences: sequence b's are the slots from cu[b] * per / rows + add * b on, an upper bound
// for what the sequences before it need.  The largest b whose first slot is at most `slot`, 64 candidates at a time.
__device__ inline int64_t first_slot(const int32_t* cu, int64_t b, int per, int rows, int add) { return (int64_t)cu[b] * per / rows + add * b; }
__device__ inline int find_seq(const int32_t* cu, int64_t seqs, int per, int rows, int add, int64_t slot, int lane) {
  int64_t lo = 0, n = seqs;
  while (n > 1) {
    const int64_t step = (n + 63) / 64, i = lo + lane * step;
    const bool ok = lane * step < n && first_slot(cu, i, per, rows, add) <= slot;
    const int64_t last = max(1, __popcll(__ballot(ok))) - 1;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return __builtin_amdgcn_readfirstlane((int)lo);
}
#endif

}  // namespace tq
