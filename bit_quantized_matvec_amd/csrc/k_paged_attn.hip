// k_paged_attn.hip -- attention of new tokens over a paged cache: one wave per
// (token, query head), a key at a time with a running maximum and sum.
#include "seq.h"

namespace tq {
namespace {

template <typename C, typename O, int D>
__global__ __launch_bounds__(64) void attn_simple_kernel(tq_paged_attn_args a, int page_shift) {
  constexpr int E = D / 64;
  const int64_t row = blockIdx.x;
  const int64_t t = row / a.heads;
  const int h = (int)(row % a.heads), kvh = h / (a.heads / a.kv_heads), lane = threadIdx.x;
  int64_t b = 0;
  SeqRange r{0, 0};
  for (; b < a.seqs; ++b) {
    r = seq_range(a.cu, b, a.tokens, a.bad_flag);
    if (t >= r.t0 && t < r.t0 + r.n) break;
  }
  if (b == a.seqs) return;
  const int64_t len = min((int64_t)max(a.kv_len[b], 0), a.table_width << page_shift);
  if (len != a.kv_len[b]) raise_flag(a.bad_flag);
  const int64_t pos = len - r.n + (t - r.t0);
  const C* q = static_cast<const C*>(a.q) + t * a.q_token + h * a.q_head + lane * E;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = (float)q[e], o[e] = 0.f;
  for (int64_t j = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0; j <= pos; ++j) {
    const int64_t page = a.block_table[b * a.table_stride + (j >> page_shift)];
    if (page < 0 || page >= a.pages) {
      raise_flag(a.bad_flag);
      continue;
    }
    const int at = (int)(j & (a.page - 1));
    const C* k = static_cast<const C*>(a.k_cache) + ((page * a.kv_heads + kvh) * a.page + at) * D + lane * E;
    const C* v = static_cast<const C*>(a.v_cache) + ((page * a.kv_heads + kvh) * D + lane * E) * a.page + at;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], (float)k[e], s);
    s = wave_sum(s) * a.scale;
    const float mn = fmaxf(m, s), keep = m == -INFINITY ? 0.f : __expf(m - mn), p = __expf(s - mn);
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(p, (float)v[e * a.page], o[e] * keep);
    m = mn;
  }
  O* out = static_cast<O*>(a.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = (O)(l > 0.f ? o[e] / l : 0.f);
  if (a.lse && lane == 0) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename C, typename O>
hipError_t launch(const tq_paged_attn_args& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.tokens * a.heads));
  const int sh = __builtin_ctz(a.page);
  if (a.dim == 64) hipLaunchKernelGGL((attn_simple_kernel<C, O, 64>), grid, dim3(64), 0, s, a, sh);
  if (a.dim == 128) hipLaunchKernelGGL((attn_simple_kernel<C, O, 128>), grid, dim3(64), 0, s, a, sh);
  if (a.dim == 256) hipLaunchKernelGGL((attn_simple_kernel<C, O, 256>), grid, dim3(64), 0, s, a, sh);
  return hipGetLastError();
}

}  // namespace

int64_t paged_attn_workspace_bytes(int64_t, int64_t, int, int, int) { return 0; }

hipError_t launch_paged_attn(const tq_paged_attn_args& a, hipStream_t s) {
  if (a.cache_type == TQ_BF16) return a.out_type == TQ_F32 ? launch<bf16, float>(a, s) : launch<bf16, bf16>(a, s);
  return a.out_type == TQ_F32 ? launch<f16, float>(a, s) : launch<f16, f16>(a, s);
}

}  // namespace tq
