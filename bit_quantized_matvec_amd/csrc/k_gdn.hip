// k_gdn.hip -- the gated delta rule, token after token.
//
// Mathematics.  With r1 = S^T k and r2 = S^T q of the state before the token,
//   d = beta (v - e^g r1),  out = scale (e^g r2 + (k.q) d),  S <- e^g S + k (x) d,
// so both products are taken in one pass over S and each token needs one
// reduction.
//
// Split.  The columns of S are independent: a workgroup of 4 waves holds
// kCols = 32 columns of one head's state in registers, DK / 32 rows of 4
// columns per thread (a wave's load covers 8 rows of 128 bytes).  The
// sums over rows are 8 lanes wide in a wave and then 4 waves wide through LDS,
// which is double-buffered, so a token costs one barrier.
//
// Bound, one token: bytes of the state, read once and written once: 64
// sequences x 48 heads of 128 x 128, 403 MB, 78 us = 5.2 TB/s, what a large copy
// reaches; one sequence 4.5 us, the launch.  Long sequences go in chunks
// (k_gdn_chunk.hip); token after token 4096 of them take 6063 us.
#include <algorithm>

#include "seq.h"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 32;

template <typename IN, typename O, int DK>
__global__ __launch_bounds__(kThreads) void gdn_step_kernel(tq_gdn_args a) {
  constexpr int R = DK / 32;  // rows per thread
  __shared__ float sums[2][4][kCols * 2];
  const int slices = a.dv / kCols;
  const int slice = (int)(blockIdx.x % slices);
  const int64_t rest = blockIdx.x / slices;
  const int h = (int)(rest % a.v_heads);
  const int64_t b = rest / a.v_heads;
  const int kh = h / (a.v_heads / a.k_heads);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane % 8, row0 = (wave * 8 + lane / 8) * R;  // 4 columns from c * 4, R rows from row0

  const SeqRange r = seq_range(a.cu, b, a.tokens, a.bad_flag);
  const int64_t slot = a.slots ? a.slots[b] : b;
  const bool kept = slot >= 0 && slot < a.states;
  if (slot >= a.states) raise_flag(a.bad_flag);

  const int64_t at = (((kept ? slot : 0) * a.v_heads + h) * DK + row0) * (int64_t)a.dv + slice * kCols + c * 4;
  float s[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float4 x{0.f, 0.f, 0.f, 0.f};
    if (kept) x = *reinterpret_cast<const float4*>(a.state + at + i * (int64_t)a.dv);
    s[i][0] = x.x, s[i][1] = x.y, s[i][2] = x.z, s[i][3] = x.w;
  }

  for (int n = 0; n < r.n; ++n) {
    const int64_t t = r.t0 + n;
    const IN* qp = static_cast<const IN*>(a.q) + t * a.q_token + kh * a.q_head;
    const IN* kp = static_cast<const IN*>(a.k) + t * a.k_token + kh * a.k_head;
    const Vec<IN, R> qi = *reinterpret_cast<const Vec<IN, R>*>(qp + row0);
    const Vec<IN, R> ki = *reinterpret_cast<const Vec<IN, R>*>(kp + row0);
    const float g = a.g[t * a.v_heads + h], beta = a.beta[t * a.v_heads + h];
    const IN* vp = static_cast<const IN*>(a.v) + t * a.v_token + h * a.v_head + slice * kCols + c * 4;
    const Vec<IN, 4> vi = *reinterpret_cast<const Vec<IN, 4>*>(vp);
    // norms and k.q over the whole head: every wave reads all of it
    float qq = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
    for (int i = 0; i < DK / 64; ++i) {
      const float x = (float)qp[lane + 64 * i], y = (float)kp[lane + 64 * i];
      qq = fmaf(x, x, qq), kk = fmaf(y, y, kk), kq = fmaf(x, y, kq);
    }
    qq = wave_sum(qq), kk = wave_sum(kk), kq = wave_sum(kq);
    const float nq = (a.l2norm ? 1.f / sqrtf(qq + a.eps) : 1.f) * a.scale, nk = a.l2norm ? 1.f / sqrtf(kk + a.eps) : 1.f;
    const float decay = expf(g);
    float q[R], k[R], r1[4] = {}, r2[4] = {};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      q[i] = (float)qi.v[i] * nq, k[i] = (float)ki.v[i] * nk;
#pragma unroll
      for (int j = 0; j < 4; ++j) r1[j] = fmaf(s[i][j], k[i], r1[j]), r2[j] = fmaf(s[i][j], q[i], r2[j]);
    }
#pragma unroll
    for (int o = 8; o < 64; o <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) r1[j] += __shfl_xor(r1[j], o, 64), r2[j] += __shfl_xor(r2[j], o, 64);
    float(*buf)[kCols * 2] = sums[n & 1];
    if (lane < 8) {
      *reinterpret_cast<float4*>(&buf[wave][c * 8]) = float4{r1[0], r1[1], r1[2], r1[3]};
      *reinterpret_cast<float4*>(&buf[wave][c * 8 + 4]) = float4{r2[0], r2[1], r2[2], r2[3]};
    }
    __syncthreads();
    float d[4];
    Vec<O, 4> o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s1 = (buf[0][c * 8 + j] + buf[1][c * 8 + j]) + (buf[2][c * 8 + j] + buf[3][c * 8 + j]);
      const float s2 = (buf[0][c * 8 + 4 + j] + buf[1][c * 8 + 4 + j]) + (buf[2][c * 8 + 4 + j] + buf[3][c * 8 + 4 + j]);
      d[j] = beta * ((float)vi.v[j] - decay * s1);
      o.v[j] = (O)fmaf(kq * nq * nk, d[j], decay * s2);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = fmaf(k[i], d[j], decay * s[i][j]);
    if (wave == 0 && lane < 8)
      *reinterpret_cast<Vec<O, 4>*>(static_cast<O*>(a.out) + (t * a.v_heads + h) * a.dv + slice * kCols + c * 4) = o;
  }
  if (kept && (r.n > 0 || a.state_out != a.state))
#pragma unroll
    for (int i = 0; i < R; ++i)
      *reinterpret_cast<float4*>(a.state_out + at + i * (int64_t)a.dv) = float4{s[i][0], s[i][1], s[i][2], s[i][3]};
}

template <typename IN, typename O>
hipError_t launch_step(const tq_gdn_args& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.seqs * a.v_heads * (a.dv / kCols)));
  if (a.dk == 64) hipLaunchKernelGGL((gdn_step_kernel<IN, O, 64>), grid, dim3(kThreads), 0, s, a);
  if (a.dk == 128) hipLaunchKernelGGL((gdn_step_kernel<IN, O, 128>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int64_t gdn_workspace_bytes(int64_t tokens, int64_t seqs, int64_t max_len, int v_heads, int dk, int dv) {
  return gdn_chunked(tokens, seqs, max_len) ? gdn_chunk_workspace_bytes(tokens, seqs, max_len, v_heads, dk, dv) : 0;
}

hipError_t launch_gdn(const tq_gdn_args& a, hipStream_t s) {
  if (a.workspace && a.cu && gdn_chunked(a.tokens, a.seqs, a.max_len)) return launch_gdn_chunk(a, s);
  switch (a.in_type) {
    case TQ_F32: return launch_step<float, float>(a, s);
    case TQ_BF16: return a.out_type == TQ_F32 ? launch_step<bf16, float>(a, s) : launch_step<bf16, bf16>(a, s);
    default: return a.out_type == TQ_F32 ? launch_step<f16, float>(a, s) : launch_step<f16, f16>(a, s);
  }
}

}  // namespace tq
