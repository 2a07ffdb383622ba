// k_rope_append.hip -- per-head RMS norm of q and k, rotary positions, and the
// append of k and v to the paged cache, in one launch.
//
// Mathematics.  One head row x of dim D: r = (mean x^2 + eps)^-1/2, n = x r w,
// then pairs (i, i + rot/2) or (2i, 2i + 1) turn by the angle p f_i.  The
// angle is formed in fp64 in half turns, a = p (f_i / pi), and reduced by
// a - 2 rint(a / 2) there, so that a position of 10^6 keeps the angle to 1e-9;
// sine and cosine are then taken in fp32.
//
// Layout.  A row is D * esz bytes; each lane holds 16 of them, so a wave holds
// 1 to 8 rows and its norm is a reduction inside those lanes.  A lane's place
// in the row is the same for every row it handles, so its cosines and sines
// are computed once per token.  A rotated pair of the half layout lies
// rot / 2 values apart: rot is a multiple of 16, so the partner of every value
// of a lane lies in one other lane (one cross-lane read each).
//
// V goes transposed into its page, so its workgroups take kVTokens tokens by
// kVCols columns through LDS and write 8 consecutive tokens of one column at
// once where their slots are consecutive and 8-aligned, single values where
// not (the ends of a run, padding tokens).
//
// Bound: bytes (every value read and written once); launch latency for a few
// tokens.  4099 fp32 tokens of 28 heads of 256: 176 MB in 52 us = 3.4 TB/s (the
// V workgroups cost 4.5 of them, forming the angles 7; two workgroups per token
// 59 us, rows asked for two to five passes ahead 53 to 56), or 39 us on the
// tensors of the call before, which the last-level cache holds in part; 64 bf16
// tokens 6.0 us; one token 4.4 us, the launch.
#include <algorithm>

#include "seq.h"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kVTokens = 128;
constexpr int kVCols = 64;

struct RopeParams {
  tq_rope_append_args a;
  int rows_per_pass;  // head rows that one workgroup takes at a time
  int splits;         // workgroups per token
  int64_t v_blocks;   // workgroups at the front of the grid that move V
  int page_shift;
};

// true and the page, place of a token's slot, if it is to be stored
__device__ inline bool slot_of(const RopeParams& p, int64_t slot, int64_t* page, int* at) {
  *page = slot >> p.page_shift;
  *at = (int)(slot & (p.a.page - 1));
  return slot >= 0 && *page < p.a.pages;
}

template <typename IN, typename C>
__device__ void move_v(const RopeParams& p, int64_t block, C* lds) {
  const auto& a = p.a;
  constexpr int VEC = 16 / sizeof(IN);
  constexpr int kRow = kVCols + 2;  // 2 values of padding: columns 8 tokens apart fall on different banks
  const int slices = a.dim / kVCols;
  const int slice = (int)(block % slices);
  const int64_t rest = block / slices;
  const int head = (int)(rest % a.kv_heads);
  const int64_t t0 = rest / a.kv_heads * kVTokens;
  const int n = (int)min((int64_t)kVTokens, a.tokens - t0);
  const IN* v = static_cast<const IN*>(a.v) + head * a.v_head + slice * kVCols;
  for (int i = threadIdx.x; i < n * (kVCols / VEC); i += kThreads) {
    const int t = i / (kVCols / VEC), c = i % (kVCols / VEC) * VEC;
    const Vec<IN, VEC> x = *reinterpret_cast<const Vec<IN, VEC>*>(v + (t0 + t) * a.v_token + c);
#pragma unroll
    for (int j = 0; j < VEC; ++j) lds[t * kRow + c + j] = (C)(float)x.v[j];
  }
  __syncthreads();
  // groups of 8 tokens start where the first token's slot reaches a multiple of 8
  const int shift = (int)(a.slots[t0] & 7);
  C* cache = static_cast<C*>(a.v_cache);
  const int groups = (n + shift + 7) / 8;
  for (int i = threadIdx.x; i < groups * kVCols; i += kThreads) {
    const int col = i % kVCols, first = i / kVCols * 8 - shift;
    const int64_t s0 = first >= 0 ? a.slots[t0 + first] : -1;
    bool run = first >= 0 && first + 8 <= n && s0 >= 0 && (s0 & 7) == 0;
    if (run)
      for (int j = 1; j < 8; ++j) run = run && a.slots[t0 + first + j] == s0 + j;
    int64_t page;
    int at;
    if (run) {
      if (!slot_of(p, s0, &page, &at)) {
        raise_flag(a.bad_flag);
        continue;
      }
      Vec<C, 8> o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = lds[(first + j) * kRow + col];
      *reinterpret_cast<Vec<C, 8>*>(cache + ((page * a.kv_heads + head) * a.dim + slice * kVCols + col) * a.page + at) = o;
      continue;
    }
    for (int t = max(first, 0); t < min(first + 8, n); ++t) {
      const int64_t s = a.slots[t0 + t];
      if (slot_of(p, s, &page, &at))
        cache[((page * a.kv_heads + head) * a.dim + slice * kVCols + col) * a.page + at] = lds[t * kRow + col];
      else if (s >= 0)
        raise_flag(a.bad_flag);
    }
  }
}

template <typename IN, typename C, int D>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeParams p) {
  constexpr int VEC = 16 / sizeof(IN);
  constexpr int LPR = D / VEC;  // lanes per row
  __shared__ __attribute__((aligned(16))) char lds[kVTokens * (kVCols + 2) * 2];
  const auto& a = p.a;
  if ((int64_t)blockIdx.x < p.v_blocks) {
    move_v<IN, C>(p, blockIdx.x, reinterpret_cast<C*>(lds));
    return;
  }
  const int64_t block = (int64_t)blockIdx.x - p.v_blocks;
  const int64_t t = block / p.splits;
  const int rows = a.heads + a.kv_heads;
  const int lane = threadIdx.x % LPR, first = (int)(block % p.splits) * p.rows_per_pass + threadIdx.x / LPR;
  const int step = p.splits * p.rows_per_pass;
  const int c0 = lane * VEC, half = a.rot / 2;
  const bool turned = c0 < a.rot, inter = a.layout == TQ_ROPE_INTERLEAVED;
  const bool upper = !inter && c0 >= half;

  Vec<IN, VEC> x;
  auto row = [&](int r) {
    return r < a.heads ? static_cast<const IN*>(a.q) + t * a.q_token + r * a.q_head
                       : static_cast<const IN*>(a.k) + t * a.k_token + (r - a.heads) * a.k_head;
  };
  if (first < rows) x = *reinterpret_cast<const Vec<IN, VEC>*>(row(first) + c0);

  float cs[VEC], sn[VEC];
  if (turned) {
    const double pos = (double)a.positions[t];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (inter && (j & 1)) {
        cs[j] = cs[j - 1];
        sn[j] = -sn[j - 1];
        continue;
      }
      const int i = inter ? (c0 + j) / 2 : c0 + j - (upper ? half : 0);
      double turn = pos * (a.inv_freq[i] * 0.31830988618379067154);  // in units of pi
      turn -= 2.0 * rint(turn * 0.5);
      float s, c;
      sincospif((float)turn, &s, &c);
      cs[j] = c * a.rope_scale;
      sn[j] = (inter || !upper ? -s : s) * a.rope_scale;  // sign of the partner's share
    }
  }
  float w[2][VEC];
  const bool normed[2] = {a.q_norm != nullptr, a.k_norm != nullptr};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* src = k ? a.k_norm : a.q_norm;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[k][j] = src ? src[c0 + j] : 1.f;
  }
  const int64_t slot = a.slots[t];
  int64_t page;
  int at;
  const bool stored = slot_of(p, slot, &page, &at);
  if (!stored && slot >= 0 && threadIdx.x == 0) raise_flag(a.bad_flag);
  // the lane that holds the partners of this lane's values (half layout)
  const int wave_lane = threadIdx.x & 63;
  const int partner = wave_lane - lane + (!turned || inter ? lane : upper ? lane - half / VEC : lane + half / VEC);

  // every lane of a wave runs the same number of passes: the cross-lane reads need all of them
  for (int base = (int)(block % p.splits) * p.rows_per_pass; base < rows; base += step) {
    const int r = base + threadIdx.x / LPR;
    const bool live = r < rows;
    Vec<IN, VEC> next = x;
    if (r + step < rows) next = *reinterpret_cast<const Vec<IN, VEC>*>(row(r + step) + c0);
    float f[VEC];
    const int kind = r < a.heads ? 0 : 1;
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = live ? (float)x.v[j] : 0.f;
    if (normed[0] || normed[1]) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) s = fmaf(f[j], f[j], s);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
      const float rs = 1.f / sqrtf(s * (1.f / D) + a.eps);
      if (normed[kind])
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = f[j] * rs * (kind ? w[1][j] : w[0][j]);
    }
    float y[VEC];
    if (a.rot > 0) {
      float other[VEC];
      if (inter) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) other[j] = f[j ^ 1];
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) other[j] = __shfl(f[j], partner, 64);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[j] = turned ? fmaf(f[j], cs[j], other[j] * sn[j]) : f[j];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[j] = f[j];
    }
    if (live && (kind == 0 || stored)) {
      Vec<C, VEC> o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) o.v[j] = (C)y[j];
      C* dst = kind == 0 ? static_cast<C*>(a.q_out) + (t * a.heads + r) * D
                         : static_cast<C*>(a.k_cache) + ((page * a.kv_heads + (r - a.heads)) * a.page + at) * D;
      *reinterpret_cast<Vec<C, VEC>*>(dst + c0) = o;
    }
    x = next;
  }
}

template <typename IN, typename C>
hipError_t launch(const tq_rope_append_args& a, hipStream_t s) {
  RopeParams p{a};
  const int rows = a.heads + a.kv_heads;
  p.rows_per_pass = kThreads / (a.dim * (int)sizeof(IN) / 16);
  // Few tokens: a workgroup per pass, so that no row waits for another; many: one workgroup per token, whose passes
  // share the angles.  2048 workgroups fill the 256 compute units eight deep.
  const int passes = (rows + p.rows_per_pass - 1) / p.rows_per_pass;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(passes, 2048 / a.tokens));
  p.v_blocks = (a.tokens + kVTokens - 1) / kVTokens * a.kv_heads * (a.dim / kVCols);
  p.page_shift = __builtin_ctz(a.page);
  const dim3 grid((unsigned)(p.v_blocks + a.tokens * p.splits));
  if (a.dim == 64) hipLaunchKernelGGL((rope_append_kernel<IN, C, 64>), grid, dim3(kThreads), 0, s, p);
  if (a.dim == 128) hipLaunchKernelGGL((rope_append_kernel<IN, C, 128>), grid, dim3(kThreads), 0, s, p);
  if (a.dim == 256) hipLaunchKernelGGL((rope_append_kernel<IN, C, 256>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

template <typename IN>
hipError_t launch_in(const tq_rope_append_args& a, hipStream_t s) {
  return a.cache_type == TQ_BF16 ? launch<IN, bf16>(a, s) : launch<IN, f16>(a, s);
}

}  // namespace

hipError_t launch_rope_append(const tq_rope_append_args& a, hipStream_t s) {
  return a.in_type == TQ_F32 ? launch_in<float>(a, s) : a.in_type == TQ_BF16 ? launch_in<bf16>(a, s) : launch_in<f16>(a, s);
}

}  // namespace tq
