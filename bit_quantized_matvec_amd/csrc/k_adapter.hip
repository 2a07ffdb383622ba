// k_adapter.hip -- low-rank adapters of many requests beside a shared
// projection: out[t] = y[t] + scale_i B_i (A_i x[t]).
//
// Tokens are sorted by adapter (expert_lists), then two kernels take tiles of
// 16 tokens of one adapter:
//   shrink: h = A_i x on 16x16x32 matrix instructions, the columns split over
//     workgroups (partial sums, added by the second kernel) and a workgroup's
//     waves (added through LDS);
//   expand: y + scale B_i h, 16 tokens x 64 features per wave.
// Memory bounds both: a token's x, y and out and an adapter's A and B are read
// or written once (A and B once per tile of its tokens, from the L2).
//
// Precision: fp32 factors are split into three bf16 terms (24 bits), fp16
// weights beside them into two (11 bits, exactly); term products below 2^-24 of
// the largest are left out.  Where x has the weights' type its products are
// exact as they are.  Sums are fp32.
#include <algorithm>

#include "batch.h"
#include "lists.h"
#include "seq.h"

namespace tq {
namespace {

typedef bf16 b8 __attribute__((ext_vector_type(8)));
typedef f16 h8 __attribute__((ext_vector_type(8)));

constexpr int kTok = 16;
constexpr int kWaves = 4;
constexpr int kFeat = 64;  // features per wave of expand

// 8 values as TERMS bf16 vectors.  A term that is not finite leaves nothing behind it.
template <int TERMS>
__device__ inline void terms8(const float* p, b8* out) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = p[i];
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack2<bf16>(x[2 * i], x[2 * i + 1]);
      if (t + 1 < TERMS) {
        float u, v;
        unpack2<bf16>(w[i], &u, &v);
        x[2 * i] = fabsf(u) < INFINITY ? x[2 * i] - u : 0.0f;
        x[2 * i + 1] = fabsf(v) < INFINITY ? x[2 * i + 1] - v : 0.0f;
      }
    }
    out[t] = __builtin_bit_cast(b8, w);
  }
}

// acc += w x over 32 places: w 8 values per lane of a row in their own type, x as three bf16 terms.
template <typename W>
__device__ inline f32x4 mma3(u32x4 w, const b8* x, f32x4 acc) {
  if constexpr (__is_same(W, bf16)) {
    const b8 v = __builtin_bit_cast(b8, w);
#pragma unroll
    for (int t = 2; t >= 0; --t) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, x[t], acc, 0, 0, 0);
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<f16>(w[i], &f[2 * i], &f[2 * i + 1]);
    b8 v[2];
    terms8<2>(f, v);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[1], x[1], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], x[2], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[1], x[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], x[1], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], x[0], acc, 0, 0, 0);
  }
  return acc;
}
template <typename W>
__device__ inline f32x4 mma1(u32x4 w, u32x4 x, f32x4 acc) {
  if constexpr (__is_same(W, bf16))
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, w), __builtin_bit_cast(b8, x), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, w), __builtin_bit_cast(h8, x), acc, 0, 0, 0);
}

struct Plan {
  int splits;   // workgroups over the columns
  int chunk;    // columns of each, a multiple of 32 kWaves
  Slots slots;
};
Plan plan(int64_t tokens, int adapters, int64_t cols) {
  Plan p;
  p.slots = list_slots(tokens, adapters, kTok);
  const int64_t tiles = std::min<int64_t>(tokens, tokens / kTok + std::min<int64_t>(adapters, tokens));
  constexpr int64_t unit = 32 * kWaves;
  const int64_t units = (cols + unit - 1) / unit;
  const int64_t want = std::min<int64_t>(std::min<int64_t>(units, 32), std::max<int64_t>(1, 512 / std::max<int64_t>(1, tiles)));
  const int64_t per = (units + want - 1) / want;
  p.chunk = (int)(per * unit);
  p.splits = (int)((units + per - 1) / per);
  return p;
}

// Places in the workspace.
struct Space {
  int64_t order, offsets, h, bytes;
};
Space space(int64_t tokens, int adapters, int rank, int64_t cols) {
  const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  Space w;
  w.order = 0;
  w.offsets = up(tokens * 4);
  w.h = w.offsets + up((adapters + 1) * int64_t(4));
  w.bytes = w.h + up((int64_t)plan(tokens, adapters, cols).splits * tokens * rank * 4);
  return w;
}

__device__ inline int rank_of(const tq_adapter_add_args& a, int i) { return a.ranks ? min(max(a.ranks[i], 0), a.rank) : a.rank; }

// h[split][place][rank] of a tile, RT tiles of 16 rank rows.
template <typename X, typename W, int RT>
__global__ __launch_bounds__(64 * kWaves) void shrink_kernel(tq_adapter_add_args a, const int32_t* order, const int32_t* offsets, float* h, int slots,
                                                            int slot0, bool places, int splits, int chunk) {
  __shared__ f32x4 sums[kWaves][RT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, qd = lane >> 4;
  const int slot = slot0 + blockIdx.x % slots, split = blockIdx.x / slots;
  const int tokens = (int)a.tokens, cols = (int)a.cols;
  const Tile tile = find_tile(offsets, a.adapters, tokens, kTok, places, slot, lane, nullptr);
  if (tile.count == 0 || tile.expert == a.adapters) return;  // uniform
  const int rank = rank_of(a, tile.expert);
  if (rank == 0) return;
  const int token = order[tile.first + min(l16, tile.count - 1)];  // places behind the tile repeat its last token and are not stored
  const X* x = static_cast<const X*>(a.x) + (int64_t)token * a.x_stride;
  const W* w = static_cast<const W*>(a.a) + (int64_t)tile.expert * a.rank * cols;
  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{0, 0, 0, 0};
  const int lo = split * chunk, hi = min(cols, lo + chunk);
  for (int c = lo + 32 * wave; c < hi; c += 32 * kWaves) {
    const int at = c + 8 * qd;
    const bool in = at < hi;  // 8 columns are inside or outside together
    u32x4 wv[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = 16 * r + l16;
      wv[r] = in && row < rank ? *reinterpret_cast<const u32x4*>(w + (int64_t)row * cols + at) : u32x4{0, 0, 0, 0};
    }
    if constexpr (sizeof(X) == 4) {
      float xv[8];
      f32x4 p = {0, 0, 0, 0}, q = {0, 0, 0, 0};
      if (in) p = *reinterpret_cast<const f32x4*>(x + at), q = *reinterpret_cast<const f32x4*>(x + at + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = p[i], xv[4 + i] = q[i];
      b8 xt[3];
      terms8<3>(xv, xt);
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (16 * r < rank) acc[r] = mma3<W>(wv[r], xt, acc[r]);
    } else {
      const u32x4 xv = in ? *reinterpret_cast<const u32x4*>(x + at) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (16 * r < rank) acc[r] = mma1<W>(wv[r], xv, acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) sums[wave][r][lane] = acc[r];
  __syncthreads();
  // lane (l16, qd) of tile r: token l16, rows 16 r + 4 qd .. + 3
  for (int r = wave; r < RT; r += kWaves) {
    f32x4 s = sums[0][r][lane];
    for (int v = 1; v < kWaves; ++v) s += sums[v][r][lane];
    const int row = 16 * r + 4 * qd;
    if (l16 < tile.count && row < a.rank) *reinterpret_cast<f32x4*>(h + ((int64_t)split * tokens + tile.first + l16) * a.rank + row) = s;
  }
}

// Where nothing is added, y as it is (-0 would become +0).
template <typename Y>
__device__ inline Y added(Y y, float add, bool any) {
  return any ? (Y)((float)y + add) : y;
}

// Features [64 wave + 256 block, + 64) of a tile of tokens.
template <typename W, typename Y>
__global__ __launch_bounds__(64 * kWaves) void expand_kernel(tq_adapter_add_args a, const int32_t* order, const int32_t* offsets, const float* h, int slots,
                                                            int slot0, bool places, int splits, bool wide) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, qd = lane >> 4;
  const int slot = slot0 + blockIdx.x % slots;
  const int64_t f0 = ((int64_t)(blockIdx.x / slots) * kWaves + wave) * kFeat, rows = a.rows;
  const int tokens = (int)a.tokens;
  const Tile tile = find_tile(offsets, a.adapters, tokens, kTok, places, slot, lane, nullptr);
  if (tile.count == 0) return;
  const bool some = tile.expert < a.adapters;
  const int token = order[tile.first + min(l16, tile.count - 1)];
  if (!some && a.bad_flag && a.index[token] >= a.adapters) raise_flag(a.bad_flag);
  const int rank = some ? rank_of(a, tile.expert) : 0;
  if (rank == 0 && a.out == a.y) return;
  const float scale = some && a.scale ? a.scale[tile.expert] : 1.0f;
  const W* b = static_cast<const W*>(a.b) + (int64_t)(some ? tile.expert : 0) * rows * a.rank;
  f32x4 acc[kFeat / 16];
#pragma unroll
  for (int f = 0; f < kFeat / 16; ++f) acc[f] = f32x4{0, 0, 0, 0};
  for (int r = 0; r < rank; r += 32) {
    const int at = r + 8 * qd;
    float hv[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (at < rank) {
      const float* p = h + ((int64_t)tile.first + min(l16, tile.count - 1)) * a.rank + at;
      for (int s = 0; s < splits; ++s, p += (int64_t)tokens * a.rank)
#pragma unroll
        for (int i = 0; i < 8; ++i) hv[i] += p[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[i] = at + i < rank ? hv[i] * scale : 0.0f;
    }
    b8 ht[3];
    terms8<3>(hv, ht);
#pragma unroll
    for (int f = 0; f < kFeat / 16; ++f) {
      const int64_t row = f0 + 16 * f + l16;
      u32x4 w = {0, 0, 0, 0};
      if (at < rank && row < rows) {
        w = *reinterpret_cast<const u32x4*>(b + row * a.rank + at);
        if (at + 8 > rank) {  // what lies behind the rank is not used
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] &= at + 2 * i + 1 < rank ? 0xFFFFFFFFu : at + 2 * i < rank ? 0xFFFFu : 0u;
        }
      }
      acc[f] = mma3<W>(w, ht, acc[f]);
    }
  }
  if (l16 >= tile.count) return;
  const Y* y = static_cast<const Y*>(a.y) + (int64_t)token * a.y_stride;
  Y* out = static_cast<Y*>(a.out) + (int64_t)token * a.out_stride;
#pragma unroll
  for (int f = 0; f < kFeat / 16; ++f) {
    const int64_t row = f0 + 16 * f + 4 * qd;
    if (row >= rows) continue;
    if (wide && row + 4 <= rows) {
      typedef Vec<Y, 4> V;
      const V v = *reinterpret_cast<const V*>(y + row);
      V o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o.v[i] = added(v.v[i], acc[f][i], rank > 0);
      *reinterpret_cast<V*>(out + row) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row + i < rows) out[row + i] = added(y[row + i], acc[f][i], rank > 0);
    }
  }
}

// At most 2^22 workgroups per launch: slots in chunks, each with `per` workgroups.
template <typename F>
hipError_t over_slots(int64_t slots, int64_t per, F launch) {
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 22) / per);
  for (int64_t s0 = 0; s0 < slots; s0 += most) {
    const int64_t now = std::min(most, slots - s0);
    launch((unsigned)(now * per), (int)now, (int)s0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename X, typename W>
hipError_t shrink(const tq_adapter_add_args& a, const Plan& p, const int32_t* order, const int32_t* offsets, float* h, hipStream_t s) {
  const dim3 block(64 * kWaves);
  return over_slots(p.slots.count, p.splits, [&](unsigned grid, int slots, int slot0) {
#define TQ_SHRINK(RT) \
  hipLaunchKernelGGL((shrink_kernel<X, W, RT>), dim3(grid), block, 0, s, a, order, offsets, h, slots, slot0, p.slots.places, p.splits, p.chunk)
    if (a.rank <= 16)
      TQ_SHRINK(1);
    else if (a.rank <= 32)
      TQ_SHRINK(2);
    else if (a.rank <= 64)
      TQ_SHRINK(4);
    else
      TQ_SHRINK(16);
#undef TQ_SHRINK
  });
}

template <typename W, typename Y>
hipError_t expand(const tq_adapter_add_args& a, const Plan& p, const int32_t* order, const int32_t* offsets, const float* h, hipStream_t s) {
  const int64_t blocks = (a.rows + kFeat * kWaves - 1) / (kFeat * kWaves);
  const bool wide = (uintptr_t)a.y % (4 * sizeof(Y)) == 0 && (uintptr_t)a.out % (4 * sizeof(Y)) == 0 && a.y_stride % 4 == 0 && a.out_stride % 4 == 0;
  return over_slots(p.slots.count, blocks, [&](unsigned grid, int slots, int slot0) {
    hipLaunchKernelGGL((expand_kernel<W, Y>), dim3(grid), dim3(64 * kWaves), 0, s, a, order, offsets, h, slots, slot0, p.slots.places, p.splits, wide);
  });
}

template <typename W>
hipError_t launch_w(const tq_adapter_add_args& a, const Plan& p, int32_t* order, int32_t* offsets, float* h, hipStream_t s) {
  const hipError_t e = a.x_type == TQ_F32 ? shrink<float, W>(a, p, order, offsets, h, s) : shrink<W, W>(a, p, order, offsets, h, s);
  if (e != hipSuccess) return e;
  return a.y_type == TQ_F32    ? expand<W, float>(a, p, order, offsets, h, s)
         : a.y_type == TQ_BF16 ? expand<W, bf16>(a, p, order, offsets, h, s)
                               : expand<W, f16>(a, p, order, offsets, h, s);
}

}  // namespace

int64_t adapter_workspace_bytes(int64_t tokens, int adapters, int rank, int64_t cols) { return space(tokens, adapters, rank, cols).bytes; }

hipError_t launch_adapter_add(const tq_adapter_add_args& a, hipStream_t s) {
  const Plan p = plan(a.tokens, a.adapters, a.cols);
  const Space w = space(a.tokens, a.adapters, a.rank, a.cols);
  char* ws = static_cast<char*>(a.workspace);
  int32_t* order = reinterpret_cast<int32_t*>(ws + w.order);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + w.offsets);
  float* h = reinterpret_cast<float*>(ws + w.h);
  const hipError_t e = launch_expert_lists(a.index, a.tokens, a.adapters, order, offsets, s);
  if (e != hipSuccess) return e;
  return a.w_type == TQ_BF16 ? launch_w<bf16>(a, p, order, offsets, h, s) : launch_w<f16>(a, p, order, offsets, h, s);
}

}  // namespace tq
