// k_adapter.hip -- low-rank adapters of many requests beside a shared
// projection: out[t] = y[t] + scale_i B_i (A_i x[t]).
//
// Kernels over tiles of tokens of one adapter:
//   shrink: h = A_i x for 16 tokens on 16x16x32 matrix instructions, the
//     columns split over workgroups (partial sums) and a workgroup's waves
//     (added through LDS);
//   join (many tokens): the partial sums of h added, scaled and split into the
//     bf16 terms that expand's matrix instructions take;
//   expand: y + scale B_i h, 64 features per wave: for 16 tokens, whose partial
//     sums a workgroup adds in LDS, or after join for up to 64, for which B_i
//     stays in registers.
// Up to 64 tokens every wave finds its tile from the index itself; more are
// sorted by adapter first (expert_lists).
//
// Memory bounds both: a token's x, y and out and an adapter's A and B are read
// or written once (A once per 16 of its tokens, or per 32 of many at ranks up to
// 64, and B once per 16, or per 64 of many, from the L2).
// 4099 tokens of 5 adapters of rank 64 (5120 columns in bf16, 7168 features in
// fp32) take 101 us: the lists 5, shrink 27, join 5, expand 69 for 297 MB, 4.3
// TB/s of a mix of reads and writes in 256-byte rows.  64 tokens of 24 adapters
// 21 us: shrink 7.6, expand 13, mostly the latency of index, weights, sums and
// y one after the other; one token 9.0.  Ranks above 64 take shrink's 16 tiles of
// rank rows and read B as it is needed: 4099 tokens beside the same matrix, us at
// ranks 64, 72, 128 and 256 used whole: 104, 166, 222, 376.
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

constexpr int kExpandTok = 64;
// Up to a wave's 64 tokens tiles are found without sorting: one token 14.3 us with a launch of the lists, 9.2 without.
constexpr int kDirect = 64;
// From 2048 tokens on partial sums are joined by a kernel and 64 tokens share B.  With / without, us (5120 columns, 7168 features;
// rank 16 and 64, 4 adapters): 1000 tokens 31 / 26 and 38 / 38, 2500 tokens 47 / 44 and 63 / 68, 4099 tokens 78 / 80 and 103 / 119.
constexpr int kJoin = 2048;
constexpr int kExpandWaves = 4;
constexpr int kFeat = 64;        // features per wave of expand
constexpr int kMaxSplits = 8;
constexpr int kMaxGroups = 768;  // workgroups that splits of the columns may make (three per compute unit)

// 8 values as TERMS (2 or 3) bf16 vectors.  The first term is held at bf16's largest, so that fp32 values above it, which would be
// rounded to infinity, leave the rest to the second; so do infinities and NaN, and nothing is left behind a term that is not finite.
template <int TERMS>
__device__ inline void terms8(const float* p, b8* out) {
  constexpr float kMost = 0x1.FEp127f;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = p[i];
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = t == 0 ? pack2<bf16>(__builtin_amdgcn_fmed3f(x[2 * i], -kMost, kMost), __builtin_amdgcn_fmed3f(x[2 * i + 1], -kMost, kMost))
                    : pack2<bf16>(x[2 * i], x[2 * i + 1]);
      if (t + 1 < TERMS) {
        float u, v;
        unpack2<bf16>(w[i], &u, &v);
        x[2 * i] = t == 0 || fabsf(u) < INFINITY ? x[2 * i] - u : 0.0f;
        x[2 * i + 1] = t == 0 || fabsf(v) < INFINITY ? x[2 * i + 1] - v : 0.0f;
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

// ---- which kernels ----

// Tokens of a tile of shrink: more read A less often, where there are many of them.
constexpr int shrink_tok(int rank, bool join) { return join && rank <= 64 ? 32 : 16; }
constexpr int shrink_tiles(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 16; }  // of 16 rank rows
constexpr int shrink_waves(int tiles) { return tiles <= 4 ? 8 : 4; }                                    // 64 KB of LDS at most

struct Plan {
  int splits;  // workgroups over the columns
  int chunk;   // columns of each, a multiple of 32 per wave
  bool direct; // tiles found from the index
  bool join;
  Slots shrink, expand;
};
Plan plan(int64_t tokens, int adapters, int rank, int64_t cols) {
  Plan p;
  p.direct = tokens <= kDirect;
  p.join = tokens >= kJoin;
  const int tok = shrink_tok(rank, p.join);
  p.shrink = list_slots(tokens, adapters, tok);
  p.expand = list_slots(tokens, adapters, p.join ? kExpandTok : 16);
  const int64_t tiles = std::min<int64_t>(tokens, tokens / tok + std::min<int64_t>(adapters, tokens));
  const int64_t unit = 32 * shrink_waves(shrink_tiles(rank));
  const int64_t units = (cols + unit - 1) / unit;
  const int64_t want = std::min<int64_t>(std::min<int64_t>(units, kMaxSplits), std::max<int64_t>(1, kMaxGroups / std::max<int64_t>(1, tiles)));
  const int64_t per = (units + want - 1) / want;
  p.chunk = (int)(per * unit);
  p.splits = (int)((units + per - 1) / per);
  return p;
}

// Rows of partial sums that a call of these sizes, or of fewer tokens, has at most.  There are fewer splits the more tiles, so that
// splits * tokens goes up and down; but it is tokens where there is one split, and otherwise below kMaxGroups / tiles * tokens with
// tokens < tiles * shrink_tok.  So a workspace serves every call of fewer tokens, adapters or columns, or of a lower rank.
int64_t partial_rows(int64_t tokens, int64_t cols) {
  constexpr int64_t kMostTok = std::max(shrink_tok(8, true), shrink_tok(256, false));
  constexpr int64_t kLeastUnit = 32 * std::min(shrink_waves(1), shrink_waves(16));
  const int64_t splits = std::min<int64_t>(kMaxSplits, (cols + kLeastUnit - 1) / kLeastUnit);
  return std::max(tokens, std::min(splits * tokens, kMaxGroups * kMostTok));
}

// Places in the workspace.
struct Space {
  int64_t order, offsets, h, terms, bytes;
};
Space space(int64_t tokens, int adapters, int rank, int64_t cols) {
  const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  const Plan p = plan(tokens, adapters, rank, cols);
  Space w;
  w.order = 0;
  w.offsets = p.direct ? 0 : up(tokens * 4);
  w.h = p.direct ? 0 : w.offsets + up((adapters + 1) * int64_t(4));
  w.terms = w.h + up(partial_rows(tokens, cols) * rank * 4);
  w.bytes = w.terms + (p.join ? up(tokens * rank * 6) : 0);
  return w;
}

struct Find {
  const int32_t *order, *offsets;
  int slots, slot0;  // of this launch
  bool places, direct;
};

__device__ inline int rank_of(const tq_adapter_add_args& a, int i) { return a.ranks ? min(max(a.ranks[i], 0), a.rank) : a.rank; }

// The tile of a slot, by each wave for itself: its adapter (a.adapters: none), how many tokens, and in lane k the k-th of them.
struct Group {
  int adapter, count, token;
};
template <int SIZE>
__device__ inline Group find_group(const tq_adapter_add_args& a, const Find& f, int slot, int lane) {
  Group g;
  const int tokens = (int)a.tokens;
  if (f.direct) {  // the tiles of the first token's adapter, then of the first token's of the others, and so on
    const int i = lane < tokens ? a.index[lane] : -1;
    const int mine = lane >= tokens ? -1 : i < 0 || i >= a.adapters ? a.adapters : i;
    uint64_t left = __ballot(lane < tokens), same = 0;
    int first = 0;
    g.count = 0;
    while (left) {
      g.adapter = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
      same = __ballot(mine == g.adapter);
      const int n = (int)__popcll(same), tiles = (n + SIZE - 1) / SIZE;
      if (slot < tiles) {
        first = SIZE * slot;
        g.count = min(SIZE, n - first);
        break;
      }
      slot -= tiles;
      left &= ~same;
    }
    const int place = __popcll(same & ((uint64_t(1) << lane) - 1));
    // each of them to the lane of its place behind the first; others to lanes that nobody reads
    const bool in = (same >> lane & 1) && place >= first;
    const int rest = 63 - (int)__popcll(__ballot(!in) & ((uint64_t(1) << lane) - 1));
    g.token = __builtin_amdgcn_ds_permute(4 * (in ? place - first : rest), lane);
  } else {
    const Tile t = find_tile(f.offsets, a.adapters, tokens, SIZE, f.places, slot, lane);
    g.adapter = t.expert, g.count = t.count;
    g.token = lane < t.count ? f.order[t.first + lane] : 0;
  }
  return g;
}
__device__ inline int token_of(const Group& g, int k) { return __shfl(g.token, min(k, g.count - 1), 64); }

// ---- A x ----

// h[split][token][rank] of a tile of 16 NT tokens, RT tiles of 16 rank rows.
template <typename X, typename W, int RT, int NT>
__global__ __launch_bounds__(64 * shrink_waves(RT)) void shrink_kernel(tq_adapter_add_args a, Find find, float* h, int chunk) {
  constexpr int kWaves = shrink_waves(RT);
  __shared__ f32x4 sums[kWaves][RT * NT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, qd = lane >> 4;
  const int split = blockIdx.x / find.slots;
  const Group g = find_group<16 * NT>(a, find, find.slot0 + blockIdx.x % find.slots, lane);
  if (g.count == 0 || g.adapter == a.adapters) return;  // uniform
  const int cols = (int)a.cols, rank = rank_of(a, g.adapter);
  if (rank == 0) return;
  int token[NT];
  const X* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    token[n] = token_of(g, 16 * n + l16);  // places behind the tile repeat its last token and are not stored
    x[n] = static_cast<const X*>(a.x) + (int64_t)token[n] * a.x_stride;
  }
  const W* w = static_cast<const W*>(a.a) + (int64_t)g.adapter * a.rank * cols;
  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0, 0, 0, 0};
  const int lo = split * chunk, hi = min(cols, lo + chunk);
  constexpr int kXV = sizeof(X) == 4 ? 2 : 1;  // 16-byte reads of 8 values
  constexpr int kSteps = RT <= 4 ? 2 : 1;      // reads of two steps are asked for before the first is used
  for (int c = lo + 32 * wave; c < hi; c += 32 * kWaves * kSteps) {
    u32x4 wv[kSteps][RT], xv[kSteps][NT][kXV];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int at = c + 32 * kWaves * s + 8 * qd;
      const bool in = at < hi;  // 8 columns are inside or outside together
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int v = 0; v < kXV; ++v) xv[s][n][v] = in ? *reinterpret_cast<const u32x4*>(x[n] + at + 4 * v) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int row = 16 * r + l16;
        wv[s][r] = in && row < rank ? *reinterpret_cast<const u32x4*>(w + (int64_t)row * cols + at) : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (sizeof(X) == 4) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(xv[s][n][i / 4][i % 4]);
          b8 xt[3];
          terms8<3>(f, xt);
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (16 * r < rank) acc[r][n] = mma3<W>(wv[s][r], xt, acc[r][n]);
        } else {
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (16 * r < rank) acc[r][n] = mma1<W>(wv[s][r], xv[s][n][0], acc[r][n]);
        }
      }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) sums[wave][r * NT + n][lane] = acc[r][n];
  __syncthreads();
  // lane (l16, qd) of tile (r, n): token 16 n + l16, rows 16 r + 4 qd .. + 3
  for (int t = wave; t < RT * NT; t += kWaves) {
    f32x4 s = sums[0][t][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) s += sums[v][t][lane];
    const int row = 16 * (t / NT) + 4 * qd, k = 16 * (t % NT) + l16;
    const int to = token_of(g, k);
    if (k < g.count && row < a.rank) *reinterpret_cast<f32x4*>(h + ((int64_t)split * a.tokens + to) * a.rank + row) = s;
  }
}

// terms[token][3][rank] of scale h, 8 columns per thread.
__global__ __launch_bounds__(256) void join_kernel(tq_adapter_add_args a, const float* h, bf16* terms, int splits) {
  const int per = a.rank / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, token = i / per;
  if (token >= a.tokens) return;
  const int adapter = a.index[token];
  if (adapter < 0 || adapter >= a.adapters) return;  // nobody reads them
  const float scale = a.scale ? a.scale[adapter] : 1.0f;
  const f32x4* p = reinterpret_cast<const f32x4*>(h + i * 8);
  const int64_t next = a.tokens * a.rank / 4;
  f32x4 s0 = {0, 0, 0, 0}, s1 = s0;
  for (int s = 0; s < splits; ++s) s0 += p[s * next], s1 += p[s * next + 1];
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = s0[j] * scale, f[4 + j] = s1[j] * scale;
  b8 t[3];
  terms8<3>(f, t);
  bf16* to = terms + token * 3 * a.rank + i % per * 8;
#pragma unroll
  for (int v = 0; v < 3; ++v) *reinterpret_cast<b8*>(to + v * a.rank) = t[v];
}

// ---- y + B h ----

// Four neighbouring values of a row, whatever its alignment.
template <typename Y>
struct __attribute__((packed, aligned(sizeof(Y)))) Four {
  Y v[4];
};

// Where nothing is added, y as it is (-0 would become +0).
template <typename Y>
__device__ inline Y added(Y y, float add, bool any) {
  return any ? (Y)((float)y + add) : y;
}

// KS: steps of 32 rank columns whose weights stay in registers (0: read when they are needed).  JOINED: h is join's terms, for
// tiles of kExpandTok tokens; otherwise shrink's partial sums, for tiles of 16, and `lds` holds their sum.
template <typename W, typename Y, int KS, bool JOINED>
__global__ __launch_bounds__(64 * kExpandWaves) void expand_kernel(tq_adapter_add_args a, Find find, const void* h, int splits) {
  // [16][rank + 4] of h, or the tile's terms [kTok][3 rank + 8], whole rows of 16 bytes (the 8 keep rows off the same banks)
  extern __shared__ float lds[];
  constexpr bool kStaged = JOINED && KS > 0;
  constexpr int kF = kFeat / 16, kTok = JOINED ? kExpandTok : 16;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, qd = lane >> 4;
  const Group g = find_group<kTok>(a, find, find.slot0 + blockIdx.x % find.slots, lane);
  if (g.count == 0) return;
  const int64_t f0 = ((int64_t)(blockIdx.x / find.slots) * kExpandWaves + wave) * kFeat, rows = a.rows;
  const bool some = g.adapter < a.adapters;
  if (!some && a.bad_flag && lane < g.count && a.index[g.token] >= a.adapters) raise_flag(a.bad_flag);
  const int rank = some ? rank_of(a, g.adapter) : 0;
  if (rank == 0 && a.out == a.y) return;
  const W* b = static_cast<const W*>(a.b) + (int64_t)(some ? g.adapter : 0) * rows * a.rank;
  const auto load_b = [&](int f, int r) __attribute__((always_inline)) {  // 8 values of feature f0 + 16 f + l16 from column r + 8 qd on
    const int64_t row = f0 + 16 * f + l16;
    const int at = r + 8 * qd;
    u32x4 w = {0, 0, 0, 0};
    if (at < rank && row < rows) {
      w = *reinterpret_cast<const u32x4*>(b + row * a.rank + at);
      if (at + 8 > rank) {  // what lies behind the rank is not used
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] &= at + 2 * i + 1 < rank ? 0xFFFFFFFFu : at + 2 * i < rank ? 0xFFFFu : 0u;
      }
    }
    return w;
  };
  const auto load_h = [&](int token, int r, b8* t) __attribute__((always_inline)) {
    const int at = r + 8 * qd;
    if constexpr (JOINED) {
      const bf16* p = kStaged ? reinterpret_cast<const bf16*>(lds) + token * (3 * a.rank + 8) + at
                              : static_cast<const bf16*>(h) + (int64_t)token * 3 * a.rank + at;
#pragma unroll
      for (int v = 0; v < 3; ++v) t[v] = at < rank ? *reinterpret_cast<const b8*>(p + v * a.rank) : b8{0, 0, 0, 0, 0, 0, 0, 0};
    } else {
      float f[8];
      const float* p = lds + l16 * (a.rank + 4) + at;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = at < rank ? p[i] : 0.0f;
      terms8<3>(f, t);
    }
  };
  typedef Four<Y> V;
  const auto load_y = [&](int token, V* v) __attribute__((always_inline)) {
    const Y* y = static_cast<const Y*>(a.y) + (int64_t)token * a.y_stride;
#pragma unroll
    for (int f = 0; f < kF; ++f) {
      const int64_t row = f0 + 16 * f + 4 * qd;
      if (row + 4 <= rows) {
        v[f] = *reinterpret_cast<const V*>(y + row);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[f].v[i] = row + i < rows ? y[row + i] : (Y)0.0f;
      }
    }
  };

  constexpr int kKeep = KS > 0 ? KS : 1;
  u32x4 wb[kF][kKeep];
  V y[kF], y_next[kF];
  int token = token_of(g, l16);
  if constexpr (kStaged) {
    const int per = 3 * a.rank / 8, all = rank ? g.count * per : 0;
    for (int i0 = 64 * wave; i0 < all; i0 += 64 * kExpandWaves) {  // (uniform, so that every lane is there to be asked for its token)
      const int i = min(i0 + lane, all - 1), k = i / per, at = i % per;
      const b8 v = static_cast<const b8*>(h)[(int64_t)__shfl(g.token, k, 64) * per + at];
      *reinterpret_cast<b8*>(reinterpret_cast<bf16*>(lds) + k * (3 * a.rank + 8) + 8 * at) = v;
    }
  } else if constexpr (!JOINED) {
    // partial sums of kAhead splits are asked for at once
    constexpr int kAhead = 4;
    const float scale = some && a.scale ? a.scale[g.adapter] : 1.0f;
    const int per = a.rank / 4, all = rank ? g.count * per : 0;
    const int64_t next = a.tokens * a.rank / 4;
    for (int i0 = 64 * wave; i0 < all; i0 += 64 * kExpandWaves) {  // (uniform, so that every lane is there to be asked for its token)
      const int i = min(i0 + lane, all - 1), k = i / per, at = i % per;
      const f32x4* p = static_cast<const f32x4*>(h) + (int64_t)__shfl(g.token, k, 64) * per + at;
      f32x4 sum = {0, 0, 0, 0};
      for (int s0 = 0; s0 < splits; s0 += kAhead) {
        f32x4 v[kAhead];
#pragma unroll
        for (int s = 0; s < kAhead; ++s) v[s] = s0 + s < splits ? p[(s0 + s) * next] : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < kAhead; ++s) sum += v[s];
      }
      *reinterpret_cast<f32x4*>(lds + k * (a.rank + 4) + 4 * at) = sum * scale;
    }
  }
  load_y(token, y);
  if constexpr (KS > 0) {
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
      for (int k = 0; k < KS; ++k) wb[f][k] = load_b(f, 32 * k);
  }
  if constexpr (kStaged || !JOINED) __syncthreads();
  for (int t0 = 0; t0 < g.count; t0 += 16) {
    f32x4 acc[kF];
#pragma unroll
    for (int f = 0; f < kF; ++f) acc[f] = f32x4{0, 0, 0, 0};
    b8 ht[kKeep][3];
    if constexpr (KS > 0) {
#pragma unroll
      for (int k = 0; k < KS; ++k) load_h(kStaged ? min(t0 + l16, g.count - 1) : token, 32 * k, ht[k]);
    }
    const int next = token_of(g, t0 + 16 + l16);
    if (JOINED && t0 + 16 < g.count) load_y(next, y_next);  // uniform
    if constexpr (KS > 0) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
        if (32 * k < rank) {  // uniform
#pragma unroll
          for (int f = 0; f < kF; ++f) acc[f] = mma3<W>(wb[f][k], ht[k], acc[f]);
        }
    } else {
      for (int r = 0; r < rank; r += 32) {
        load_h(token, r, ht[0]);
#pragma unroll
        for (int f = 0; f < kF; ++f) acc[f] = mma3<W>(load_b(f, r), ht[0], acc[f]);
      }
    }
    if (t0 + l16 < g.count) {
      Y* out = static_cast<Y*>(a.out) + (int64_t)token * a.out_stride;
#pragma unroll
      for (int f = 0; f < kF; ++f) {
        const int64_t row = f0 + 16 * f + 4 * qd;
        V o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o.v[i] = added(y[f].v[i], acc[f][i], rank > 0);
        if (row + 4 <= rows) {
          *reinterpret_cast<V*>(out + row) = o;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row + i < rows) out[row + i] = o.v[i];
        }
      }
    }
    if constexpr (!JOINED) break;
    token = next;
#pragma unroll
    for (int f = 0; f < kF; ++f) y[f] = y_next[f];
  }
}

// At most 2^22 workgroups per launch: slots in chunks, each with `per` workgroups.
template <typename F>
hipError_t over_slots(const Slots& slots, int64_t per, Find f, F launch) {
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 22) / per);
  f.places = slots.places;
  for (int64_t s0 = 0; s0 < slots.count; s0 += most) {
    const int64_t now = std::min(most, slots.count - s0);
    f.slots = (int)now, f.slot0 = (int)s0;
    launch((unsigned)(now * per), f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename X, typename W, int RT, int NT>
hipError_t shrink_t(const tq_adapter_add_args& a, const Plan& p, const Find& f, float* h, hipStream_t s) {
  return over_slots(p.shrink, p.splits, f, [&](unsigned grid, const Find& g) {
    hipLaunchKernelGGL((shrink_kernel<X, W, RT, NT>), dim3(grid), dim3(64 * shrink_waves(RT)), 0, s, a, g, h, p.chunk);
  });
}
template <typename X, typename W>
hipError_t shrink(const tq_adapter_add_args& a, const Plan& p, const Find& f, float* h, hipStream_t s) {
  const bool two = shrink_tok(a.rank, p.join) == 32;
  switch (shrink_tiles(a.rank)) {
    case 1: return two ? shrink_t<X, W, 1, 2>(a, p, f, h, s) : shrink_t<X, W, 1, 1>(a, p, f, h, s);
    case 2: return two ? shrink_t<X, W, 2, 2>(a, p, f, h, s) : shrink_t<X, W, 2, 1>(a, p, f, h, s);
    case 4: return two ? shrink_t<X, W, 4, 2>(a, p, f, h, s) : shrink_t<X, W, 4, 1>(a, p, f, h, s);
    default: return shrink_t<X, W, 16, 1>(a, p, f, h, s);
  }
}

template <typename W, typename Y, int KS>
hipError_t expand_t(const tq_adapter_add_args& a, const Plan& p, const Find& f, const void* h, hipStream_t s) {
  constexpr int kAll = kFeat * kExpandWaves;
  return over_slots(p.expand, (a.rows + kAll - 1) / kAll, f, [&](unsigned grid, const Find& g) {
    const dim3 block(64 * kExpandWaves);
    if (p.join)
      hipLaunchKernelGGL((expand_kernel<W, Y, KS, true>), dim3(grid), block, KS ? kExpandTok * (3 * a.rank + 8) * sizeof(bf16) : 0, s, a, g, h, p.splits);
    else
      hipLaunchKernelGGL((expand_kernel<W, Y, KS, false>), dim3(grid), block, 16 * (a.rank + 4) * sizeof(float), s, a, g, h, p.splits);
  });
}
template <typename W, typename Y>
hipError_t expand(const tq_adapter_add_args& a, const Plan& p, const Find& f, const void* h, hipStream_t s) {
  return a.rank <= 32 ? expand_t<W, Y, 1>(a, p, f, h, s) : a.rank <= 64 ? expand_t<W, Y, 2>(a, p, f, h, s) : expand_t<W, Y, 0>(a, p, f, h, s);
}

template <typename W>
hipError_t launch_w(const tq_adapter_add_args& a, const Plan& p, const Find& f, float* h, bf16* terms, hipStream_t s) {
  hipError_t e = a.x_type == TQ_F32 ? shrink<float, W>(a, p, f, h, s) : shrink<W, W>(a, p, f, h, s);
  if (e != hipSuccess) return e;
  if (p.join) {
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)((a.tokens * (a.rank / 8) + 255) / 256)), dim3(256), 0, s, a, h, terms, p.splits);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const void* to = p.join ? static_cast<const void*>(terms) : h;
  return a.y_type == TQ_F32 ? expand<W, float>(a, p, f, to, s) : a.y_type == TQ_BF16 ? expand<W, bf16>(a, p, f, to, s) : expand<W, f16>(a, p, f, to, s);
}

}  // namespace

int64_t adapter_workspace_bytes(int64_t tokens, int adapters, int rank, int64_t cols) { return space(tokens, adapters, rank, cols).bytes; }

hipError_t launch_adapter_add(const tq_adapter_add_args& a, hipStream_t s) {
  const Plan p = plan(a.tokens, a.adapters, a.rank, a.cols);
  const Space w = space(a.tokens, a.adapters, a.rank, a.cols);
  char* ws = static_cast<char*>(a.workspace);
  int32_t* order = reinterpret_cast<int32_t*>(ws + w.order);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + w.offsets);
  if (!p.direct) {
    const hipError_t e = launch_expert_lists(a.index, a.tokens, a.adapters, order, offsets, s);
    if (e != hipSuccess) return e;
  }
  const Find f{order, offsets, 0, 0, true, p.direct};
  float* h = reinterpret_cast<float*>(ws + w.h);
  bf16* terms = reinterpret_cast<bf16*>(ws + w.terms);
  return a.w_type == TQ_BF16 ? launch_w<bf16>(a, p, f, h, terms, s) : launch_w<f16>(a, p, f, h, terms, s);
}

}  // namespace tq
