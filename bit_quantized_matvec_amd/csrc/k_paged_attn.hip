// k_paged_attn.hip -- attention of new tokens over a paged cache.
//
// Mathematics.  For one key head the query rows are (token, head of the group)
// pairs; their scores S = scale Q K^T and outputs O = softmax(S) V are taken in
// one pass over the keys with a running maximum m and sum l per row (base 2:
// p = 2^(s - m), s scaled by scale log2 e), so S never leaves registers.
//
// Operands.  Both products are computed transposed, S^T = K Q^T and
// O^T = V^T P^T: a column of a matrix-instruction tile is a query row, so a
// row's m, l and rescaling belong to a lane.  The key a lane finds in its
// S^T registers depends on which K row was fed as which A row, and that
// is free to choose: rows are fed in the order that leaves lane group g with
// the consecutive keys 8g .. 8g + 7, which is the layout the B operand of the
// second product wants.  So P goes from the first product to the second
// without a lane exchange, and V^T (stored transposed) is read 16 bytes = 8
// consecutive keys at a time.
//
// Rounding.  Q, K, V enter as they are; products are exact and summed in
// fp32.  P enters the second product as 2 (fp16) or 3 (bf16) terms whose sum
// holds 22 or 24 bits when the output is fp32.  When the output has the cache's
// type, attn_rows, which waits for memory anyway, takes 2 terms (16 or 22 bits),
// and attn_chunk, bound by the matrix units, one: half a step of that type per
// probability, independent over the keys, beside the output's own half step.
// fp16 P is scaled by 2^11 (removed by the division by l, which carries it
// too), so that small probabilities stay normal.  attn_chunk moves a row's
// maximum, and so rescales O, only when a score passes it by more than kSlack
// (base 2): P is at most 2^kSlack, 2^15 with the scaling in fp16.
//
// Unseen keys.  Their scores become -inf; their V values are made zero where
// no row of the workgroup sees them, as 0 * NaN would spoil a sum.  A value
// that is not finite and that some rows see spoils the others too, and an
// infinity times a term of P that is zero or negative becomes NaN: a result
// with a NaN is therefore computed a second time with pv_each(), which takes
// finite values as before and counts infinities and NaN per (row, column) with
// the 0/1 visibility in the place of P.  Finite caches never come there.
//
// Two kernels:
//
//   attn_rows    16 query rows per workgroup, 4 waves that each take every
//                fourth block of 32 keys straight from memory to registers; no
//                LDS before the waves are joined.  For few rows (single
//                tokens): bound by the cache's bytes.  One stream over 131075
//                keys, 2 x 256: 71 us, of which 38 stream the 268 MB (7 TB/s,
//                partly from the last-level cache), 7 pass before the first
//                keys arrive and 12 in two joins; 32 streams of 2 to 8 thousand
//                keys, 4 x 128: 91 us, 4.2 TB/s.
//   attn_chunk   128 query rows per workgroup, 32 per wave; K and V tiles go
//                straight from memory into LDS, double-buffered, shared by the
//                waves.  Bound by the matrix units and the exponentials beside
//                them: 2048 tokens over 8100 keys, 48 x 128: 393 to 409 us, 870
//                to 905 TFLOP/s (a large library product reaches 1170); with the
//                probabilities as two terms and 256 columns, 6 prompts in a
//                window of 1024: 153 us.
//
// Few workgroups: the keys of a tile are split over several, whose partial
// (m, l, O) go to the workspace.  The last to arrive of each 16 joins them, the
// last of those joins the joined ones (a tree of two levels, up to 256 parts):
// a join reads 16 x 12 KB through one compute unit, 5 us.  Splitting only the
// tiles of attn_chunk's last round, so that it fills the card, changed nothing
// at 128 columns and cost a quarter at 256.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kernels.h"
#include "seq.h"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kRowsTile = 16;    // query rows of an attn_rows workgroup
constexpr int kChunkTile = 128;  // query rows of an attn_chunk workgroup
constexpr int kBlock = 32;       // keys per step of an attn_rows wave
constexpr int kFan = 16;         // parts joined at once
constexpr int kMaxSplits = kFan * kFan;
constexpr int kMaxParts = 2048;  // parts of all tiles together
constexpr int kMaxChunkParts = 512;
constexpr int kLong = 32;
constexpr int kLeastTiles = 8;  // of an attn_chunk part: joining parts of many rows costs what some tiles do
constexpr int kCounters = kFan + 1;
constexpr int64_t kHeader = (int64_t)kMaxParts * kCounters * 4;  // the counters, before the parts
static_assert(kHeader % 256 == 0, "");
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// A wave holds 32 rows of Q and of O: at 256 columns those leave no room for a second wave on its SIMD, so two waves share
// the rows, compute the scores both and take half of O's columns each (6 windowed prompts: 172 -> 154 us).
constexpr int chunk_threads(int dim) { return dim == 256 ? 512 : 256; }

struct AttnParams {
  tq_paged_attn_args a;
  float scale2;  // scale * log2 e
  // Part 0 of every tile, then part 1, ...: the workgroups that find nothing to do come last.  (With a tile's parts together
  // and a quarter of them live, the live ones all went to the same compute units: 8 streams x 4000 keys x 2 tokens, 256
  // columns: 110 us.)
  int tiles, splits;
  // A tile's parts on different XCDs (workgroups go round the 8 of them): tiles differ in length.
  __device__ int tile_of(int place, int part) const { return (int)((unsigned)(place + 3 * part) % (unsigned)tiles); }
  int group, page_shift;
  int slot_per, slot_add;  // a sequence's first tile among all: cu slot_per / rows + slot_add b
  int places_shift;  // log2 of the workgroups that the card holds at once
  int tiles_each;    // tiles per sequence of one token
  unsigned group_mul, group_shift;
  // row / group for 0 <= row < 2^31
  __device__ int token_of(int row) const { return (int)(__umulhi((unsigned)row << 1, group_mul) >> group_shift); }
};

template <typename C>
struct Half;
template <>
struct Half<bf16> {
  typedef bf16 frag __attribute__((ext_vector_type(8)));
  static constexpr unsigned kExp = 0x7F807F80u;  // exponent bits of both halves of a dword
  static constexpr unsigned short kOne = 0x3F80;
  static constexpr float kShift = 0.f, kSlack = 8.f;
  static constexpr int kTerms = 3;
  static __device__ f32x4 mma(frag a, frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  static __device__ f32x16 mma(frag a, frag b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <>
struct Half<f16> {
  typedef f16 frag __attribute__((ext_vector_type(8)));
  static constexpr unsigned kExp = 0x7C007C00u;
  static constexpr unsigned short kOne = 0x3C00;
  static constexpr float kShift = 11.f, kSlack = 4.f;
  static constexpr int kTerms = 2;
  static __device__ f32x4 mma(frag a, frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  static __device__ f32x16 mma(frag a, frag b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};
template <typename C>
using Frag = typename Half<C>::frag;

// Zeroes the keys of an 8-key chunk (first key k) outside [begin, end).
__device__ inline u32x4 keep_keys(u32x4 x, int k, int begin, int end) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = k + 2 * i >= begin && k + 2 * i < end, hi = k + 2 * i + 1 >= begin && k + 2 * i + 1 < end;
    x[i] &= (lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
  }
  return x;
}

// What a workgroup computes: query rows row0 .. of sequence b for one key head, and which keys any of them sees.
struct Tile {
  int64_t t0;       // first token of the sequence
  int64_t b;
  int row0, rows;   // first row and count in this tile (rows <= 0: none)
  int kvh;
  int first_pos;    // position of the sequence's first new token (may be negative)
  int last_pos;     // position of the last row's token
  int begin, end;   // keys that the table has and some row sees: [begin, end), or 0, 0
};

// First key in the window of a token at this position.  (One before the first key sees nothing, and is taken as at it: no sum
// leaves 31 bits, whatever the window.)
__device__ inline int first_seen(int window, int pos) { return window > 0 ? max(0, max(pos, 0) - window + 1) : 0; }

template <int ROWS>
__device__ inline Tile find_tile(const AttnParams& p, int tile, int lane) {
  const auto& a = p.a;
  Tile r;
  const int slot = tile / (unsigned)a.kv_heads;
  r.kvh = tile - slot * a.kv_heads;
  r.b = a.cu ? find_seq(a.cu, a.seqs, p.slot_per, ROWS, p.slot_add, slot, lane) : p.tiles_each == 1 ? slot : slot / p.tiles_each;
  const SeqRange s = seq_range(a.cu, r.b, a.tokens, a.bad_flag);
  const int64_t slot0 = a.cu ? first_slot(a.cu, r.b, p.slot_per, ROWS, p.slot_add) : r.b * p.tiles_each;
  const int64_t row0 = (slot - slot0) * ROWS, all = (int64_t)s.n * p.group;
  r.t0 = s.t0;
  r.row0 = (int)row0;
  r.rows = row0 < 0 || row0 >= all ? 0 : (int)min((int64_t)ROWS, all - row0);
  const int64_t len = a.kv_len[r.b], keys = a.table_width << p.page_shift;
  if (len < 0 || len > keys) raise_flag(a.bad_flag);
  r.first_pos = (int)(max(len, (int64_t)0) - s.n);
  r.last_pos = r.first_pos + p.token_of(max(0, r.row0 + r.rows - 1));
  r.begin = first_seen(a.window, r.first_pos + p.token_of(r.row0));
  r.end = r.rows > 0 ? (int)min((int64_t)r.last_pos + 1, keys) : 0;
  if (r.begin >= r.end) r.begin = r.end = 0;
  return r;
}

// acc += V P, where V values that are not finite reach the rows that see their keys and no other.
template <typename C, int TERMS, typename ACC>
__device__ __forceinline__ ACC pv_each(u32x4 v, const Frag<C>* p, Frag<C> seen, ACC acc) {
  typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
  constexpr unsigned short e = Half<C>::kExp & 0xFFFF;
  const u16x8 x = __builtin_bit_cast(u16x8, v);
  u16x8 kind[4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool inf = (x[j] & 0x7FFF) == e, odd = (x[j] & e) == e;
    kind[0][j] = odd ? 0 : x[j];
    kind[1][j] = inf && !(x[j] & 0x8000) ? Half<C>::kOne : 0;
    kind[2][j] = inf && (x[j] & 0x8000) ? Half<C>::kOne : 0;
    kind[3][j] = odd && !inf ? Half<C>::kOne : 0;
  }
#pragma unroll
  for (int t = 0; t < TERMS; ++t) acc = Half<C>::mma(__builtin_bit_cast(Frag<C>, kind[0]), p[t], acc);
  const float what[3] = {INFINITY, -INFINITY, NAN};
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    ACC n;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(ACC) / 4); ++i) n[i] = 0.f;
    n = Half<C>::mma(__builtin_bit_cast(Frag<C>, kind[c + 1]), seen, n);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(ACC) / 4); ++i)
      if (n[i] > 0.f) acc[i] += what[c];
  }
  return acc;
}

__device__ inline void in_order() { asm volatile("" ::: "memory"); }  // loads before it are issued before it
__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- joining parts -------------------------------------------------------------------------------------------------

// A part: m [ROWS], l [ROWS], O [ROWS][D].  Stores and loads go through to the level that all XCDs share (sc1).
template <int ROWS, int D>
constexpr int part_floats() {
  return ROWS * (D + 2);
}
struct Parts {
  __amdgpu_buffer_rsrc_t r;
  static constexpr int kThrough = 16;
  __device__ Parts(const AttnParams& p)
      : r(__builtin_amdgcn_make_buffer_rsrc(static_cast<uint8_t*>(p.a.workspace) + kHeader, 0, (int)min(p.a.workspace_bytes - kHeader, (int64_t)INT32_MAX), 0x00027000)) {}
  __device__ void put(int at, float v) const { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at * 4, 0, kThrough); }
  __device__ void put4(int at, const float* v) const {
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, r, at * 4, 0, kThrough);
  }
  __device__ float get(int at) const { return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at * 4, 0, kThrough)); }
  __device__ f32x4 get4(int at) const { return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at * 4, 0, kThrough)); }
};

// Called by the whole workgroup after its stores to the workspace: whether it is the last of `count` to arrive.  The
// counter goes back to zero.
__device__ inline bool last_of(unsigned* counter, int count, int* shared) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // this wave's stores are done
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned n = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *shared = n == (unsigned)(count - 1);
    if (*shared) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  const bool last = *shared;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
  return last;
}

template <typename O>
__device__ inline void store4(O* dst, const float* v) {
  struct alignas(4 * sizeof(O)) V4 {
    O v[4];
  } o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o.v[j] = (O)v[j];
  *reinterpret_cast<V4*>(dst) = o;
}

// Final values of 4 columns of a row.
template <typename C, typename O, int D>
__device__ inline void finish(const AttnParams& p, const Tile& t, int row, int col, float m, float l, const float* o) {
  const int r = t.row0 + row, i = p.token_of(r), h = t.kvh * p.group + r - i * p.group;
  const int64_t at = (t.t0 + i) * p.a.heads + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float v[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
  store4(static_cast<O*>(p.a.out) + at * D + col, v);
  if (p.a.lse && col == 0) p.a.lse[at] = l == 0.f ? -INFINITY : (m - Half<C>::kShift + log2f(l)) * kLn2;
}

// Joins `count` parts from place `src` on, to the part at `dst` or, if that is negative, into the output.  `lds` has room for
// 2 (kFan + 1) ROWS values.
template <typename C, typename O, int ROWS, int D, int THREADS>
__device__ void join(const AttnParams& p, const Tile& t, const Parts& parts, int src, int count, int dst, float* lds) {
  constexpr int step = part_floats<ROWS, D>();
  constexpr int ITEMS = ROWS == kRowsTile ? std::max(1, ROWS * (D / 4) / THREADS) : 1;  // groups of 4 columns that a thread asks for at once
  const int all = t.rows * (D / 4);
  f32x4 os[ITEMS][kFan];
  auto ask = [&](int first) {  // everything before the first use: the memory is 1 to 2 us away
#pragma unroll
    for (int e = 0; e < kFan; ++e)
      if (e < count)
#pragma unroll
        for (int x = 0; x < ITEMS; ++x) os[x][e] = parts.get4(src + e * step + 2 * ROWS + min(first + x * THREADS, all - 1) * 4);
  };
  int first = threadIdx.x;
  ask(first);
  for (int i = threadIdx.x; i < 2 * ROWS * count; i += THREADS) lds[i] = parts.get(src + i / (2 * ROWS) * step + i % (2 * ROWS));
  __syncthreads();
  // each row's maximum and sum, and in the place of the parts' maxima their weights
  float m = -INFINITY, l = 0.f;
  if (threadIdx.x < ROWS) {
    float* row = lds + threadIdx.x;
    for (int e = 0; e < count; ++e) m = fmaxf(m, row[e * 2 * ROWS]);
    for (int e = 0; e < count; ++e) {
      const float w = row[e * 2 * ROWS] == -INFINITY ? 0.f : exp2_(row[e * 2 * ROWS] - m);
      l = fmaf(w, row[e * 2 * ROWS + ROWS], l);
      row[e * 2 * ROWS] = w;
    }
    lds[2 * ROWS * kFan + threadIdx.x] = m, lds[2 * ROWS * kFan + ROWS + threadIdx.x] = l;
  }
  __syncthreads();
#pragma unroll 1
  while (first < all) {
#pragma unroll
    for (int x = 0; x < ITEMS; ++x) {
      const int i = first + x * THREADS, row = min(i, all - 1) / (D / 4), col = i % (D / 4) * 4;
      float o[4] = {};
#pragma unroll
      for (int e = 0; e < kFan; ++e) {
        if (e >= count) continue;
        const float w = lds[e * 2 * ROWS + row];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fmaf(w, os[x][e][j], o[j]);
      }
      if (i >= all) continue;
      const float mr = lds[2 * ROWS * kFan + row], lr = lds[2 * ROWS * kFan + ROWS + row];
      if (dst < 0) {
        finish<C, O, D>(p, t, row, col, mr, lr, o);
      } else {
        parts.put4(dst + 2 * ROWS + row * D + col, o);
        if (col == 0) parts.put(dst + row, mr), parts.put(dst + ROWS + row, lr);
      }
    }
    first += ITEMS * THREADS;
    if (first < all) ask(first);
  }
}

// Two-level join over the `active` parts of a tile; called by every one of them after it has stored its part.
template <typename C, typename O, int ROWS, int D, int THREADS>
__device__ void join_tree(const AttnParams& p, const Tile& t, const Parts& parts, int tile, int part, int active, int* shared, float* lds) {
  unsigned* counters = static_cast<unsigned*>(p.a.workspace) + (int64_t)tile * kCounters;
  constexpr int step = part_floats<ROWS, D>();
  const int mine = tile * p.splits * step;
  const int joined = (p.tiles * p.splits + tile * ((p.splits + kFan - 1) / kFan)) * step;
  const int set = part / kFan, sets = (active + kFan - 1) / kFan, in_set = min(kFan, active - set * kFan);
  int counter = set, src = mine + set * kFan * step, count = in_set, dst = sets == 1 ? -1 : joined + set * step;
  while (last_of(counters + counter, count, shared)) {
    join<C, O, ROWS, D, THREADS>(p, t, parts, src, count, dst, lds);
    if (dst < 0) return;
    counter = kFan, src = joined, count = sets, dst = -1;
  }
}

// ---- few rows ------------------------------------------------------------------------------------------------------

template <typename C, typename O, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attn_rows_kernel(AttnParams p) {
  constexpr int KK = D / 32, DT = D / 16;
  constexpr int TERMS = sizeof(O) == 4 ? Half<C>::kTerms : 2;
  typedef Half<C> H;
  __shared__ __attribute__((aligned(16))) float stage[kWaves][kRowsTile][D + 4];
  __shared__ float stat[kWaves][2][kRowsTile];
  __shared__ int shared;
  const auto& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.x / (unsigned)p.tiles, tile = p.tile_of(blockIdx.x - part * p.tiles, part);
  const Tile t = find_tile<kRowsTile>(p, tile, lane);
  if (t.rows <= 0) return;
  // Blocks of 32 keys, every fourth of a part for each wave.  A wave that has none (less than 97 keys, or parts of 3 blocks)
  // leaves m = -inf, l = 0, and the joins pass over it.
  const int first = t.begin / kBlock, blocks = t.end > 0 ? (t.end + kBlock - 1) / kBlock - first : 0;
  // Parts of equal length that fill the places once; of kLong blocks at most where sequences may differ in length, so that
  // the longest does not hold up the end (32 streams of 2 to 8 thousand keys, 128 columns: 144 us in one round, 91 in parts
  // of 32 blocks, 95 of 16).
  const int even = (int)(((int64_t)blocks * p.tiles + (1 << p.places_shift) - 1) >> p.places_shift);
  const unsigned unit = max(kWaves, a.seqs == 1 ? even : min(even, kLong));
  const unsigned active = max(1u, min((unsigned)p.splits, (blocks + unit - 1) / unit));
  if ((unsigned)part >= active) return;
  const int each = blocks / active, more = blocks - each * active;  // the first `more` parts have one more
  const int lo = first + each * part + min(part, more), hi = lo + each + (part < more ? 1 : 0);

  const int r = lane & 15, g = lane >> 4;
  const bool row_ok = r < t.rows;
  const int row = t.row0 + (row_ok ? r : 0);
  const int token = p.token_of(row);
  const int least = first_seen(a.window, t.first_pos + token), pos = min(t.first_pos + token, t.end - 1);  // this row sees [least, pos]
  const int pos_lo = min(t.first_pos + p.token_of(t.row0), t.end - 1), pos_hi = t.last_pos;  // every row sees (pos_hi - window, pos_lo]

  Frag<C> q[KK];
  {
    const C* src = static_cast<const C*>(a.q) + (t.t0 + token) * a.q_token + (int64_t)(t.kvh * p.group + row - token * p.group) * a.q_head + 8 * g;
    const Frag<C> zero = {};
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) q[kk] = row_ok ? *reinterpret_cast<const Frag<C>*>(src + 32 * kk) : zero;
  }

  const C* kc = static_cast<const C*>(a.k_cache);
  const C* vc = static_cast<const C*>(a.v_cache);
  u32x4 k[2][KK], v[DT];
  // Pages of the two halves of a block's keys, -1 where the table's entry is no page.  Entries outside those of keys that
  // somebody sees are not read.
  int pages[2], ahead[2];
  const int32_t* table = a.block_table + t.b * a.table_stride;
  auto look = [&](int block) {
    const int low = t.begin >> p.page_shift, high = (t.end - 1) >> p.page_shift;
#pragma unroll
    for (int h = 0; h < 2; ++h) ahead[h] = table[min(max((block * kBlock + 16 * h) >> p.page_shift, low), high)];
  };
  auto turn = [&]() {  // (not right after look(): a check there would wait for the entries and for everything asked for before)
    if (min(ahead[0], ahead[1]) < 0 || max(ahead[0], ahead[1]) >= a.pages) raise_flag(a.bad_flag);
#pragma unroll
    for (int h = 0; h < 2; ++h) pages[h] = ahead[h] < 0 || ahead[h] >= a.pages ? -1 : ahead[h];
  };
  auto load_k = [&](int block) {  // A row r of tile c is key 8 (r / 4) + 4 c + r % 4
    const int pg = max(r < 8 ? pages[0] : pages[1], 0);
    const int at = (block * kBlock + 8 * (r >> 2) + (r & 3)) & (a.page - 1);
    const C* src = kc + ((int64_t)(pg * (int64_t)a.kv_heads + t.kvh) * a.page + at) * D + 8 * g;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) k[c][kk] = *reinterpret_cast<const u32x4*>(src + 4 * c * D + 32 * kk);
  };
  auto load_v = [&](int block) {
    const int pg = max(g < 2 ? pages[0] : pages[1], 0);
    const int at = (block * kBlock + 8 * g) & (a.page - 1);
    const C* src = vc + ((int64_t)(pg * (int64_t)a.kv_heads + t.kvh) * D + r) * a.page + at;
#pragma unroll
    for (int d = 0; d < DT; ++d) v[d] = *reinterpret_cast<const u32x4*>(src + (int64_t)d * 16 * a.page);
  };

  f32x4 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  int block = lo + wave;
  auto begin = [&]() {
    if (block < hi) {
      look(block);
      turn();
      load_k(block);
      load_v(block);
      look(block + kWaves);
    }
  };
  bool careful = false;
  begin();
  while (block < hi) {
    const int k0 = block * kBlock, ok0 = pages[0], ok1 = pages[1], next = block + kWaves;
    f32x4 s[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      s[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) s[c] = H::mma(__builtin_bit_cast(Frag<C>, k[c][kk]), q[kk], s[c]);
    }
    if (next < hi) {
      turn();
      load_k(next);
      look(next + kWaves);  // a block ahead of its use
    }
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = s[j >> 2][j & 3] * p.scale2;
    const bool whole = ok0 >= 0 && ok1 >= 0 && k0 + kBlock - 1 <= pos_lo && (a.window <= 0 || k0 > pos_hi - a.window);
    const bool ok = (g < 2 ? ok0 : ok1) >= 0;
    auto seen = [&](int j) {
      const int key = k0 + 8 * g + j;
      return ok && key <= pos && key >= least;
    };
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!seen(j)) x[j] = -INFINITY;
#pragma unroll
      for (int d = 0; d < DT; ++d) v[d] = ok ? keep_keys(v[d], k0 + 8 * g, t.begin, t.end) : u32x4{0u, 0u, 0u, 0u};
    }
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) mx = fmaxf(mx, x[j]);
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    if (__any(mx > m)) {
      const float mn = fmaxf(m, mx), keep = m == -INFINITY ? 0.f : exp2_(m - mn);
      m = mn;
      l *= keep;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= keep;
    }
    const float base = (m == -INFINITY ? 0.f : m) - H::kShift;
    float pr[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      pr[j] = exp2_(x[j] - base);
      l += pr[j];
    }
    Frag<C> pt[TERMS];
    split_terms<TERMS>(pr, pt);
    if (careful) {
      Frag<C> sf;
#pragma unroll
      for (int j = 0; j < 8; ++j) sf[j] = seen(j) ? (C)1.f : (C)0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = pv_each<C, TERMS>(v[d], pt, sf, o[d]);
    } else {
#pragma unroll
      for (int tm = 0; tm < TERMS; ++tm)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = H::mma(__builtin_bit_cast(Frag<C>, v[d]), pt[tm], o[d]);
    }
    if (next < hi) load_v(next);
    block = next;
    if (block >= hi && !careful) {  // a NaN: once more, with care
      bool odd = false;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) odd = odd || o[d][j] != o[d][j];
      if (__any(odd)) {
        careful = true;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
        m = -INFINITY, l = 0.f, block = lo + wave;
        begin();
      }
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // the waves' results through LDS: O^T registers hold columns 16 d + 4 g .. + 3 of row r
#pragma unroll
  for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(&stage[wave][r][16 * d + 4 * g]) = o[d];
  if (g == 0) stat[wave][0][r] = m, stat[wave][1][r] = l;
  __syncthreads();
  const Parts parts(p);
  const int dst = active > 1 ? (tile * p.splits + part) * part_floats<kRowsTile, D>() : -1;
  for (int i = threadIdx.x; i < t.rows * (D / 4); i += kThreads) {
    const int rr = i / (D / 4), col = i % (D / 4) * 4;
    float M = -INFINITY, L = 0.f, out[4] = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, stat[w][0][rr]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = stat[w][0][rr], lw = stat[w][1][rr], f = mw == -INFINITY ? 0.f : exp2_(mw - M);
      if (f == 0.f && lw == 0.f) continue;
      const f32x4 x = *reinterpret_cast<const f32x4*>(&stage[w][rr][col]);
      L = fmaf(f, lw, L);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] = fmaf(f, x[j], out[j]);
    }
    if (dst < 0) {
      finish<C, O, D>(p, t, rr, col, M, L, out);
    } else {
      parts.put4(dst + 2 * kRowsTile + rr * D + col, out);
      if (col == 0) parts.put(dst + rr, M), parts.put(dst + kRowsTile + rr, L);
    }
  }
  if (dst >= 0) join_tree<C, O, kRowsTile, D, kThreads>(p, t, parts, tile, part, active, &shared, &stage[0][0][0]);
}

// ---- many rows -----------------------------------------------------------------------------------------------------

// 16 bytes per lane from memory straight into LDS, lane i's at dst + 16 i.
__device__ inline void to_lds(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) unsigned*)src, (__attribute__((address_space(3))) unsigned*)dst, 16, 0, 0);
}
__device__ inline void to_lds(__amdgpu_buffer_rsrc_t r, int own, int at, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, own, at, 0, 0);
}
__device__ inline float max_halves(float x) {  // over lanes i and i + 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

constexpr int chunk_keys(int dim) { return dim == 256 ? 32 : 64; }  // keys of a tile: two tiles of K and V take 68 KB of LDS at most

// Places in LDS, of 16-byte pieces.  A read of 16 bytes takes 16 lanes at a time from 64 banks, so 16 consecutive rows'
// pieces of one column have to lie on 16 different places of 256 bytes.  K row by row, pieces exchanged by k_swap; V^T
// (rows of 64 or 128 bytes) as the loads leave it, 1 KB per instruction, pieces exchanged by v_swap, which is the same for a
// lane in every instruction (a lane's keys lie in one page then), and every second KB of 8 rows shifted by 128 bytes.
template <int D>
__device__ inline int k_swap(int key) {
  return D == 64 ? key >> 1 & 7 : key & 15;
}
template <int D>
__device__ inline int v_swap(int row) {
  return D == 256 ? row >> 2 & 3 : row & 7;
}
constexpr int v_block(int dim) { return dim == 256 ? 512 : 576; }  // values from one instruction's place to the next's
constexpr int v_values(int dim) { return dim * chunk_keys(dim) / 512 * v_block(dim); }
template <int D>
__device__ inline int v_place(int row, int piece) {
  constexpr int KT = chunk_keys(D), ROWS = 512 / KT;
  return row / ROWS * v_block(D) + row % ROWS * KT + (piece ^ v_swap<D>(row)) * 8;
}

// The row that a lane works on: its Q, and the keys [least, pos] that it sees.
template <typename C, int D>
struct ChunkRows {
  Frag<C> q[D / 16];
  int pos, least;
};

// Tiles [lo, hi) of KT keys for the 32 rows of each wave and DT tiles of 32 columns from column 32 d0 on.  CAREFUL: with
// pv_each.
template <typename C, int D, int TERMS, int DT, bool CAREFUL>
__device__ __forceinline__ void chunk_pass(const AttnParams& p, const Tile& t, int lo, int hi, const ChunkRows<C, D>& rows, C* kbuf, C* vbuf, int d0,
                                           f32x16 (&o)[DT], float& m, float& l) {
  typedef Half<C> H;
  constexpr int KT = chunk_keys(D), KK = D / 16, SB = KT / 32;
  {
    m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x16{};
  }
  constexpr int KC = D / 8, VC = KT / 8;                      // 16-byte pieces per row of K and V
  constexpr int NI = KT * D / 8 / chunk_threads(D);           // DMA instructions per wave, for K and for V
  constexpr int KSTEP = 64 / KC, VSTEP = 64 / VC;             // rows per instruction
  const auto& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31, g = lane >> 5;
  // The piece of V that this lane moves: row d0 + i * VSTEP, place pos, keys 8 * vchunk ..
  const int v_d0 = wave * NI * VSTEP + lane / VC, vchunk = lane % VC ^ v_swap<D>(v_d0);
  const int k_row0 = wave * NI * KSTEP + lane / KC;
  const C* kc = static_cast<const C*>(a.k_cache);
  const C* vc = static_cast<const C*>(a.v_cache);
  const int32_t* table = a.block_table + t.b * a.table_stride;
  const int first_page = t.begin >> p.page_shift;

  auto look = [&](int tile) {  // the page of this lane's keys of V; lane 2 q's is that of the tile's q-th 16 keys
    const int key = tile * KT + 8 * vchunk, at = key >> p.page_shift;
    int pg = -1;
    if (key < t.end && at >= first_page && tile < hi) {
      pg = table[at];
      if (pg < 0 || pg >= a.pages) raise_flag(a.bad_flag), pg = -1;
    }
    return pg;
  };
  // A page's K and V of this key head are one piece of memory each: its address goes through scalar registers, a lane's place
  // in it is the same for every tile but for the rows' exchange (415 -> 395 us for 2048 tokens over 8100 keys, 48 x 128).
  const int page_bytes = a.page * D * 2, k_off = lane / KC * D * 2, k_piece = lane % KC;
  const int v_off = v_d0 * a.page * 2 + vchunk * 16;
  auto fetch = [&](int tile, int pg, int buf) {
    const int64_t kpg = max(__builtin_amdgcn_readlane(pg, 2 * (wave * NI * KSTEP / 16)), 0);
    const auto kr = __builtin_amdgcn_make_buffer_rsrc(const_cast<C*>(kc + (kpg * a.kv_heads + t.kvh) * (int64_t)a.page * D), 0, page_bytes, 0x00027000);
    const int k_at = ((tile * KT + wave * NI * KSTEP) & (a.page - 1)) * D * 2;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      to_lds(kr, k_off + (k_piece ^ k_swap<D>(k_row0 + i * KSTEP)) * 16, k_at + i * KSTEP * D * 2, kbuf + buf * KT * D + (wave * NI + i) * 512);
    if (a.page >= KT) {  // the tile lies in one page
      const int64_t vpg = max(__builtin_amdgcn_readlane(pg, 0), 0);
      const auto vr = __builtin_amdgcn_make_buffer_rsrc(const_cast<C*>(vc + (vpg * a.kv_heads + t.kvh) * (int64_t)a.page * D), 0, page_bytes, 0x00027000);
      const int v_at = (tile * KT & (a.page - 1)) * 2;
#pragma unroll
      for (int i = 0; i < NI; ++i) to_lds(vr, v_off, v_at + i * VSTEP * a.page * 2, vbuf + buf * v_values(D) + (wave * NI + i) * v_block(D));
    } else {
      const int64_t vpg = max(pg, 0);
      const C* vs = vc + ((vpg * a.kv_heads + t.kvh) * D + v_d0) * (int64_t)a.page + ((tile * KT + 8 * vchunk) & (a.page - 1));
#pragma unroll
      for (int i = 0; i < NI; ++i) to_lds(vs + (int64_t)i * VSTEP * a.page, vbuf + buf * v_values(D) + (wave * NI + i) * v_block(D));
    }
  };

  int pg = look(lo), next_pg = -1;
  if (lo < hi) fetch(lo, pg, 0);
  next_pg = look(lo + 1);
  const int pos_lo = min(t.first_pos + p.token_of(t.row0), t.end - 1), pos_hi = t.last_pos;  // every row sees (pos_hi - window, pos_lo]
#pragma unroll 1
  for (int tile = lo, buf = 0; tile < hi; ++tile, buf ^= 1) {
    // the tile has arrived, and every wave has left the other buffer
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __syncthreads();
    const uint64_t there = __ballot(pg >= 0);
    pg = next_pg;
    if (tile + 1 < hi) fetch(tile + 1, pg, buf ^ 1);
    next_pg = look(tile + 2);
    const C* kt = kbuf + buf * KT * D;
    const C* vt = vbuf + buf * v_values(D);
    const int k0 = tile * KT;
    const bool whole = there == ~uint64_t(0) && k0 + KT - 1 <= pos_lo && (a.window <= 0 || k0 > pos_hi - a.window);
    if (!whole) {  // V of keys that no row sees: zeros
      for (int i = threadIdx.x; i < D * VC; i += chunk_threads(D)) {
        const int piece = i % VC, key = k0 + 8 * piece;
        u32x4* v = reinterpret_cast<u32x4*>(vbuf + buf * v_values(D) + v_place<D>(i / VC, piece));
        *v = there >> (piece & ~1) & 1 ? keep_keys(*v, key, t.begin, t.end) : u32x4{0u, 0u, 0u, 0u};
      }
      __syncthreads();
    }
    {
      // Operands are read from LDS one group ahead of the products that take them.
      f32x16 s[SB] = {};
      {
        constexpr int G = 4, GROUPS = SB * KK / G;
        Frag<C> f[2][G];
        auto read = [&](int q) {
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const int key = 32 * (q * G / KK) + (n & 0x13) + ((n & 4) << 1) + ((n & 8) >> 1), kk = q * G % KK + i;
            f[q & 1][i] = *reinterpret_cast<const Frag<C>*>(kt + key * D + ((2 * kk + g) ^ k_swap<D>(key)) * 8);
          }
        };
        read(0);
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
          if (q + 1 < GROUPS) read(q + 1);
          in_order();
#pragma unroll
          for (int i = 0; i < G; ++i)
            s[q * G / KK] = H::mma(f[q & 1][i], rows.q[q * G % KK + i], s[q * G / KK]);
        }
      }
      u32x4 v[2][DT];
      auto read_v = [&](int q) {
#pragma unroll
        for (int d = 0; d < DT; ++d) v[q & 1][d] = *reinterpret_cast<const u32x4*>(vt + v_place<D>(32 * (d0 + d) + n, 2 * q + g));
      };
      read_v(0);
      in_order();
      auto seen = [&](int b, int i) {
        const int at = 32 * b + 16 * (i >> 3) + 8 * g + (i & 7), key = k0 + at;
        return (there >> (2 * (at >> 4)) & 1) && key <= rows.pos && key >= rows.least;
      };
      if (!whole)
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!seen(b, i)) s[b][i] = -INFINITY;
      Frag<C> pf[SB][2][TERMS], sf[SB][2];
      {
        float mx = s[0][0];
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
        mx = max_halves(mx) * p.scale2;
        if (__any(mx > m + H::kSlack)) {
          const float mn = fmaxf(m, mx), keep = m == -INFINITY ? 0.f : exp2_(m - mn);
          m = mn;
          l *= keep;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] *= keep;
        }
        const float base = (m == -INFINITY ? 0.f : m) - H::kShift;
#pragma unroll
        for (int b = 0; b < SB; ++b) {
          float e[16], sum = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            e[i] = exp2_(fmaf(s[b][i], p.scale2, -base));
            sum += e[i];
          }
          l += sum;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            split_terms<TERMS>(e + 8 * h, pf[b][h]);
            if constexpr (CAREFUL)
#pragma unroll
              for (int j = 0; j < 8; ++j) sf[b][h][j] = (C)(seen(b, 8 * h + j) ? 1.f : 0.f);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 2 * SB; ++q) {
        if (q + 1 < 2 * SB) read_v(q + 1);
        in_order();
#pragma unroll
        for (int d = 0; d < DT; ++d)
          {
            if constexpr (CAREFUL) {
              o[d] = pv_each<C, TERMS>(v[q & 1][d], pf[q >> 1][q & 1], sf[q >> 1][q & 1], o[d]);
            } else {
#pragma unroll
              for (int e = 0; e < TERMS; ++e) o[d] = H::mma(__builtin_bit_cast(Frag<C>, v[q & 1][d]), pf[q >> 1][q & 1][e], o[d]);
            }
          }
      }
    }
  }
  __syncthreads();  // the buffers are free again
}

template <typename C, typename O, int D>
__global__ __launch_bounds__(chunk_threads(D), 2) void attn_chunk_kernel(AttnParams p) {
  constexpr int KT = chunk_keys(D), KK = D / 16, DT = D / 32 * 256 / chunk_threads(D), ROWS = kChunkTile;
  constexpr int TERMS = sizeof(O) == 4 ? Half<C>::kTerms : 1;
  __shared__ __attribute__((aligned(128))) C buffers[2 * (KT * D + v_values(D))];
  C *kbuf = buffers, *vbuf = buffers + 2 * KT * D;
  __shared__ int shared;
  const auto& a = p.a;
  const int lane = threadIdx.x & 63, waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = waves & 3, n = lane & 31, g = lane >> 5;
  const int d0 = waves / 4 * DT;  // this wave's first 32 columns
  const int part = blockIdx.x / (unsigned)p.tiles, tile = p.tile_of(blockIdx.x - part * p.tiles, part);
  const Tile t = find_tile<ROWS>(p, tile, lane);
  if (t.rows <= 0) return;
  const int first = t.begin / KT, blocks = t.end > 0 ? (t.end + KT - 1) / KT - first : 0;
  const int active = max(1, min(p.splits, blocks / kLeastTiles));
  if (part >= active) return;
  const int each = (unsigned)blocks / (unsigned)active, more = blocks - each * active;  // the first `more` parts have one more
  const int lo = first + each * part + min(part, more), hi = lo + each + (part < more ? 1 : 0);

  ChunkRows<C, D> rows;
  {
    const int in = wave * 32 + n;
    const bool ok = in < t.rows;
    const int row = t.row0 + (ok ? in : 0);
    const int token = p.token_of(row);
    rows.pos = min(t.first_pos + token, t.end - 1);
    rows.least = first_seen(a.window, t.first_pos + token);
    const C* src = static_cast<const C*>(a.q) + (t.t0 + token) * a.q_token + (int64_t)(t.kvh * p.group + row - token * p.group) * a.q_head + 8 * g;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      u32x4 x = *reinterpret_cast<const u32x4*>(src + 16 * kk);
      if (!ok) x = u32x4{0u, 0u, 0u, 0u};
      if (a.scale < 0.f) x ^= 0x80008000u;  // p.scale2 is positive
      rows.q[kk] = __builtin_bit_cast(Frag<C>, x);
    }
  }
  const Parts parts(p);
  const int dst = active > 1 ? (tile * p.splits + part) * part_floats<ROWS, D>() : -1;
  auto store = [&](int d, const f32x16& o, float m, float sum) {
    const int in = wave * 32 + n;
    if (in >= t.rows) return;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int col = 32 * d + 2 * i + 4 * g;
      const float v[4] = {o[i], o[i + 1], o[i + 2], o[i + 3]};
      if (dst < 0) {
        finish<C, O, D>(p, t, in, col, m, sum, v);
      } else {
        parts.put4(dst + 2 * ROWS + in * D + col, v);
        if (col == 0) parts.put(dst + in, m), parts.put(dst + ROWS + in, sum);
      }
    }
  };
  f32x16 o[DT];
  float m, l;
  chunk_pass<C, D, TERMS, DT, false>(p, t, lo, hi, rows, kbuf, vbuf, d0, o, m, l);
  bool odd = false;
  {
    l = sum_halves(l);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) odd = odd || o[d][i] != o[d][i];
  }
  if (!__syncthreads_or(odd)) {
#pragma unroll
      for (int d = 0; d < DT; ++d) store(d0 + d, o[d], m, l);
  } else {  // a NaN: once more, with care, 32 columns at a time
#pragma unroll 1
    for (int d = 0; d < DT; ++d) {
      f32x16 x[1];
      chunk_pass<C, D, TERMS, 1, true>(p, t, lo, hi, rows, kbuf, vbuf, d0 + d, x, m, l);
      store(d0 + d, x[0], m, sum_halves(l));
    }
  }
  if (dst >= 0) join_tree<C, O, ROWS, D, chunk_threads(D)>(p, t, parts, tile, part, active, &shared, reinterpret_cast<float*>(buffers));
  static_assert(sizeof(buffers) >= 2 * (kFan + 1) * ROWS * 4, "");
}

// ---- host ----------------------------------------------------------------------------------------------------------

// Registers and LDS allow two workgroups of four waves per compute unit, one of eight (or of four at 256 columns).
int places_shift(int dim) { return dim == 256 ? 8 : 9; }

// Tiles of the token axis, at most: as many per token as one token's rows take, or what all their rows take and one per
// sequence; whichever is fewer.  What is left over finds no rows.
int64_t tiles_of(int64_t tokens, int64_t seqs, int group, int rows) {
  return std::min(tokens * ((group + rows - 1) / rows), tokens * group / rows + seqs);
}

// attn_rows reads the cache once per 16 rows, attn_chunk once per 128, but computes tiles of 128 whatever their rows and
// joins longer.  attn_chunk where attn_rows would have two tiles or more per sequence and an eighth as many as the card
// holds: over 4000 keys, rows against chunk, in us: 1 stream x 16 tokens x 12 heads, 2 x 256: 30, 58 (24 tiles); 8 streams
// x 2 tokens: 35, 34 (32 tiles), x 4: 62, 42, x 16: 170, 69; 4 x 128, 8 streams x 2: 30, 31 (64 tiles), x 4: 43, 36.
bool in_chunks(int64_t tokens, int64_t seqs, int64_t max_len, int heads, int kv_heads, int dim) {
  if (tokens <= seqs) return false;
  const int group = heads / kv_heads;
  const int64_t rows = (max_len > 0 ? std::min(max_len, tokens) : (tokens + seqs - 1) / seqs) * group;
  return rows > kRowsTile && tiles_of(tokens, seqs, group, kRowsTile) * kv_heads >= (1 << places_shift(dim)) / 8;
}
bool in_chunks(const tq_paged_attn_args& a) { return in_chunks(a.tokens, a.seqs, a.max_len, a.heads, a.kv_heads, a.dim); }
// `parts` and what joins them: one per kFan of a tile's.
int64_t parts_bytes(int64_t parts, int rows, int dim) { return (parts + parts / 2 + kFan) * rows * (dim + 2) * 4; }

template <typename C, typename O, int D>
hipError_t launch_dim(AttnParams& p, hipStream_t s) {
  const auto& a = p.a;
  const bool chunks = in_chunks(a);
  p.places_shift = places_shift(D);
  const int rows = chunks ? kChunkTile : kRowsTile;
  p.tiles_each = (p.group + rows - 1) / rows;
  const int64_t slots = tiles_of(a.tokens, a.seqs, p.group, rows);
  const bool by_token = slots == a.tokens * p.tiles_each;
  p.slot_per = by_token ? p.tiles_each * rows : p.group, p.slot_add = by_token ? 0 : 1;
  const int64_t tiles = slots * a.kv_heads, keys = a.table_width * a.page;
  p.tiles = (int)tiles;
  p.splits = 1;
  if (a.workspace) {
    const int64_t units = chunks ? (keys + chunk_keys(D) - 1) / chunk_keys(D) : (keys + kWaves * kBlock - 1) / (kWaves * kBlock);
    // attn_chunk: parts only while they find free places; attn_rows decides in the kernel, from the lengths
    const int64_t room = chunks ? (1 << p.places_shift) / tiles : kMaxParts / tiles;
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({room, units, kMaxSplits}));
  }
  const dim3 grid((unsigned)(tiles * p.splits));
  if (chunks) {
    hipLaunchKernelGGL((attn_chunk_kernel<C, O, D>), grid, dim3(chunk_threads(D)), 0, s, p);
  } else {
    hipLaunchKernelGGL((attn_rows_kernel<C, O, D>), grid, dim3(kThreads), 0, s, p);
  }
  return hipGetLastError();
}

template <typename C, typename O>
hipError_t launch_type(AttnParams& p, hipStream_t s) {
  return p.a.dim == 64 ? launch_dim<C, O, 64>(p, s) : p.a.dim == 128 ? launch_dim<C, O, 128>(p, s) : launch_dim<C, O, 256>(p, s);
}

}  // namespace

int64_t paged_attn_workspace_bytes(int64_t tokens, int64_t seqs, int heads, int kv_heads, int dim) {
  if (tokens == 0) return 0;
  // whether attn_chunk runs depends on max_len too: room for it wherever it may
  const bool chunks = tokens > seqs && tokens * (heads / kv_heads) > kRowsTile;
  return kHeader + std::max(parts_bytes(kMaxParts, kRowsTile, dim), chunks ? parts_bytes(kMaxChunkParts, kChunkTile, dim) : 0);
}

int paged_attn_tile_rows(int64_t tokens, int64_t seqs, int64_t max_len, int heads, int kv_heads, int dim) {
  return tokens > 0 && in_chunks(tokens, seqs, max_len, heads, kv_heads, dim) ? kChunkTile : kRowsTile;
}

hipError_t launch_paged_attn(const tq_paged_attn_args& a, hipStream_t s) {
  AttnParams p{a};
  // attn_chunk takes a negative scale's sign into Q, and masks by -inf before the scaling: a scale of zero is the least
  p.scale2 = a.scale * kLog2e;
  p.group = a.heads / a.kv_heads;
  p.page_shift = __builtin_ctz(a.page);
  // row / group = row * ceil(2^(31 + s) / group) >> (31 + s) with 2^s >= group: 2 row times that, its high word, >> s
  const int sh = p.group == 1 ? 0 : 32 - __builtin_clz(p.group - 1);
  const uint64_t mul = ((uint64_t(1) << (31 + sh)) + p.group - 1) / p.group;
  p.group_mul = (unsigned)mul, p.group_shift = (unsigned)sh;
  if (in_chunks(a)) p.scale2 = std::max(std::fabs(p.scale2), FLT_MIN);
  if (a.cache_type == TQ_BF16) return a.out_type == TQ_F32 ? launch_type<bf16, float>(p, s) : launch_type<bf16, bf16>(p, s);
  return a.out_type == TQ_F32 ? launch_type<f16, float>(p, s) : launch_type<f16, f16>(p, s);
}

}  // namespace tq
