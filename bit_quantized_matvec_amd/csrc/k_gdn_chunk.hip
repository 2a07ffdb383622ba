// k_gdn_chunk.hip -- the gated delta rule over chunks of 64 tokens.
//
// Mathematics.  Within a chunk let G_i be the running sum of g, k_i and q_i the
// (normalised) rows, S the state before it.  Unrolling the recurrence, the
// values x_i = d_i that token i writes solve the unit triangular system
//   x_i + sum_{j<i} A_ij x_j = r_i,   A_ij = beta_i e^(G_i - G_j) k_i.k_j,
//   r_i = beta_i v_i - beta_i e^(G_i) S^T k_i,
// and with T = (I + A)^-1, P_ij = scale e^(G_i - G_j) q_i.k_j (j <= i):
//   X = T R,   out_i = scale e^(G_i) S^T q_i + sum_j P_ij x_j,
//   S <- e^(G_63) S + sum_j k_j (x) e^(G_63 - G_j) x_j.
// Every exponent is at most 0.  T and P do not depend on S: a first kernel
// computes them for all chunks at once; a second one walks the chunks of each
// sequence, one wave per 16 columns of a head's state (columns do not meet).
//
// Precision.  All products run on the bf16 matrix instructions with fp32 sums;
// operands are split into bf16 terms whose sum holds them: fp32 values as 3
// terms (24 bits, bf16's range is fp32's), fp16 as 2, bf16 as 1, and products
// of terms below 2^-24 of the whole are left out.  Q and K enter as given;
// norms and decays multiply rows of results.  Where out has 16 bits, what goes
// only into it (S in S^T q, P, X in P X) takes 2 terms: 2^-17 of the values'
// size beside the 2^-9 or 2^-12 of the output's own rounding.
// T is built in fp32 on the fp32 matrix instructions.  T maps R to X, as the
// recurrence does: with beta |k|^2 <= 2, which l2norm and beta <= 2 ensure, its
// transitions shrink the state and T's entries stay small.  The recursion over
// blocks forms T's own entries and, between them, A21 T11: sums of at most 32
// products of A (at most beta each) and T.  Keys that are longer and not
// normalised let T grow as the recurrence itself grows.
//
// Layout.  A matrix-instruction result leaves lane (n, g) with rows 4g .. 4g+3
// of column n, and an operand wants 8g .. 8g+7 of the summed index.  Rows of
// the left operands are therefore fed in the order row r of tile (s, c) =
// 32s + 8(r/4) + 4c + r%4, which leaves lane group g with 32s + 8g + 4c + i:
// two tiles make one operand, and the state, R and X go from product to product
// in the registers that they are in.  The first kernel writes K, Q, K^T, T and
// P as operands: 1 KB per fragment, 16 consecutive bytes per lane, zeros past
// the sequence's end.  K^T is K times the identity, whose result is K
// transposed in just that order.
//
// Values that are not finite reach only later tokens of the recurrence, but
// every row of a matrix product.  A chunk with any in q, k, beta, with g > 0 or
// a 1 / |k| above kMostNorm is walked token after token instead (as are
// sequences of less than kStepLen tokens), and so is one in which a token writes
// what is not finite or above 2^63: the second kernel looks at X before it is
// used, and keeps the state before the chunk until then.  A column whose state is
// not finite stays so, and all its outputs with it, either way: after the first
// chunk that it has walked it is not looked at any more.
//
// Bound.  The walk: one chunk after another on 4 SIMDs per 32 columns, 2.4 us a
// chunk at bf16, of which the matrix units take 0.7: splitting into terms, LDS
// between the products and three barriers are the rest.  4096 bf16 tokens, 48
// heads of 128 x 128: 179 us, 44 of them in the first kernel (149 MB written);
// token after token 6063.  Five fp32 sequences of 77 to 701 tokens: 175 us (1290).
// What else was measured at the first: one wave per 16 columns without LDS 1777
// us (its loads wait one by one), eight waves of 16 columns that all do the same
// 264, four waves that compute the outputs too 251.
#include <algorithm>
#include <cstddef>

#include "kernels.h"
#include "seq.h"

namespace tq {
namespace {

constexpr int kChunk = 64;
// Tokens from which a chunk is worth its first kernel: 16 key and 48 value heads of 128 x 128, steps against chunks: one
// sequence of 12 tokens 18 against 15 (bf16) and 22 us (fp32), of 16 23 against 15 and 22; eight of 12 48 against 48 and 66,
// of 16 63 against 48 and 66, of 20 76 against 48 and 67.
constexpr int kStepLen = 16;
constexpr int kPrepThreads = 256;
constexpr int64_t kBudget = int64_t(256) << 20;  // workspace: what the last-level cache holds
constexpr int kFragBytes = 1024;
constexpr int kScalarBytes = 2048;
constexpr float kLeastG = -1024.f;  // e^g is 0 in fp32 far above
constexpr float kMostNorm = 0x1p60f;  // of 1 / |k|: what a token writes, below 2^64, stays finite times it

typedef bf16 frag __attribute__((ext_vector_type(8)));

// Per chunk and value head.  beta is NaN in a chunk that is to be walked.  decay is one value, repeated: as a value that
// all lanes share the compiler would move it to a scalar register, and wait for it, right after its load.
struct Scalars {
  float beta[kChunk], far_k[kChunk], far_q[kChunk], last_k[kChunk], decay[kChunk];
};
static_assert(sizeof(Scalars) <= kScalarBytes, "");

template <typename IN>
constexpr int terms_in() {
  return sizeof(IN) == 4 ? 3 : __is_same(IN, bf16) ? 1 : 2;
}
constexpr int key_frags(int dk, int tk) { return 12 * (dk / 32) * tk; }  // K, Q, K^T of a chunk and key head
constexpr int tri_frags(int terms) { return 6 * terms; }                 // lower triangle in tiles of 16 x 32

struct ChunkParams {
  tq_gdn_args a;
  uint8_t* units;
  float* carry;  // states between launches, [nseq][v_heads][dk][dv]
  int64_t unit_bytes, seq0, slots;
  int nseq, chunk0, chunks;  // this launch: chunks [chunk0, chunk0 + chunks) of sequences [seq0, seq0 + nseq)
  int whole;                 // one launch for everything: chunks laid out by cu
  int last;
  int heads;  // value heads per workgroup of the first kernel
};

__device__ inline f32x4 mma(frag a, frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline f32x4 mma4(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// c += a b over the terms' products above 2^-24 of the whole
template <int TA, int TB>
__device__ inline f32x4 mma_terms(const frag* a, const frag* b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
      if (i + j < 3) c = mma(a[i], b[j], c);
  return c;
}

// place of row r of 16-row tile t in the chunk (or the head's rows)
__device__ inline int place(int t, int r) { return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3); }
__device__ inline int tri_at(int tile, int s) { return tile < 2 ? tile : 2 * tile - 2 + s; }

template <typename IN>
__device__ inline void load8(const IN* p, float* x) {
  const Vec<IN, 8> v = *reinterpret_cast<const Vec<IN, 8>*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (float)v.v[j];
}

__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// x[k] -= A[k][j] x[j] for k > j, lane k of each 16 holding row k of A.
template <int J, int K>
__device__ inline void step(const float* row, float* x) {
  if constexpr (K < 16) {
    const int a = __builtin_amdgcn_update_dpp(0, __float_as_int(row[J]), 0x150 + K, 0xF, 0xF, true);  // row_newbcast:K
    x[K] = fmaf(-__int_as_float(a), x[J], x[K]);
    step<J, K + 1>(row, x);
  }
}
template <int J>
__device__ inline void steps(const float* row, float* x) {
  if constexpr (J < 15) {
    step<J, J + 1>(row, x);
    steps<J + 1>(row, x);
  }
}

// ---- T, P and the operands of every chunk --------------------------------------------------------------------------

template <typename IN, int DK, int OT>
__global__ __launch_bounds__(kPrepThreads, 2) void gdn_prepare_kernel(ChunkParams p) {
  constexpr int KS = DK / 32, TK = terms_in<IN>(), W = kChunk + 4;
  constexpr int kStage = std::max<int>(4 * KS * TK * kFragBytes, kChunk * W * 4);
  __shared__ __attribute__((aligned(16))) float A[kChunk][W];
  __shared__ __attribute__((aligned(16))) char stage[kStage];  // K's operands, then T
  frag(*ks)[KS][TK][64] = reinterpret_cast<frag(*)[KS][TK][64]>(stage);
  float(*T)[W] = reinterpret_cast<float(*)[W]>(stage);
  __shared__ double sums[kChunk];
  __shared__ float norms[kChunk];
  const auto& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, g = lane >> 4;
  // `heads` value heads of one key head: K Q^T and K K^T serve them all
  const int sets = a.v_heads / p.heads, h0 = (int)(blockIdx.x % sets) * p.heads, group = a.v_heads / a.k_heads, kh = h0 / group;
  const int64_t slot = blockIdx.x / sets;
  const int64_t b = p.whole ? find_seq(a.cu, a.seqs, 1, kChunk, 1, slot, lane) : p.seq0 + slot / p.chunks;
  const SeqRange r = seq_range(a.cu, b, a.tokens, nullptr);
  const int64_t c = p.whole ? slot - (r.t0 / kChunk + b) : p.chunk0 + slot % p.chunks;
  if (r.n < kStepLen || c < 0 || c * kChunk >= r.n) return;
  const int64_t t0 = r.t0 + c * kChunk;
  const int len = min(kChunk, r.n - (int)c * kChunk);

  uint8_t* unit = p.units + slot * p.unit_bytes;
  uint8_t* keys = unit + (int64_t)kh * (key_frags(DK, TK) * kFragBytes);
  auto put = [&](uint8_t* at, int index, frag f) { *reinterpret_cast<frag*>(at + index * kFragBytes + lane * 16) = f; };
  const bool writes_keys = h0 % group == 0;

  // this wave's 16 tokens, as right operands; column n is token i
  const int i = place(wave, n);
  const IN* kp = static_cast<const IN*>(a.k) + t0 * a.k_token + kh * a.k_head + 8 * g;
  const IN* qp = static_cast<const IN*>(a.q) + t0 * a.q_token + kh * a.q_head + 8 * g;
  frag qf[KS][TK], kf[KS][TK];
  float qq = 0.f, kk = 0.f;
  {
    const int at = min(i, len - 1);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8], y[8];
      load8(qp + at * a.q_token + 32 * s, x);
      load8(kp + at * a.k_token + 32 * s, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        qq = fmaf(x[j], x[j], qq), kk = fmaf(y[j], y[j], kk);
        if (len < kChunk && i >= len) x[j] = y[j] = 0.f;
      }
      split_terms<TK>(x, qf[s]);
      split_terms<TK>(y, kf[s]);
#pragma unroll
      for (int t = 0; t < TK; ++t) ks[wave][s][t][lane] = kf[s][t];
    }
  }
  qq += __shfl_xor(qq, 16, 64), kk += __shfl_xor(kk, 16, 64);
  qq += __shfl_xor(qq, 32, 64), kk += __shfl_xor(kk, 32, 64);
  float nq = (a.l2norm ? 1.f / sqrtf(qq + a.eps) : 1.f) * a.scale, nk = a.l2norm ? 1.f / sqrtf(kk + a.eps) : 1.f;
  const bool odd_rows = i < len && (!(qq < INFINITY) || !(kk < INFINITY) || !(fabsf(nq) < INFINITY) || !(nk < kMostNorm));
  if (i >= len) nq = nk = 0.f;
  if (g == 0) norms[i] = nk;
  __syncthreads();
  f32x4 akk[2][2] = {}, aqk[2][2] = {};
#pragma unroll
  for (int s2 = 0; s2 < 2; ++s2) {
    if (s2 > wave >> 1) continue;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        frag kt[TK];
#pragma unroll
        for (int e = 0; e < TK; ++e) kt[e] = ks[2 * s2 + t][s][e][lane];
        akk[s2][t] = mma_terms<TK, TK>(kt, kf[s], akk[s2][t]), aqk[s2][t] = mma_terms<TK, TK>(kt, qf[s], aqk[s2][t]);
      }
  }
  if (writes_keys) {
    const int s2 = wave >> 1, c2 = wave & 1;  // this wave transposes every second tile of the head's rows
    frag one;
#pragma unroll
    for (int j = 0; j < 8; ++j) one[j] = (bf16)(8 * g + j == place(c2, n) ? 1.f : 0.f);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int t = 0; t < TK; ++t) {
        const f32x4 lo = mma(ks[2 * s2][s][t][lane], one, f32x4{}), hi = mma(ks[2 * s2 + 1][s][t][lane], one, f32x4{});
        frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = (bf16)lo[j], f[4 + j] = (bf16)hi[j];
        put(keys + 8 * KS * TK * kFragBytes, ((2 * s + c2) * 2 + s2) * TK + t, f);
        put(keys, (wave * KS + s) * TK + t, kf[s][t]);
        put(keys + 4 * KS * TK * kFragBytes, (wave * KS + s) * TK + t, qf[s][t]);
      }
  }
  float beta = 0.f, gate = 0.f;
  auto load_head = [&](int h) {
    if (i < len) beta = a.beta[(t0 + i) * a.v_heads + h];
    if (lane < len) gate = a.g[(t0 + lane) * a.v_heads + h];
  };
  load_head(h0);
#pragma unroll 1
  for (int h = h0; h < h0 + p.heads; ++h) {
    uint8_t* tri = unit + (int64_t)a.k_heads * (key_frags(DK, TK) * kFragBytes) + (int64_t)h * (tri_frags(3 + OT) * kFragBytes + kScalarBytes);
    Scalars* sc = reinterpret_cast<Scalars*>(tri + tri_frags(3 + OT) * kFragBytes);
    if (wave == 0) {
      double sum = fmaxf(gate, kLeastG) * 1.4426950408889634074;  // in powers of two
#pragma unroll
      for (int o = 1; o < kChunk; o <<= 1) {
        const double y = __shfl_up(sum, o, 64);
        if (lane >= o) sum += y;
      }
      sums[lane] = sum;
    }
    const bool odd = __syncthreads_or(odd_rows || !(fabsf(beta) < INFINITY) || !(gate <= 0.f));
    const float be = beta, nb = beta * nk;
    if (h + 1 < h0 + p.heads) load_head(h + 1);
    if (odd) {
      if (g == 0) sc->beta[i] = NAN;
      continue;
    }
    const double mine = sums[i], all = sums[kChunk - 1];
#pragma unroll
    for (int s2 = 0; s2 < 2; ++s2) {
      if (s2 > wave >> 1) continue;
      float ra[8], rp[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = 32 * s2 + 8 * g + j;
        const float e = exp2_(fminf((float)(mine - sums[row]), 0.f)) * norms[row];
        const float q = nq * e * aqk[s2][j >> 2][j & 3], k = nb * e * akk[s2][j >> 2][j & 3];
        rp[j] = row <= i ? q : 0.f;
        ra[j] = row < i ? k : 0.f;
      }
      *reinterpret_cast<float4*>(&A[i][32 * s2 + 8 * g]) = float4{ra[0], ra[1], ra[2], ra[3]};
      *reinterpret_cast<float4*>(&A[i][32 * s2 + 8 * g + 4]) = float4{ra[4], ra[5], ra[6], ra[7]};
      frag pf[OT];
      split_terms<OT>(rp, pf);
#pragma unroll
      for (int t = 0; t < OT; ++t) put(tri + tri_frags(3) * kFragBytes, tri_at(wave, s2) * OT + t, pf[t]);
    }
    if (g == 0) {
      const float far = exp2_((float)mine);
      sc->beta[i] = be;
      sc->far_k[i] = be * far * nk;
      sc->far_q[i] = far * nq;
      sc->last_k[i] = exp2_((float)(all - mine)) * nk;
      sc->decay[i] = exp2_((float)all);
    }

    // T: the diagonal blocks of 16 by substitution, one block in 16 lanes of the first wave: a lane holds row n of A and
    // column n of T, and a step takes A's row k from lane k ...
    __syncthreads();
    if (wave == 0) {
      float row[16], x[16];
#pragma unroll
      for (int k = 0; k < 16; k += 4) *reinterpret_cast<f32x4*>(row + k) = *reinterpret_cast<const f32x4*>(&A[16 * g + n][16 * g + k]);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = k == n ? 1.f : 0.f;
      steps<0>(row, x);
#pragma unroll
      for (int k = 0; k < 16; ++k) T[16 * g + k][16 * g + n] = x[k];
    } else if (wave < 3) {  // the blocks above the diagonal that operands of 32 columns reach
#pragma unroll
      for (int k = 0; k < 4; ++k) T[32 * (wave - 1) + 4 * g + k][32 * (wave - 1) + 16 + n] = 0.f;
    }
    __syncthreads();
    // ... then T21 = -T22 (A21 T11), for blocks of 16 and of 32.  A step's 4 summed indices are 4g + s: what a result holds.
    auto block = [&](const float(*l)[W], int li, int lj, f32x4 right, f32x4 sum, float sign) {
#pragma unroll
      for (int s = 0; s < 4; ++s) sum = mma4(sign * l[16 * li + n][16 * lj + 4 * g + s], right[s], sum);
      return sum;
    };
    auto column = [&](int bi, int bj) {
      f32x4 v;
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = T[16 * bi + 4 * g + s][16 * bj + n];
      return v;
    };
    auto store = [&](int bi, int bj, f32x4 v) {
#pragma unroll
      for (int s = 0; s < 4; ++s) T[16 * bi + 4 * g + s][16 * bj + n] = v[s];
    };
    if (wave < 2) {
      const f32x4 m = block(A, 2 * wave + 1, 2 * wave, column(2 * wave, 2 * wave), f32x4{}, 1.f);
      store(2 * wave + 1, 2 * wave, block(T, 2 * wave + 1, 2 * wave + 1, m, f32x4{}, -1.f));
    }
    __syncthreads();
    if (wave < 2) {
      f32x4 m[2] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k < wave) continue;
        const f32x4 v = column(k, wave);
#pragma unroll
        for (int t = 0; t < 2; ++t) m[t] = block(A, 2 + t, k, v, m[t], 1.f);
      }
      store(2, wave, block(T, 2, 2, m[0], f32x4{}, -1.f));
      store(3, wave, block(T, 3, 3, m[1], block(T, 3, 2, m[0], f32x4{}, -1.f), -1.f));
    }
    __syncthreads();
#pragma unroll 1
    for (int s2 = 0; s2 <= wave >> 1; ++s2) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = T[i][32 * s2 + 8 * g + j];
      frag f[3];
      split_terms<3>(x, f);
#pragma unroll
      for (int t = 0; t < 3; ++t) put(tri, tri_at(wave, s2) * 3 + t, f[t]);
    }
  }
}

// ---- the walk over the chunks --------------------------------------------------------------------------------------

constexpr int kWalkThreads = 512;

// Waits for this wave's LDS traffic alone: loads from memory stay in flight across it.
__device__ inline void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

typedef bf16 half_frag __attribute__((ext_vector_type(4)));
template <int TERMS>
__device__ inline void split4(f32x4 v, half_frag* out) {
  const float x[4] = {v[0], v[1], v[2], v[3]};
  split_terms<TERMS>(x, out);
}

// A value as it is loaded, and as a number: 16 bits wait in a register of their own until they are needed.
template <typename IN>
struct Raw {
  typedef unsigned short mem;
  typedef unsigned type;
  static __device__ float number(unsigned x) { return (float)__builtin_bit_cast(IN, (unsigned short)x); }
};
template <>
struct Raw<float> {
  typedef float mem, type;
  static __device__ float number(float x) { return x; }
};

// Stores that drop what lies past the `bytes` from `base` on.
__device__ inline void put_out(__amdgpu_buffer_rsrc_t r, int at, float v) { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at * 4, 0, 0); }
template <typename C>
__device__ inline void put_out(__amdgpu_buffer_rsrc_t r, int at, C v) {
  __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), r, at * 2, 0, 0);
}
__device__ inline void in_order() { asm volatile("" ::: "memory"); }  // loads before it are issued before it

// A workgroup has 32 columns of one head's state.  Four waves, one per SIMD, carry the recurrence from chunk to chunk; four
// more, beside them, compute the outputs, which nothing waits for.  A chunk is three steps between barriers:
//   1  K S, R            |  P X and the stores of the chunk before
//   2  X = T R           |  Q S
//   3  the next state    |  X as right operands of P X
template <typename IN, typename O, int DK>
__global__ __launch_bounds__(kWalkThreads, 2) void gdn_walk_kernel(ChunkParams p) {
  constexpr int KS = DK / 32, HT = KS / 2, TK = terms_in<IN>(), OT = sizeof(O) == 4 ? 3 : 2;
  constexpr int AHEAD = TK == 1 ? 1 : 0;  // reads of right operands ahead of their products: where the left ones leave registers
  // right operands: the state, R and X with the decays to the chunk's end; X itself, the 8 values of an operand's lane together
  __shared__ __attribute__((aligned(16))) frag sf[KS][2][3][64], rf[2][2][3][64], zf[2][2][3][64];
  __shared__ __attribute__((aligned(16))) float xs[2][2][64][8], sums[2][4][2][32], norms[2][4][4];
  __shared__ __attribute__((aligned(16))) int odds[4];
  const auto& a = p.a;
  const int lane = threadIdx.x & 63, waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = waves & 3, n = lane & 15, g = lane >> 4;
  const bool carries = waves < 4;
  const int slices = a.dv / 32;
  // Slices of a head read the same operands, heads of a group the same K and Q: they share an XCD (workgroups go round the
  // 8 of them), unless that left XCDs without work.
  const int group = a.v_heads / a.k_heads, together = (int64_t)p.nseq * a.k_heads >= 8 ? group : 1;
  const int64_t x = blockIdx.x / 8 / (slices * together) * 8 + blockIdx.x % 8;
  const int in = blockIdx.x / 8 % (slices * together);
  const int64_t head = x * together + in / slices;
  if (head >= (int64_t)p.nseq * a.v_heads) return;
  const int col = in % slices * 32, h = (int)(head % a.v_heads), kh = h / group;
  const int64_t b = p.seq0 + head / a.v_heads;

  SeqRange r = seq_range(a.cu, b, a.tokens, a.bad_flag);
  r.t0 = __builtin_amdgcn_readfirstlane((int)r.t0), r.n = __builtin_amdgcn_readfirstlane(r.n);  // for scalar addresses
  const bool first = p.chunk0 == 0;
  const int64_t from = (int64_t)p.chunk0 * kChunk;
  if (!first && from >= r.n) return;
  const int64_t slot = a.slots ? a.slots[b] : b;
  const bool kept = slot >= 0 && slot < a.states;
  if (slot >= a.states) raise_flag(a.bad_flag);
  const bool ends = p.last || from + (int64_t)p.chunks * kChunk >= r.n;

  // Wave w of either four has tiles w * HT .. of the state's rows and tile w of a chunk's tokens.
  f32x4 s[HT][2] = {};
  float* carry = p.carry ? p.carry + ((b - p.seq0) * a.v_heads + h) * DK * (int64_t)a.dv : nullptr;
  const int64_t state_at = ((kept ? slot : 0) * a.v_heads + h) * DK * (int64_t)a.dv;
  auto row_of = [&](int e) { return 32 * ((wave * HT + e) >> 1) + 8 * g + 4 * ((wave * HT + e) & 1); };  // 4 rows from there
  if (carries && (!first || kept)) {
    const float* src = first ? a.state + state_at : carry;
#pragma unroll
    for (int e = 0; e < HT; ++e)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[e][m][j] = src[(row_of(e) + j) * a.dv + col + 16 * m + n];
  }

  // Tokens [t, end) one after another.
  int parity = 0;
  auto walk = [&](int64_t t, int64_t end) {
    if (!carries) {
      for (; t < end; ++t) lds_barrier();
      return;
    }
#pragma unroll 1
    for (; t < end; ++t, parity ^= 1) {
      const IN* qp = static_cast<const IN*>(a.q) + t * a.q_token + kh * a.q_head;
      const IN* kp = static_cast<const IN*>(a.k) + t * a.k_token + kh * a.k_head;
      const IN* vp = static_cast<const IN*>(a.v) + t * a.v_token + h * a.v_head + col + n;
      float q[HT][4], k[HT][4], qq = 0.f, kk = 0.f, kq = 0.f, r1[2] = {}, r2[2] = {};
#pragma unroll
      for (int e = 0; e < HT; ++e) {
        const Vec<IN, 4> qi = *reinterpret_cast<const Vec<IN, 4>*>(qp + row_of(e)), ki = *reinterpret_cast<const Vec<IN, 4>*>(kp + row_of(e));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = q[e][j] = (float)qi.v[j], y = k[e][j] = (float)ki.v[j];
          qq = fmaf(x, x, qq), kk = fmaf(y, y, kk), kq = fmaf(x, y, kq);
#pragma unroll
          for (int m = 0; m < 2; ++m) r1[m] = fmaf(s[e][m][j], y, r1[m]), r2[m] = fmaf(s[e][m][j], x, r2[m]);
        }
      }
#pragma unroll
      for (int o = 16; o < 64; o <<= 1) {
        qq += __shfl_xor(qq, o, 64), kk += __shfl_xor(kk, o, 64), kq += __shfl_xor(kq, o, 64);
#pragma unroll
        for (int m = 0; m < 2; ++m) r1[m] += __shfl_xor(r1[m], o, 64), r2[m] += __shfl_xor(r2[m], o, 64);
      }
      if (g == 0)
#pragma unroll
        for (int m = 0; m < 2; ++m) sums[parity][wave][0][16 * m + n] = r1[m], sums[parity][wave][1][16 * m + n] = r2[m];
      if (lane == 0) norms[parity][wave][0] = qq, norms[parity][wave][1] = kk, norms[parity][wave][2] = kq;
      lds_barrier();
      auto total = [](const float* x, int step) { return (x[0] + x[step]) + (x[2 * step] + x[3 * step]); };
      qq = total(&norms[parity][0][0], 4), kk = total(&norms[parity][0][1], 4), kq = total(&norms[parity][0][2], 4);
      const float nq = (a.l2norm ? 1.f / sqrtf(qq + a.eps) : 1.f) * a.scale, nk = a.l2norm ? 1.f / sqrtf(kk + a.eps) : 1.f;
      const float decay = expf(a.g[t * a.v_heads + h]), beta = a.beta[t * a.v_heads + h];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float s1 = total(&sums[parity][0][0][16 * m + n], 64) * nk, s2 = total(&sums[parity][0][1][16 * m + n], 64) * nq;
        const float d = beta * ((float)vp[16 * m] - decay * s1);
        if (wave == 0 && g == 0) static_cast<O*>(a.out)[(t * a.v_heads + h) * a.dv + col + 16 * m + n] = (O)fmaf(kq * nq * nk, d, decay * s2);
#pragma unroll
        for (int e = 0; e < HT; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[e][m][j] = fmaf(k[e][j] * nk, d, decay * s[e][m][j]);
      }
    }
  };
  auto half = [&](frag* f, int c) -> half_frag* { return reinterpret_cast<half_frag*>(f + lane) + c; };
  auto put_state = [&]() {
#pragma unroll
    for (int e = 0; e < HT; ++e)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int t = wave * HT + e;
        half_frag f[3];
        split4<3>(s[e][m], f);
#pragma unroll
        for (int i = 0; i < 3; ++i) *half(sf[t >> 1][m][i], t & 1) = f[i];
      }
  };

  uint64_t seen[2] = {~uint64_t(0), ~uint64_t(0)};  // the lanes whose column's state may be finite
  int64_t done = r.n < kStepLen ? 0 : from;
  const int64_t stop = r.n < kStepLen ? 0 : min((int64_t)r.n, from + (int64_t)p.chunks * kChunk);
  while (true) {
    // Chunks up to `stop`, or to one that has to be walked; then that, or the rest (sequences too short for chunks, and what
    // a wrong max_len left over).
    int64_t walk_to = ends ? r.n : done;
    bool odd = false;
    if (done < stop) {
      const int s2 = wave >> 1, c2 = wave & 1, row = 32 * s2 + 8 * g + 4 * c2;  // of this wave's tokens, 4 from there
      uint8_t* unit = p.units + (p.whole ? r.t0 / kChunk + b + done / kChunk : (b - p.seq0) * p.chunks + done / kChunk - p.chunk0) * p.unit_bytes;
      // Places in a chunk's unit are scalar offsets beside a lane's own: no vector arithmetic for addresses.
      const int kq_at = kh * key_frags(DK, TK) * kFragBytes;
      const int t_at = (a.k_heads * key_frags(DK, TK) + h * tri_frags(3 + OT)) * kFragBytes + h * kScalarBytes;
      const int p_at = t_at + tri_frags(3) * kFragBytes, sc_at = t_at + tri_frags(3 + OT) * kFragBytes;
      const int second = s2 ? kFragBytes : 0;  // from a tile's first part of T or P, and per term, to its second (the upper tiles: the first again)
      auto get = [&](int own, int at) {
        return __builtin_bit_cast(frag, __builtin_amdgcn_raw_buffer_load_b128(__builtin_amdgcn_make_buffer_rsrc(unit, 0, (int)p.unit_bytes, 0x00027000), own, at, 0));
      };
      auto row4 = [&](int at) {
        return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(__builtin_amdgcn_make_buffer_rsrc(unit, 0, (int)p.unit_bytes, 0x00027000),
                                                                               row * 4, sc_at + at, 0));
      };
      // Each role keeps what it takes from memory for a chunk in registers, and asks for a part again, for the next chunk,
      // after its last use.  The loops have one way out: any other would have the compiler move registers that are being
      // loaded, and wait for them.  So a chunk that has to be walked goes on to the end of the body, and its results are
      // dropped.
      if (carries) {
        typedef typename Raw<IN>::mem mem;
        const mem* vp = static_cast<const mem*>(a.v) + (r.t0 + done) * a.v_token + h * a.v_head + col + n;
        frag kf[KS][TK], xf[HT][2][TK], tf[2][3];
        f32x4 be, fk, lk;
        typename Raw<IN>::type v[2][4];
        float decay;
        int64_t v_at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v_at[j] = (row + j) * a.v_token;
        auto load_k = [&](int len) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < TK; ++e) kf[k][e] = get(lane * 16, kq_at + ((wave * KS + k) * TK + e) * kFragBytes);
          if (len < kChunk)  // rows past the end: the last one again
#pragma unroll
            for (int j = 0; j < 4; ++j) v_at[j] = min(row + j, len - 1) * a.v_token;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < 2; ++m) v[m][j] = vp[v_at[j] + 16 * m];
          be = row4(offsetof(Scalars, beta)), fk = row4(offsetof(Scalars, far_k));
        };
        auto load_t = [&]() {
#pragma unroll
          for (int k = 0; k < 2; ++k)  // (not used, but loaded, where there is no second one: the waits count loads)
#pragma unroll
            for (int e = 0; e < 3; ++e) tf[k][e] = get(lane * 16 + k * 3 * second, t_at + (tri_at(wave, 0) * 3 + e) * kFragBytes);
          lk = row4(offsetof(Scalars, last_k));
        };
        auto load_x = [&]() {
#pragma unroll
          for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < TK; ++e)
                xf[t][k][e] = get(lane * 16, kq_at + (8 * KS * TK + ((wave * HT + t) * 2 + k) * TK + e) * kFragBytes);
          decay = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(__builtin_amdgcn_make_buffer_rsrc(unit, 0, (int)p.unit_bytes, 0x00027000), row * 4,
                                                                       sc_at + (int)offsetof(Scalars, decay), 0));
        };
        int len = (int)min((int64_t)kChunk, stop - done);
        load_k(len);
        load_t();
        load_x();
        __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // or the loop's waits would count from here, in whatever order these were issued
        put_state();
        lds_barrier();
#pragma unroll 1
        do {
          const int now = len;
          if (done + kChunk < stop) {  // the next chunk's places (the last chunk's are asked for twice)
            len = (int)min((int64_t)kChunk, stop - done - kChunk);
            unit += p.unit_bytes, vp += kChunk * a.v_token;
          }
          // K S: each operand is read while the one before it is multiplied
          f32x4 y[2] = {}, y2[2] = {};
          {
            frag f[AHEAD + 1][2][3];
            auto read = [&](int k) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 3; ++e) f[k & AHEAD][m][e] = sf[k][m][e][lane];
            };
            if (AHEAD) read(0);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              if (k + AHEAD < KS) read(k + AHEAD);
              in_order();
#pragma unroll
              for (int i = 0; i < TK; ++i)
#pragma unroll
                for (int e = 0; e < 3; ++e)
#pragma unroll
                  for (int m = 0; m < 2; ++m)
                    if (i + e < 3) (k & 1 ? y2 : y)[m] = mma(kf[k][i], f[k & AHEAD][m][e], (k & 1 ? y2 : y)[m]);
            }
          }
          // R = beta V - far_k (K S)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float vj = row + j < now ? Raw<IN>::number(v[m][j]) : 0.f;
              y[m][j] = fmaf(be[j], vj, -fk[j] * (y[m][j] + y2[m][j]));
            }
            half_frag f[3];
            split4<3>(y[m], f);
#pragma unroll
            for (int e = 0; e < 3; ++e) *half(rf[s2][m][e], c2) = f[e];
          }
          load_k(len);
          lds_barrier();
          // X = T R
          {
            frag f[2][2][3];
            auto read = [&](int k) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 3; ++e) f[k][m][e] = rf[k][m][e][lane];
            };
            auto product = [&](int k) {
#pragma unroll
              for (int e = 0; e < 3; ++e)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  y[m] = mma(tf[k][e], f[k][m][0], y[m]);
                  y2[m] = mma(tf[k][e == 2 ? 0 : e], f[k][m][e == 2 ? 2 : 1], y2[m]);
                }
            };
#pragma unroll
            for (int m = 0; m < 2; ++m) y[m] = f32x4{}, y2[m] = f32x4{};
            read(0);
            if (s2 && AHEAD) read(1);
            in_order();
            product(0);
            if (s2 && !AHEAD) read(1);
            if (s2) product(1);
          }
          // Squares: infinite or NaN long before a term is (lk is below kMostNorm), and T's ones bring what is not finite in R
          // (beta, v, the state, or an overflow) to X.
          float size[2] = {};
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            y[m] += y2[m];
#pragma unroll
            for (int j = 0; j < 4; ++j) size[m] = fmaf(y[m][j], y[m][j], size[m]);
            half_frag f[3];
            split4<3>(y[m] * lk, f);
#pragma unroll
            for (int e = 0; e < 3; ++e) *half(zf[s2][m][e], c2) = f[e];
            *reinterpret_cast<f32x4*>(&xs[s2][m][lane][4 * c2]) = y[m];
          }
          load_t();
          const uint64_t bad = (__ballot(!(size[0] < INFINITY)) & seen[0]) | (__ballot(!(size[1] < INFINITY)) & seen[1]);
          if (lane == 0) odds[wave] = bad != 0;
          lds_barrier();
          odd = __builtin_amdgcn_readfirstlane(odds[0] | odds[1] | odds[2] | odds[3]) != 0;
          // S = decay S + K^T Z
#pragma unroll
          for (int t = 0; t < HT; ++t)
#pragma unroll
            for (int m = 0; m < 2; ++m) s[t][m] *= decay;
          {
            frag f[AHEAD + 1][2][3];
            auto read = [&](int k) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 3; ++e) f[k & AHEAD][m][e] = zf[k][m][e][lane];
            };
            if (AHEAD) read(0);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (k + AHEAD < 2) read(k + AHEAD);
              in_order();
#pragma unroll
              for (int i = 0; i < TK; ++i)
#pragma unroll
                for (int e = 0; e < 3; ++e)
#pragma unroll
                  for (int t = 0; t < HT; ++t)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                      if (i + e < 3) s[t][m] = mma(xf[t][k][i], f[k & AHEAD][m][e], s[t][m]);
            }
          }
          if (!odd) put_state();
          load_x();
          lds_barrier();
          done += kChunk;
        } while (!odd && done < stop);
        if (odd)  // the state before the chunk: its terms' sum, which is exact
#pragma unroll
          for (int e = 0; e < HT; ++e)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int t = wave * HT + e;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                auto term = [&](int i) { return (float)(*half(sf[t >> 1][m][i], t & 1))[j]; };
                s[e][m][j] = (term(2) + term(1)) + term(0);
              }
            }
      } else {
        frag qf[KS][TK], pf[2][OT];
        f32x4 fq;
        auto load_q = [&]() {
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < TK; ++e) qf[k][e] = get(lane * 16, kq_at + (4 * KS * TK + (wave * KS + k) * TK + e) * kFragBytes);
          fq = row4(offsetof(Scalars, far_q));
        };
        auto load_p = [&]() {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < OT; ++e) pf[k][e] = get(lane * 16 + k * OT * second, p_at + (tri_at(wave, 0) * OT + e) * kFragBytes);
        };
        load_q();
        load_p();
        __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
        lds_barrier();
#pragma unroll 1
        do {
          const int now = (int)min((int64_t)kChunk, stop - done);
          if (done + kChunk < stop) unit += p.unit_bytes;
          lds_barrier();
          // far_q (Q S)
          f32x4 o[2] = {};
          {
            frag f[2][2][OT];
            auto read = [&](int k) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < OT; ++e) f[k & 1][m][e] = sf[k][m][e][lane];
            };
            read(0);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              if (k + 1 < KS) read(k + 1);
              in_order();
#pragma unroll
              for (int i = 0; i < TK; ++i)
#pragma unroll
                for (int e = 0; e < OT; ++e)
#pragma unroll
                  for (int m = 0; m < 2; ++m)
                    if (i + e < 3) o[m] = mma(qf[k][i], f[k & 1][m][e], o[m]);
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) o[m] *= fq;
          load_q();
          lds_barrier();
          odd = __builtin_amdgcn_readfirstlane(odds[0] | odds[1] | odds[2] | odds[3]) != 0;
          frag f[2][2][OT];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (k <= s2)
#pragma unroll
              for (int m = 0; m < 2; ++m) split_terms<OT>(&xs[k][m][lane][0], f[k][m]);
          lds_barrier();
          // out = far_q (Q S) + P X
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (k <= s2)
#pragma unroll
              for (int m = 0; m < 2; ++m) o[m] = mma_terms<OT, OT>(pf[k], f[k][m], o[m]);
          load_p();
          const auto op = __builtin_amdgcn_make_buffer_rsrc(static_cast<O*>(a.out) + (r.t0 + done) * a.v_heads * a.dv, 0,
                                                            odd ? 0 : now * a.v_heads * a.dv * (int)sizeof(O), 0x00027000);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < 2; ++m) put_out(op, ((row + j) * a.v_heads + h) * a.dv + col + 16 * m + n, (O)o[m][j]);
          done += kChunk;
        } while (!odd && done < stop);
      }
      if (odd) {
        done -= kChunk;
        walk_to = min(done + kChunk, stop);
      } else {
        done = stop;
        walk_to = ends ? r.n : stop;
      }
    }
    if (walk_to > done) walk(r.t0 + done, r.t0 + walk_to), done = walk_to;
    if (!odd) break;
    if (carries) {
      unsigned mine = 0;  // bit 16 m + n: column n of m, as far as this wave's rows go
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        bool any = false;
#pragma unroll
        for (int e = 0; e < HT; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) any = any || !(fabsf(s[e][m][j]) < INFINITY);
        const uint64_t b = __ballot(any);
        mine |= ((unsigned)(b | b >> 16 | b >> 32 | b >> 48) & 0xFFFFu) << 16 * m;
      }
      if (lane == 0) odds[wave] = mine;
    }
    lds_barrier();
    if (carries) {
      const unsigned lost = __builtin_amdgcn_readfirstlane(odds[0] | odds[1] | odds[2] | odds[3]);
#pragma unroll
      for (int m = 0; m < 2; ++m) seen[m] = ~(uint64_t(0x0001000100010001) * (lost >> 16 * m & 0xFFFFu));
    }
  }

  if (!carries || (ends && (!kept || (r.n == 0 && a.state_out == a.state)))) return;
  float* dst = ends ? a.state_out + state_at : carry;
#pragma unroll
  for (int e = 0; e < HT; ++e)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[(row_of(e) + j) * a.dv + col + 16 * m + n] = s[e][m][j];
}

// ---- host ----------------------------------------------------------------------------------------------------------

int64_t unit_bytes(int k_heads, int v_heads, int dk, int tk, int ot) {
  return (int64_t)k_heads * key_frags(dk, tk) * kFragBytes + (int64_t)v_heads * (tri_frags(3 + ot) * kFragBytes + kScalarBytes);
}
int64_t longest(int64_t tokens, int64_t max_len) { return max_len > 0 ? std::min(max_len, tokens) : tokens; }

template <typename IN, typename O, int DK>
void launch_walk(const ChunkParams& p, hipStream_t s) {
  const int group = p.a.v_heads / p.a.k_heads, slices = p.a.dv / 32;
  const int64_t heads = (int64_t)p.nseq * p.a.v_heads, together = (int64_t)p.nseq * p.a.k_heads >= 8 ? group : 1;
  const int64_t blocks = (heads / together + 7) / 8 * 8 * together * slices;
  hipLaunchKernelGGL((gdn_walk_kernel<IN, O, DK>), dim3((unsigned)blocks), dim3(kWalkThreads), 0, s, p);
}

template <typename IN, typename O, int DK>
hipError_t launch_all(const tq_gdn_args& a, hipStream_t s) {
  constexpr int OT = sizeof(O) == 4 ? 3 : 2;
  ChunkParams p{a};
  p.unit_bytes = unit_bytes(a.k_heads, a.v_heads, DK, terms_in<IN>(), OT);
  p.units = static_cast<uint8_t*>(a.workspace);
  auto run = [&]() {
    const int group = a.v_heads / a.k_heads;
    // A key head's value heads in one workgroup where those fill the card twice (16 key and 48 value heads, one sequence, bf16
    // and fp32, one head each against three: 64 tokens 16.5, 23.2 against 22.0, 28.3 us; 1024 54.2, 85.3 against 55.7, 80.7;
    // 4096 184, 382 against 179, 371)
    p.heads = p.slots * a.k_heads >= 512 ? group : 1;
    hipLaunchKernelGGL((gdn_prepare_kernel<IN, DK, OT>), dim3((unsigned)(p.slots * (a.v_heads / p.heads))), dim3(kPrepThreads), 0, s, p);
    launch_walk<IN, O, DK>(p, s);
    return hipGetLastError();
  };
  const int64_t all = a.tokens / kChunk + a.seqs;
  if (all * p.unit_bytes <= a.workspace_bytes) {
    p.whole = 1, p.last = 1, p.slots = all, p.nseq = (int)a.seqs, p.chunks = 1 << 24;
    return run();
  }
  // In groups of sequences and, within a group, in runs of chunks: at least 16 at a time if one sequence's fit
  const int64_t state = (int64_t)a.v_heads * DK * a.dv * 4;
  const int64_t need = (longest(a.tokens, a.max_len) + kChunk - 1) / kChunk;
  const int64_t nseq = std::max<int64_t>(1, std::min(a.seqs, a.workspace_bytes / (std::min<int64_t>(16, need) * p.unit_bytes + state)));
  p.chunks = (int)std::min(need, (a.workspace_bytes / nseq - state) / p.unit_bytes);
  p.carry = reinterpret_cast<float*>(p.units + nseq * p.chunks * p.unit_bytes);
  for (p.seq0 = 0; p.seq0 < a.seqs; p.seq0 += nseq) {
    p.nseq = (int)std::min(nseq, a.seqs - p.seq0);
    p.slots = (int64_t)p.nseq * p.chunks;
    for (int64_t c = 0; c < need; c += p.chunks) {
      p.chunk0 = (int)c, p.last = c + p.chunks >= need;
      const hipError_t e = run();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

template <typename IN, typename O>
hipError_t launch_dk(const tq_gdn_args& a, hipStream_t s) {
  return a.dk == 64 ? launch_all<IN, O, 64>(a, s) : launch_all<IN, O, 128>(a, s);
}

}  // namespace

bool gdn_chunked(int64_t tokens, int64_t seqs, int64_t max_len) {
  return longest(tokens, max_len) >= kStepLen && tokens > seqs;
}

// Room for one launch, or kBudget; one chunk and one state at least, whatever the types and key heads.
int64_t gdn_chunk_workspace_bytes(int64_t tokens, int64_t seqs, int64_t, int v_heads, int dk, int dv) {
  const int64_t unit = unit_bytes(v_heads, v_heads, dk, 3, 3);
  const int64_t least = unit + (int64_t)v_heads * dk * dv * 4;
  return std::max(least, std::min((tokens / kChunk + seqs) * unit, kBudget));
}

hipError_t launch_gdn_chunk(const tq_gdn_args& a, hipStream_t s) {
  switch (a.in_type) {
    case TQ_F32: return launch_dk<float, float>(a, s);
    case TQ_BF16: return a.out_type == TQ_F32 ? launch_dk<bf16, float>(a, s) : launch_dk<bf16, bf16>(a, s);
    default: return a.out_type == TQ_F32 ? launch_dk<f16, float>(a, s) : launch_dk<f16, f16>(a, s);
  }
}

}  // namespace tq
