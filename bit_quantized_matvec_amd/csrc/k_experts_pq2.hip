// k_experts_pq2.hip -- ternary products whose matrix is chosen per pair (token,
// place): repacked pq2_0 matrices of all experts x q8_K, on int8 MFMA.
//
// The arithmetic of each pair is the matrix-vector product's (k_gemv_pq2.hip)
// bit for bit: wave w of a workgroup sums run w of its superchunks, in fp64,
// and the runs are added in order.  A workgroup takes a tile of 16 pairs (32
// where experts have many) of one expert and a range of that expert's 16-row
// blocks; operands and layouts are those of the prompt product
// (k_gemm_pq2.hip), with each lane reading its pair's activations at an address
// of its own.
//
// Few pairs: bound by the codes.  One token's 8 experts of 2048 x 5120 take 8.6
// us (22 MB, 4.3 at a large copy's rate, one launch 3.6), 48 tokens x 8 of 64
// experts of 5120 x 1024 29 us (89 MB of codes, 19 at that rate).  Many pairs:
// bound by the vector units, see below.
//
// Slots and tiles: lists.h.  Workgroups of slots without a tile end at once;
// pairs without an expert get zeros.
#include <algorithm>

#include "batch.h"
#include "kernels.h"
#include "lists.h"
#include "pq2_mfma.h"
#include "seq.h"

namespace tq {
namespace {

constexpr int kMaxRuns = 4;  // waves per workgroup: the matrix-vector plan's runs
constexpr int kTok = 16;     // pairs of a tile

struct ExpertShape {
  int nrg;    // row ranges per tile of pairs
  int base;   // 16-row blocks per range: base, the first `extra` ranges one more
  int extra;
};

// A range's blocks are taken MRB at a time; the superchunks of all of them are one stream, RD of which are asked for ahead.
//
// Workgroups go to the XCDs in turn (id modulo 8): each XCD takes every eighth row range of all slots, so that what is read once is
// spread evenly, however the pairs are spread over the experts.
template <int RD, int MRB, bool LOOP>
__global__ __launch_bounds__(64 * kMaxRuns, 2) void gemm_experts_kernel(tq_gemm_experts_args g, int64_t expert_bytes, int nsc, int spw,
                                                                        int slots, int slot0, bool places, ExpertShape gs) {
  constexpr int kAcc = MRB * 4;
  extern __shared__ double sums[];
  __shared__ int pair_of[kTok];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), nruns = blockDim.x >> 6;
  const int l16 = lane & 15, qd = lane >> 4;
  const int id = blockIdx.x, rem = id % (8 * slots);
  const int rg = id / (8 * slots) * 8 + rem % 8, local = rem / 8;
  const int pairs = (int)g.pairs, rows = (int)g.rows;
  check_offsets(g.offsets, g.experts, pairs, g.bad_flag);
  if (rg >= gs.nrg || local >= slots) return;
  const int slot = slot0 + local;
  const Tile tile = find_tile(g.offsets, g.experts, pairs, kTok, places, slot, lane);
  if (tile.count == 0) return;  // uniform over the workgroup
  const int b0 = rg * gs.base + min(rg, gs.extra), blocks = gs.base + (rg < gs.extra ? 1 : 0);
  if (tid < kTok) {
    int p = tid < tile.count ? g.order[tile.first + tid] : -1;
    if (tid < tile.count && (p < 0 || p >= pairs)) {
      raise_flag(g.bad_flag);
      p = -1;
    }
    pair_of[tid] = p;
  }
  __syncthreads();
  if (tile.expert == g.experts) {  // no expert: zeros
    const int r0 = b0 * 16, nr = min(rows, (b0 + blocks) * 16) - r0;
    for (int i = tid; i < nr * kTok; i += blockDim.x) {
      const int p = pair_of[i / nr];
      if (p >= 0) g.y[(int64_t)p * rows + r0 + i % nr] = 0.0f;
    }
    return;
  }

  const int K = nsc * 256;
  const int sc0 = wave * spw, n = min(nsc, sc0 + spw) - sc0;  // this wave's run, at least 1
  constexpr int kUnit = (int)kPq2UnitBytes;
  const int tile0 = b0 >> 2, ntl = min((blocks + 6) / 4, (rows + 63) / 64 - tile0);  // 64-row tiles of this range
  const uint8_t* units = static_cast<const uint8_t*>(g.w) + tile.expert * expert_bytes + (int64_t)tile0 * nsc * kUnit;
  const buf_t none = make_buf(units, 0);
  const buf_t a_buf = make_buf(units, ntl * nsc * kUnit);
  const buf_t s_buf = make_buf(units + kPq2ScaleOffset, ntl * nsc * kUnit - (int)kPq2ScaleOffset);
  const int a_lane = (64 * qd + l16) * 16, s_lane = 4 * l16;
  // Token t of a block of 16 sits in MFMA row 4 (t % 4) + t / 4.  Places without a pair read the first input and are not stored.
  const int trow = 4 * (l16 & 3) + (l16 >> 2);
  const int share = (int)(g.pairs / g.inputs);
  const int8_t* qp = g.q + (int64_t)(max(0, pair_of[trow]) / share) * K + 16 * qd + 256 * sc0;
  const float* dp = g.d + (int64_t)(max(0, pair_of[l16]) / share) * nsc + sc0;

  v4u ra[RD][MRB];
  uint32_t rs[RD][MRB];
  v4u rb[RD][4];
  float rx[RD];
  const int groups = (blocks + MRB - 1) / MRB;
  int ahead_group = 0, ahead_k = 0;  // what is asked for next
  const bool keep = n == 1;          // one superchunk: its activations stay
  // Asks for the next superchunk of the stream, into slot J.  Past the end, and blocks past the range, nothing is read.
  auto fetch = [&](int J, bool acts) __attribute__((always_inline)) {
    const bool real = ahead_group < groups;
    const int sc = sc0 + ahead_k, first = ahead_group * MRB;
    if (acts) {
#pragma unroll
      for (int c = 0; c < 4; ++c) rb[J][c] = *reinterpret_cast<const v4u*>(qp + 256 * ahead_k + 64 * c);
      rx[J] = dp[ahead_k];
    }
#pragma unroll
    for (int i = 0; i < MRB; ++i) {
      const bool use = real && first + i < blocks;
      const int b = b0 + first + i, at = ((b >> 2) - tile0) * nsc * kUnit + kUnit * sc;
      ra[J][i] = load16(use ? a_buf : none, a_lane, at + 16 * (b & 3) * 16);
      rs[J][i] = load4(use ? s_buf : none, s_lane, at + 16 * (b & 3) * 4);
    }
    if (++ahead_k == n) ahead_k = 0, ++ahead_group;
  };
  double yacc[MRB][4];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MRB; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) yacc[i][v] = 0.0;
  };
  const int slots_used = (tile.count + 3) / 4;  // result slot v of a lane holds token 4 v + qd
  int nrb = min(MRB, blocks);                   // blocks of the present group

  auto step = [&](int J) __attribute__((always_inline)) {
    double xd[4];
    const int xi = __builtin_bit_cast(int, rx[J]);
#pragma unroll
    for (int v = 0; v < 4; ++v) xd[v] = (double)__builtin_bit_cast(float, __shfl(xi, 4 * v + qd, 64)) * 0.015625;
#pragma unroll
    for (int i = 0; i < MRB; ++i) {
      if (i >= nrb) continue;
      v4i acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const v4i w = expand64(ra[J][i][c]);
        acc[c >> 1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, rb[J][c]), w, acc[c >> 1], 0, 0, 0);
      }
      const double d0 = lo_half(rs[J][i]), d1 = hi_half(rs[J][i]);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (v >= slots_used) continue;  // uniform
        const double inner = __builtin_fma(d1, (double)acc[1][v], d0 * (double)acc[0][v]);
        yacc[i][v] = __builtin_fma(xd[v], inner, yacc[i][v]);
      }
    }
  };

  // The runs of a group added in run order.
  auto finish = [&](int group) __attribute__((always_inline)) {
    if (group > 0) __syncthreads();  // the sums before are read
#pragma unroll
    for (int i = 0; i < MRB; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (v < slots_used) sums[((size_t)wave * kAcc + 4 * i + v) * 64 + lane] = yacc[i][v];
    __syncthreads();
    for (int sl = wave; sl < kAcc; sl += nruns) {
      const int i = sl / 4, v = sl % 4;
      if (i >= nrb || v >= slots_used) continue;
      double rv[kMaxRuns];
#pragma unroll
      for (int w = 0; w < kMaxRuns; ++w) rv[w] = sums[((size_t)min(w, nruns - 1) * kAcc + sl) * 64 + lane];
      double t = rv[0];
#pragma unroll
      for (int w = 1; w < kMaxRuns; ++w)
        if (w < nruns) t += rv[w];
      const int row = (b0 + group * MRB + i) * 16 + l16, pr = pair_of[4 * v + qd];
      if (row < rows && pr >= 0) g.y[(int64_t)pr * rows + row] = (float)t;
    }
  };

  if constexpr (LOOP) {
    static_assert(RD == 1, "conditions between the steps would drain a longer ring at every join");
    fetch(0, true);
    for (int group = 0; group < groups; ++group) {
      nrb = min(MRB, blocks - group * MRB);
      clear();
      for (int k = 0; k < n; ++k) {
        step(0);
        fetch(0, !keep);
      }
      finish(group);
    }
  } else {
    // one group.  No step inside the loop is conditional, so that the compiler's wait counts stay per slot of the ring.
    clear();
#pragma unroll
    for (int J = 0; J < RD; ++J) fetch(J, true);
    const int full = n / RD;
    for (int c = 0; c < full; ++c) {
#pragma unroll
      for (int J = 0; J < RD; ++J) {
        step(J);
        fetch(J, true);
      }
    }
#pragma unroll
    for (int J = 0; J + 1 < RD; ++J)
      if (J < n - full * RD) step(J);
    finish(0);
  }
}

template <int RD, int MRB, bool LOOP>
hipError_t launch_t(const tq_gemm_experts_args& g, int64_t active, int64_t work, hipStream_t s) {
  const Dims dm = dims(g.rows, g.cols);
  const int64_t expert_bytes = pq2_code_bytes(dm) + pq2_scale_bytes(dm);
  ExpertShape gs;
  const Slots slots = list_slots(g.pairs, g.experts, kTok);
  // Row ranges: about `work` workgroups with a tile, at most 64 blocks each (a range's codes stay within a buffer's 2^31 bytes)
  const int64_t nblk = 4 * dm.ntiles;
  const int64_t most_blocks = LOOP ? 64 : MRB;
  const int64_t want = std::max((nblk + most_blocks - 1) / most_blocks, std::min(nblk, (work + active - 1) / active));
  gs.nrg = (int)want;
  gs.base = (int)(nblk / want), gs.extra = (int)(nblk % want);
  const GemvPlan p = plan_gemv_pq2(dm, false);  // the runs of the matrix-vector product
  const int nruns = (int)((dm.nsc + p.spw - 1) / p.spw);
  const size_t lds = (size_t)nruns * MRB * 4 * 64 * 8;
  // at most 2^22 workgroups per launch, as in the prompt product
  const int64_t most = std::max<int64_t>(8, (int64_t(1) << 22) / gs.nrg / 8 * 8);
  for (int64_t s0 = 0; s0 < slots.count; s0 += most) {
    const int64_t now = std::min(most, slots.count - s0);
    const int64_t grid = (gs.nrg + 7) / 8 * 8 * now;
    hipLaunchKernelGGL((gemm_experts_kernel<RD, MRB, LOOP>), dim3((unsigned)grid), dim3(64 * nruns), lds, s, g, expert_bytes, (int)dm.nsc, p.spw, (int)now,
                       (int)s0, slots.places, gs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- many pairs of one expert ----
//
// A workgroup's four waves take up to 256 rows (kWideBlocks 16-row blocks each) and the same 32 pairs, so that these pairs'
// activations come from memory once for 256 rows: with a wave per run of columns (the kernel above) they come once for 48.
// Superchunk after superchunk the activations are staged in LDS in the order of the matrix instructions' operands, one ahead of the
// products; a wave's codes are asked for one superchunk ahead in registers.  A wave goes through all runs of the matrix-vector
// product in turn; the sum of those before waits in LDS.  An XCD takes an eighth of the slots, one after the other, each with all
// its row ranges: the ranges of a tile share its activations in that XCD's L2, and neighbouring tiles, mostly of one expert, its codes.
//
// Bound by the vector units: per 16 rows, 32 pairs and superchunk 28 instructions expand the codes, 40 make the fp64 sums (5 to 6
// cycles each with two waves per SIMD), and 8 matrix instructions of 16 cycles run beside them.  2048 tokens x 4 of 32 experts of
// 2048 x 5120: 191 to 207 us, vector units 56 % and matrix units 20 % busy.  (Eight waves of 2 blocks, four per SIMD: 216, more reads of
// the staged operands and 4 spilled registers; eight waves of 4 blocks, one workgroup per compute unit: 206.)
constexpr int kWideWaves = 4;
constexpr int kPieces = 8 / kWideWaves;  // 16-byte pieces of a superchunk that a thread stages
constexpr int kWideBlocks = 4;
constexpr int kWideTok = 32;
constexpr int kWideStage = 8 * 1024;  // bytes of a superchunk of 32 pairs

// BLOCKS: 16-row blocks of a wave (missing ones read zeros: without branches one block's sums hide another's matrix instructions).
template <int BLOCKS>
__global__ __launch_bounds__(64 * kWideWaves, 2) void gemm_experts_wide_kernel(tq_gemm_experts_args g, int64_t expert_bytes, int nsc, int spw, int slots,
                                                                               int slot0, bool places, ExpertShape gs) {
  // [2][kWideStage] activations, [2][32] d_x / 64, then the sums of the runs before, [block][pair block][4][thread]
  extern __shared__ double lds[];
  __shared__ int pair_of[kWideTok];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, qd = lane >> 4;
  const int at = blockIdx.x / 8, share = (slots + 7) / 8;
  const int rg = at % gs.nrg, local = blockIdx.x % 8 * share + at / gs.nrg;
  const int pairs = (int)g.pairs, rows = (int)g.rows;
  check_offsets(g.offsets, g.experts, pairs, g.bad_flag);
  if (local >= slots || at / gs.nrg >= share) return;
  const Tile tile = find_tile(g.offsets, g.experts, pairs, kWideTok, places, slot0 + local, lane);
  if (tile.count == 0) return;  // uniform over the workgroup
  const int r0 = rg * gs.base + min(rg, gs.extra), blocks = gs.base + (rg < gs.extra ? 1 : 0);
  if (tid < kWideTok) {
    int p = tid < tile.count ? g.order[tile.first + tid] : -1;
    if (tid < tile.count && (p < 0 || p >= pairs)) {
      raise_flag(g.bad_flag);
      p = -1;
    }
    pair_of[tid] = p;
  }
  __syncthreads();
  if (tile.expert == g.experts) {  // no expert: zeros
    const int first = r0 * 16, nr = min(rows, (r0 + blocks) * 16) - first;
    for (int i = tid; i < nr * kWideTok; i += blockDim.x) {
      const int p = pair_of[i / nr];
      if (p >= 0) g.y[(int64_t)p * rows + first + i % nr] = 0.0f;
    }
    return;
  }

  constexpr int kUnit = (int)kPq2UnitBytes;
  const int b0 = r0 + wave * BLOCKS, nb = max(0, min(BLOCKS, blocks - wave * BLOCKS));
  const int tile0 = b0 >> 2, ntl = max(0, min((BLOCKS + 6) / 4, (rows + 63) / 64 - tile0));
  const uint8_t* units = static_cast<const uint8_t*>(g.w) + tile.expert * expert_bytes + (nb > 0 ? (int64_t)tile0 * nsc * kUnit : 0);
  const buf_t none = make_buf(units, 0);
  const buf_t a_buf = nb > 0 ? make_buf(units, ntl * nsc * kUnit) : none;
  const buf_t s_buf = nb > 0 ? make_buf(units + kPq2ScaleOffset, ntl * nsc * kUnit - (int)kPq2ScaleOffset) : none;
  const int a_lane = (64 * qd + l16) * 16, s_lane = 4 * l16;
  const int per_input = (int)(g.pairs / g.inputs);

  // Staging: thread (token, piece) has bytes 16 piece .. + 15 of its token's superchunk, which lane 16 (piece % 4) + row of the
  // operand (token / 16, piece / 4) takes; token t of a block of 16 sits in row 4 (t % 4) + t / 4.
  const int piece = tid & 15;
  const int8_t* q_from[kPieces];
  int q_to[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int st = (tid >> 4) + 4 * kWideWaves * p;
    q_from[p] = g.q + (int64_t)(max(0, pair_of[st]) / per_input) * nsc * 256 + 16 * piece;
    q_to[p] = ((st >> 4) * 4 + (piece >> 2)) * 1024 + (16 * (piece & 3) + 4 * (st & 3) + ((st & 15) >> 2)) * 16;
  }
  const float* d_from = g.d + (int64_t)(max(0, pair_of[tid & 31]) / per_input) * nsc;
  uint8_t* stage = reinterpret_cast<uint8_t*>(lds);
  double* scale = lds + 2 * kWideStage / 8;
  double* before = scale + 2 * kWideTok;

  constexpr int kAhead = 4;                      // activations are asked for so many superchunks before they are staged
  constexpr int kCodes = 2;                      // and codes one superchunk before they are used
  v4u ra[kCodes][BLOCKS], q_ring[kAhead][kPieces];
  uint32_t rs[kCodes][BLOCKS];
  float d_ring[kAhead];
  const auto ask_codes = [&](int J, int sc) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
      const bool use = i < nb && sc < nsc;
      const int b = b0 + i, o = ((b >> 2) - tile0) * nsc * kUnit + kUnit * sc;
      ra[J][i] = load16(use ? a_buf : none, a_lane, o + 16 * (b & 3) * 16);
      rs[J][i] = load4(use ? s_buf : none, s_lane, o + 16 * (b & 3) * 4);
    }
  };
  const auto ask_acts = [&](int J, int sc) __attribute__((always_inline)) {
    const int s = min(sc, nsc - 1);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) q_ring[J][p] = *reinterpret_cast<const v4u*>(q_from[p] + 256 * s);
    d_ring[J] = sc < nsc ? d_from[s] : 0.0f;  // (behind the last zero: 0 times its scale would be NaN where that is not finite)
  };
  const auto put_acts = [&](int J, int to) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) *reinterpret_cast<v4u*>(stage + to * kWideStage + q_to[p]) = q_ring[J][p];
    if (tid < kWideTok) scale[to * kWideTok + tid] = (double)d_ring[J] * 0.015625;
  };

  double acc[BLOCKS][2][4];
  double before_last = 0;  // the last sum's, in a register: the others' place in LDS is all that two workgroups leave each other
  const auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][t][v] = 0.0;
  };
  clear();
#pragma unroll
  for (int J = 0; J < kAhead; ++J) ask_acts(J, J);
#pragma unroll
  for (int J = 0; J + 1 < kCodes; ++J) ask_codes(J, J);
  put_acts(0, 0);
  ask_acts(0, kAhead);
  __syncthreads();
  int run = 0, k = 0;
  // Four superchunks a pass; those behind the last have no codes and add zeros.
  for (int s0 = 0; s0 < nsc; s0 += kAhead) {
#pragma unroll
    for (int J = 0; J < kAhead; ++J) {
      const int sc = s0 + J;
      ask_codes((J + kCodes - 1) % kCodes, sc + kCodes - 1);
      put_acts((J + 1) % kAhead, (J + 1) & 1);
      ask_acts((J + 1) % kAhead, sc + 1 + kAhead);
      v4i b[2][4];
      double xd[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) b[t][c] = *reinterpret_cast<const v4i*>(stage + (J & 1) * kWideStage + (t * 4 + c) * 1024 + lane * 16);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) xd[t][v] = scale[(J & 1) * kWideTok + 16 * t + 4 * v + qd];
#pragma unroll
      for (int i = 0; i < BLOCKS; ++i) {
        v4i m[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) m[t][0] = m[t][1] = v4i{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const v4i w = expand64(ra[J % kCodes][i][c]);
#pragma unroll
          for (int t = 0; t < 2; ++t) m[t][c >> 1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[t][c], w, m[t][c >> 1], 0, 0, 0);
        }
        const double d0 = lo_half(rs[J % kCodes][i]), d1 = hi_half(rs[J % kCodes][i]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const double inner = __builtin_fma(d1, (double)m[t][1][v], d0 * (double)m[t][0][v]);
            acc[i][t][v] = __builtin_fma(xd[t][v], inner, acc[i][t][v]);
          }
      }
      __syncthreads();
      if (++k == spw && sc + 1 < nsc) {  // the run's end: runs are added in order, ((s0 + s1) + s2) + s3
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              double* p = before + ((i * 2 + t) * 4 + v) * (64 * kWideWaves) + tid;
              const bool kept = (i * 2 + t) * 4 + v == BLOCKS * 8 - 1;
              const double was = kept ? before_last : *p;  // (before the first run's end not used)
              const double sum = run ? was + acc[i][t][v] : acc[i][t][v];
              if (kept)
                before_last = sum;
              else
                *p = sum;
            }
        clear();
        k = 0, ++run;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < BLOCKS; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const bool kept = (i * 2 + t) * 4 + v == BLOCKS * 8 - 1;
        const double was = kept ? before_last : before[((i * 2 + t) * 4 + v) * (64 * kWideWaves) + tid];
        const double sum = run ? was + acc[i][t][v] : acc[i][t][v];
        const int row = (b0 + i) * 16 + l16, pr = pair_of[16 * t + 4 * v + qd];
        if (i < nb && row < rows && pr >= 0) g.y[(int64_t)pr * rows + row] = (float)sum;
      }
}

hipError_t launch_wide(const tq_gemm_experts_args& g, hipStream_t s) {
  const Dims dm = dims(g.rows, g.cols);
  const int64_t expert_bytes = pq2_code_bytes(dm) + pq2_scale_bytes(dm);
  const Slots slots = list_slots(g.pairs, g.experts, kWideTok);
  ExpertShape gs;
  const int64_t nblk = (dm.rows + 15) / 16;
  gs.nrg = (int)((nblk + kWideWaves * kWideBlocks - 1) / (kWideWaves * kWideBlocks));
  gs.base = (int)(nblk / gs.nrg), gs.extra = (int)(nblk % gs.nrg);
  const GemvPlan p = plan_gemv_pq2(dm, false);
  const int each = (int)((gs.base + (gs.extra > 0) + kWideWaves - 1) / kWideWaves);
  const size_t lds = 2 * kWideStage + 2 * kWideTok * 8 + ((size_t)each * 8 - 1) * 64 * kWideWaves * 8;
  const auto kernel = each == 1 ? gemm_experts_wide_kernel<1> : each == 2 ? gemm_experts_wide_kernel<2> : each == 3 ? gemm_experts_wide_kernel<3> : gemm_experts_wide_kernel<4>;
  const int64_t most = std::max<int64_t>(8, (int64_t(1) << 21) / gs.nrg / 8 * 8);  // workgroups per launch, as above
  for (int64_t s0 = 0; s0 < slots.count; s0 += most) {
    const int64_t now = std::min(most, slots.count - s0);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((now + 7) / 8 * 8 * gs.nrg)), dim3(64 * kWideWaves), lds, s, g, expert_bytes, (int)dm.nsc,
                       p.spw, (int)now, (int)s0, slots.places, gs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_gemm_experts_pq2(const tq_gemm_experts_args& g, hipStream_t s) {
  const int64_t active = std::min<int64_t>(g.experts, g.pairs);
  const int64_t work = (g.rows + 15) / 16 * active;  // 16-row blocks of the experts that can have a pair
  // Many pairs per expert.  wide / up to 48 rows per workgroup, us: 32 pairs per expert of 2048 x 5120 68 / 58, of 2048 x 2048 27 / 22;
  // 48 pairs 71 / 83; 64 pairs 28 / 36 (2048 x 2048); 256 pairs 187 / 341, of 192 x 5120 41 / 108, of 128 x 1024 13 / 23.
  if (g.pairs > 40 * active) return launch_wide(g, s);
  // A workgroup for several groups of 48 rows, which the tile's activations and its start are shared by, where there are many
  // blocks or each run is one superchunk.  Several / one, us: 20480 blocks 30 / 45 (1024 columns), 50 / 67 (2048); 8192 blocks
  // 16 / 22 (1024), 46 / 48 (5120); 4096 blocks 55 / 44 (5120); 2048 blocks 8.6 / 9.6 (1024), 17 / 15 (2048).
  if (work > (g.cols <= 256 * kMaxRuns ? 1536 : 6144)) return launch_t<1, 3, true>(g, active, 1024, s);
  return launch_t<2, 3, false>(g, active, 512, s);
}

}  // namespace tq
