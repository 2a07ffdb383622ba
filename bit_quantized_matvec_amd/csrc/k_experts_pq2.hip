// k_experts_pq2.hip -- ternary products whose matrix is chosen per pair (token,
// place): repacked pq2_0 matrices of all experts x q8_K, on int8 MFMA.
//
// The arithmetic of each pair is the matrix-vector product's (k_gemv_pq2.hip)
// bit for bit: wave w of a workgroup sums run w of its superchunks, in fp64,
// and the runs are added in order.  A workgroup takes a tile of 16 NT pairs of
// one expert and a range of that expert's 16-row blocks; operands and layouts
// are those of the prompt product (k_gemm_pq2.hip), with each lane reading its
// pair's activations at an address of its own.
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

struct ExpertShape {
  int nrg;    // row ranges per tile, a multiple of 8 with padding
  int nreal;  // real ones
  int base;   // blocks per range: base, the first `extra` ranges one more
  int extra;
};

// Workgroup id = ((rg / 8) * slots + slot) * 8 + rg % 8: the tiles of one row range run on one XCD, so that the tiles of an
// expert share its codes in that XCD's L2.
template <int NT, int RD, int MRB>
__global__ __launch_bounds__(64 * kMaxRuns, 2) void gemm_experts_kernel(tq_gemm_experts_args g, int64_t expert_bytes, int nsc, int spw, int slots, int slot0, bool places,
                                                                        ExpertShape gs) {
  constexpr int kTok = 16 * NT;
  constexpr int kAcc = MRB * NT * 4;
  extern __shared__ double sums[];
  __shared__ int pair_of[kTok];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), nruns = blockDim.x >> 6;
  const int l16 = lane & 15, qd = lane >> 4;
  const int id = blockIdx.x, grp = id / (8 * slots), rem = id % (8 * slots);
  const int rg = grp * 8 + rem % 8, slot = slot0 + rem / 8;
  if (rg >= gs.nreal) return;
  const int pairs = (int)g.pairs, rows = (int)g.rows;
  const Tile tile = find_tile(g.offsets, g.experts, pairs, kTok, places, slot, lane, g.bad_flag);
  if (tile.count == 0) return;  // uniform over the workgroup
  const int b0 = rg * gs.base + min(rg, gs.extra), nrb = gs.base + (rg < gs.extra ? 1 : 0);
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
    const int r0 = b0 * 16, nr = min(rows, (b0 + nrb) * 16) - r0;
    for (int i = tid; i < nr * kTok; i += blockDim.x) {
      const int p = pair_of[i / nr];
      if (p >= 0) g.y[(int64_t)p * rows + r0 + i % nr] = 0.0f;
    }
    return;
  }

  const int K = nsc * 256;
  const int sc0 = wave * spw, n = min(nsc, sc0 + spw) - sc0;  // this wave's run, at least 1
  constexpr int kUnit = (int)kPq2UnitBytes;
  const int tile0 = b0 >> 2, ntl = min((MRB + 6) / 4, (rows + 63) / 64 - tile0);  // 64-row tiles of this range
  const uint8_t* units = static_cast<const uint8_t*>(g.w) + tile.expert * expert_bytes + (int64_t)tile0 * nsc * kUnit;
  const buf_t none = make_buf(units, 0);
  const buf_t a_buf = make_buf(units, ntl * nsc * kUnit);
  const buf_t s_buf = make_buf(units + kPq2ScaleOffset, ntl * nsc * kUnit - (int)kPq2ScaleOffset);
  int a_off[MRB], s_off[MRB];
#pragma unroll
  for (int i = 0; i < MRB; ++i) {
    const int b = b0 + i, tl = (b >> 2) - tile0, rbi = b & 3;
    a_off[i] = tl * nsc * kUnit + 16 * rbi * 16;
    s_off[i] = tl * nsc * kUnit + 16 * rbi * 4;
  }
  const int a_lane = (64 * qd + l16) * 16, s_lane = 4 * l16;
  // Token t of a block of 16 sits in MFMA row 4 (t % 4) + t / 4.  Places without a pair read the first input and are not stored.
  const int trow = 4 * (l16 & 3) + (l16 >> 2);
  const int share = (int)(g.pairs / g.inputs);
  const int8_t* qp[NT];
#pragma unroll
  for (int nb = 0; nb < NT; ++nb) qp[nb] = g.q + (int64_t)(max(0, pair_of[16 * nb + trow]) / share) * K + 16 * qd + 256 * sc0;
  const float* dp = g.d + (int64_t)(max(0, pair_of[lane & (kTok - 1)]) / share) * nsc + sc0;

  v4u ra[RD][MRB];
  uint32_t rs[RD][MRB];
  v4u rb[NT][4];
  float rx;
  auto codes = [&](int J, int k) __attribute__((always_inline)) {
    const bool real = k < n;
#pragma unroll
    for (int i = 0; i < MRB; ++i) {
      const bool use = real && i < nrb;
      ra[J][i] = load16(use ? a_buf : none, a_lane, a_off[i] + kUnit * (sc0 + k));
      rs[J][i] = load4(use ? s_buf : none, s_lane, s_off[i] + kUnit * (sc0 + k));
    }
  };
  auto acts = [&](int k) __attribute__((always_inline)) {
    const int kk = min(k, n - 1);
#pragma unroll
    for (int nb = 0; nb < NT; ++nb)
#pragma unroll
      for (int c = 0; c < 4; ++c) rb[nb][c] = *reinterpret_cast<const v4u*>(qp[nb] + 256 * kk + 64 * c);
    rx = dp[kk];
  };
  double yacc[MRB][NT][4];
#pragma unroll
  for (int i = 0; i < MRB; ++i)
#pragma unroll
    for (int nb = 0; nb < NT; ++nb)
#pragma unroll
      for (int v = 0; v < 4; ++v) yacc[i][nb][v] = 0.0;
  const int slots_used = NT == 1 ? (tile.count + 3) / 4 : 4;  // result slot v of a lane holds token 4 v + qd

  auto step = [&](int J) __attribute__((always_inline)) {
    double xd[NT][4];
    const int xi = __builtin_bit_cast(int, rx);
#pragma unroll
    for (int nb = 0; nb < NT; ++nb)
#pragma unroll
      for (int v = 0; v < 4; ++v) xd[nb][v] = (double)__builtin_bit_cast(float, __shfl(xi, 16 * nb + 4 * v + qd, 64)) * 0.015625;
#pragma unroll
    for (int i = 0; i < MRB; ++i) {
      if (i >= nrb) continue;
      v4i acc[NT][2];
#pragma unroll
      for (int nb = 0; nb < NT; ++nb) acc[nb][0] = acc[nb][1] = v4i{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const v4i w = expand64(ra[J][i][c]);
#pragma unroll
        for (int nb = 0; nb < NT; ++nb)
          acc[nb][c >> 1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, rb[nb][c]), w, acc[nb][c >> 1], 0, 0, 0);
      }
      const double d0 = lo_half(rs[J][i]), d1 = hi_half(rs[J][i]);
#pragma unroll
      for (int nb = 0; nb < NT; ++nb)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (NT == 1 && v >= slots_used) continue;  // uniform
          const double inner = __builtin_fma(d1, (double)acc[nb][1][v], d0 * (double)acc[nb][0][v]);
          yacc[i][nb][v] = __builtin_fma(xd[nb][v], inner, yacc[i][nb][v]);
        }
    }
  };

  acts(0);
#pragma unroll
  for (int J = 0; J < RD; ++J) codes(J, J);
  const int full = n / RD;
  for (int c = 0; c < full; ++c) {
#pragma unroll
    for (int J = 0; J < RD; ++J) {
      step(J);
      acts(c * RD + J + 1);
      codes(J, c * RD + J + RD);
    }
  }
#pragma unroll
  for (int J = 0; J + 1 < RD; ++J)
    if (J < n - full * RD) {
      step(J);
      acts(full * RD + J + 1);
    }

  // runs added in run order; phases bound the LDS
  constexpr int kPh = kAcc > 20 ? 2 : 1, kPer = kAcc / kPh;
  static_assert(kAcc % kPh == 0, "phases split the slots evenly");
#pragma unroll
  for (int p = 0; p < kPh; ++p) {
    if (p > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < MRB; ++i)
#pragma unroll
      for (int nb = 0; nb < NT; ++nb)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int sl = (i * NT + nb) * 4 + v;
          if (sl / kPer == p) sums[((size_t)wave * kPer + sl % kPer) * 64 + lane] = yacc[i][nb][v];
        }
    __syncthreads();
    for (int sl = p * kPer + wave; sl < (p + 1) * kPer; sl += nruns) {
      const int i = sl / (NT * 4), nb = (sl / 4) % NT, v = sl % 4;
      if (i >= nrb) continue;
      double rv[kMaxRuns];
#pragma unroll
      for (int w = 0; w < kMaxRuns; ++w) rv[w] = sums[((size_t)min(w, nruns - 1) * kPer + sl % kPer) * 64 + lane];
      double t = rv[0];
#pragma unroll
      for (int w = 1; w < kMaxRuns; ++w)
        if (w < nruns) t += rv[w];
      const int row = (b0 + i) * 16 + l16, pr = pair_of[16 * nb + 4 * v + qd];
      if (row < rows && pr >= 0) g.y[(int64_t)pr * rows + row] = (float)t;
    }
  }
}

template <int NT, int RD, int MRB>
hipError_t launch_t(const tq_gemm_experts_args& g, int tiles, hipStream_t s) {
  const Dims dm = dims(g.rows, g.cols);
  const int64_t expert_bytes = pq2_code_bytes(dm) + pq2_scale_bytes(dm);
  const int size = 16 * NT;
  ExpertShape gs;
  const Slots slots = list_slots(g.pairs, g.experts, size);
  const int64_t nblk = 4 * dm.ntiles;
  const int64_t want = std::max((nblk + MRB - 1) / MRB, std::min<int64_t>(nblk, (512 + tiles - 1) / tiles));
  gs.nreal = (int)want;
  gs.base = (int)(nblk / want), gs.extra = (int)(nblk % want);
  gs.nrg = (int)((want + 7) / 8 * 8);
  const GemvPlan p = plan_gemv_pq2(dm, false);  // the runs of the matrix-vector product
  const int nruns = (int)((dm.nsc + p.spw - 1) / p.spw);
  constexpr int kAcc = MRB * NT * 4;
  const size_t lds = (size_t)nruns * (kAcc > 20 ? kAcc / 2 : kAcc) * 64 * 8;
  // at most 2^22 workgroups per launch, as in the prompt product
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 22) / gs.nrg);
  for (int64_t s0 = 0; s0 < slots.count; s0 += most) {
    const int64_t now = std::min(most, slots.count - s0);
    hipLaunchKernelGGL((gemm_experts_kernel<NT, RD, MRB>), dim3((unsigned)(gs.nrg * now)), dim3(64 * nruns), lds, s, g, expert_bytes, (int)dm.nsc, p.spw,
                       (int)now, (int)s0, slots.places, gs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_gemm_experts_pq2(const tq_gemm_experts_args& g, hipStream_t s) {
  const int64_t active = std::min<int64_t>(g.experts, g.pairs);
  if (g.pairs > 24 * active) return launch_t<2, 1, 5>(g, (int)std::min<int64_t>(1 << 20, g.pairs / 32 + active), s);
  return launch_t<1, 2, 3>(g, (int)active, s);
}

}  // namespace tq
