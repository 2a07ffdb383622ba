// k_route.hip -- the choice of experts for each token, and the pairs (token,
// place) sorted by expert.
//
// route: one wave per token.  Scores s and what is compared (c = s + bias) are
// fp64: 64 to 256 scores of a softmax differ by less than fp32 resolves often
// enough that a choice in fp32 differs from the definition's.  Without a bias,
// and where no two scores of a group are added, the order of c is the order of
// the logits, which are compared themselves (and exactly).  Comparable numbers
// are unsigned keys (ordered_key); an absent expert has key 0.
//   * k rounds: each lane's largest key, the wave's by DPP, the lowest expert
//     that has it (lanes hold experts lane + 64 j, so the lowest j, then the
//     lowest lane), which is then taken out.
//   * groups: c of all experts in LDS; lane g sums the group's largest; ranks
//     of groups by counting those worth more.
// Bound by latency for few tokens (one token of 64 experts 2.9 us), by
// instructions for many (an fp64 exponential and a division per score, some 50
// instructions per round): 4099 tokens of 256 experts with groups 13 us, vector
// units 67 % busy, 2 MB read.
//
// expert_lists: one workgroup per expert reads every id and writes that
// expert's pairs in their order: no atomics, so the lists do not depend on
// timing.  Each wave has a contiguous share of the pairs, counts those below
// and those of its expert, and, after one exchange, writes.  32792 pairs of 256
// experts 11 us, a chain of reads, an exchange and the reads again (with ids
// read one per lane and counted by ballots 22).
#include <algorithm>

#include "batch.h"
#include "lanes.h"
#include "seq.h"

namespace tq {
namespace {

constexpr int kWaves = 4;

template <typename T>
__device__ inline float load_f32(const T* p) {
  return (float)*p;
}

// Unsigned numbers in the order of the values, above 0; -0 counts as +0.
__device__ inline uint64_t ordered_key(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
  return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}
__device__ inline uint32_t ordered_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b >> 31 ? ~b : b | 0x80000000u;
}

// WIDE: keys of fp64 c; otherwise keys of the logits, in the high half.
template <typename T, int NJ, bool WIDE>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(tq_route_args a) {
  extern __shared__ double lds[];  // per wave: s[experts], then c[experts] with groups
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= a.tokens) return;  // whole waves; no barrier below
  const int n = a.experts;
  double* sl = lds + (size_t)wave * n * (a.groups > 1 ? 2 : 1);
  double* cl = sl + n;
  const T* row = static_cast<const T*>(a.logits) + t * a.logit_stride;

  float x[NJ];
  float most = -INFINITY;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 64 * j;
    x[j] = e < n ? load_f32(row + e) : -INFINITY;
    if (!(x[j] == x[j])) x[j] = -INFINITY;
    most = fmaxf(most, x[j]);
  }
  double s[NJ];
  if (a.score == TQ_SOFTMAX) {
    {  // (exact: the largest key's value)
      const uint32_t k = wave_max_u32(most > -INFINITY ? ordered_key(most) : 0u);
      most = k ? __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k) : -INFINITY;
    }
    double sum = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      s[j] = x[j] == -INFINITY ? 0.0 : x[j] == most ? 1.0 : exp((double)x[j] - (double)most);
      sum += s[j];
    }
    sum = wave_total(sum);
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] = sum > 0 ? s[j] / sum : 0.0;
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j] = x[j] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)x[j]));
  }
  uint64_t key[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + 64 * j;
    const bool there = e < n && x[j] > -INFINITY;
    double c = WIDE ? s[j] : (double)x[j];
    if (WIDE && a.bias && there) c += (double)a.bias[e];
    const bool takes_part = there && c > -INFINITY;
    key[j] = !takes_part ? 0 : WIDE ? ordered_key(c) : (uint64_t)ordered_key(x[j]) << 32;
    if (e < n) {
      sl[e] = s[j];
      if (a.groups > 1) cl[e] = takes_part ? c : -INFINITY;
    }
  }
  if (a.groups > 1) {
    const int size = n / a.groups;
    double v = -INFINITY;
    if (lane < a.groups) {
      double first = -INFINITY, second = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const double c = cl[lane * size + i];
        second = fmax(second, fmin(first, c));
        first = fmax(first, c);
      }
      v = a.group_best == 2 ? first + second : first;
      if (!(v == v)) v = -INFINITY;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(v, g, 64);
      rank += o > v || (o == v && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + 64 * j;
      if (e < n && !(kept >> (e / size) & 1)) key[j] = 0;
    }
  }

  int mine = -1;  // lane i: the i-th chosen
  for (int i = 0; i < a.k; ++i) {
    uint64_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < NJ; ++j)
      if (key[j] > best) best = key[j], at = j;
    const uint32_t hi = wave_max_u32((uint32_t)(best >> 32));
    if (hi == 0) break;  // no expert left (uniform)
    bool top = (uint32_t)(best >> 32) == hi;
    if (WIDE) {
      const uint32_t lo = wave_max_u32(top ? (uint32_t)best : 0u);
      top = top && (uint32_t)best == lo;
    }
    const uint64_t tie = __ballot(top);
    int winner = 64 * at + lane;
    if (NJ > 1 && (tie & (tie - 1))) {  // several lanes: the lowest expert
      winner = (int)~wave_max_u32(top ? ~(uint32_t)winner : 0u);
    } else {
      winner = __builtin_amdgcn_readlane(winner, __builtin_ctzll(tie));
    }
    if (lane == i) mine = winner;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (lane + 64 * j == winner) key[j] = 0;
  }

  double w = mine >= 0 ? sl[mine] : 0.0;
  if (a.renorm) {
    const double sum = wave_total(w);
    w = sum > 0 ? w / sum : 0.0;
  }
  if (lane < a.k) {
    a.weights[t * a.k + lane] = (float)(w * (double)a.scale);
    a.ids[t * a.k + lane] = mine;
  }
}

template <typename T, int NJ>
hipError_t launch_route_t(const tq_route_args& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + kWaves - 1) / kWaves)), block(64 * kWaves);
  const size_t lds = (size_t)kWaves * a.experts * (a.groups > 1 ? 2 : 1) * sizeof(double);
  if (a.bias || (a.groups > 1 && a.group_best == 2))
    hipLaunchKernelGGL((route_kernel<T, NJ, true>), grid, block, lds, s, a);
  else
    hipLaunchKernelGGL((route_kernel<T, NJ, false>), grid, block, lds, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_route_n(const tq_route_args& a, hipStream_t s) {
  const int nj = (a.experts + 63) / 64;
  return nj <= 1   ? launch_route_t<T, 1>(a, s)
         : nj <= 2 ? launch_route_t<T, 2>(a, s)
         : nj <= 4 ? launch_route_t<T, 4>(a, s)
         : nj <= 8 ? launch_route_t<T, 8>(a, s)
                   : launch_route_t<T, 16>(a, s);
}

constexpr int kListWaves = 16;
constexpr int kStep = 4;  // reads of 256 ids in flight

struct __attribute__((packed, aligned(4))) Ids {
  unsigned v[4];
};

// Workgroup e: the pairs of expert e (e == experts: those without one) and offsets[e].
__global__ __launch_bounds__(64 * kListWaves) void lists_kernel(const int32_t* __restrict__ ids, int pairs, int experts, int32_t* __restrict__ order,
                                                                int32_t* __restrict__ offsets) {
  __shared__ unsigned below[kListWaves], ours[kListWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const unsigned e = blockIdx.x;  // ids as unsigned: those outside [0, experts) are at least `experts`
  const int share = ((pairs + waves - 1) / waves + 255) / 256 * 256;
  const int first = (int)min((int64_t)pairs, (int64_t)wave * share), last = (int)min((int64_t)pairs, (int64_t)first + share);
  // Four neighbouring ids of each lane per read; behind the end one that is no expert's and not below any.
  const auto read = [&](int i, Ids* id) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      const int p = i + 256 * j + 4 * lane;
      if (p + 4 <= last) {
        id[j] = *reinterpret_cast<const Ids*>(ids + p);
#pragma unroll
        for (int c = 0; c < 4; ++c) id[j].v[c] = min(id[j].v[c], (unsigned)experts);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) id[j].v[c] = p + c < last ? min((unsigned)ids[p + c], (unsigned)experts) : 0xFFFFFFFFu;
      }
    }
  };
  unsigned lt = 0, eq = 0;  // this lane's
  for (int i = first; i < last; i += 256 * kStep) {
    Ids id[kStep];
    read(i, id);
#pragma unroll
    for (int j = 0; j < kStep; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) lt += id[j].v[c] < e, eq += id[j].v[c] == e;
  }
  lt = wave_total(lt), eq = wave_total(eq);
  if (lane == 0) below[wave] = lt, ours[wave] = eq;
  __syncthreads();
  // lane w: wave w's
  const unsigned b = lane < waves ? below[lane] : 0, o = lane < waves ? ours[lane] : 0;
  const unsigned all = wave_total(b);
  int at = (int)(all + lane_value(wave_scan(o) - o, wave));
  if (threadIdx.x == 0) offsets[e] = (int)all;
  if (eq == 0) return;
  for (int i = first; i < last; i += 256 * kStep) {
    Ids id[kStep];
    read(i, id);
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      uint64_t hits[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) hits[c] = __ballot(id[j].v[c] == e);
      if ((hits[0] | hits[1] | hits[2] | hits[3]) == 0) continue;  // uniform
      const uint64_t lower = (uint64_t(1) << lane) - 1;
      int to = at + __popcll(hits[0] & lower) + __popcll(hits[1] & lower) + __popcll(hits[2] & lower) + __popcll(hits[3] & lower);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (id[j].v[c] == e) order[to++] = i + 256 * j + 4 * lane + c;
      at += __popcll(hits[0]) + __popcll(hits[1]) + __popcll(hits[2]) + __popcll(hits[3]);
    }
  }
}

}  // namespace

hipError_t launch_route(const tq_route_args& a, hipStream_t s) {
  return a.in_type == TQ_F32 ? launch_route_n<float>(a, s) : a.in_type == TQ_BF16 ? launch_route_n<bf16>(a, s) : launch_route_n<f16>(a, s);
}

hipError_t launch_expert_lists(const int32_t* ids, int64_t pairs, int experts, int32_t* order, int32_t* offsets, hipStream_t s) {
  const int waves = (int)std::min<int64_t>(kListWaves, std::max<int64_t>(1, (pairs + 255) / 256));
  hipLaunchKernelGGL(lists_kernel, dim3((unsigned)experts + 1), dim3(64 * waves), 0, s, ids, (int)pairs, experts, order, offsets);
  return hipGetLastError();
}

}  // namespace tq
