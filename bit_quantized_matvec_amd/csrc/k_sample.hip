// k_sample.hip -- the next token of each row of logits, from a given random
// number: temperature, top-k, top-p, min-p.
//
// The filters each keep a beginning of one order (logits descending, equal
// ones by index), so what stays after top-k and top-p is "keys above K, and
// the first j of those equal to K", found without sorting.  min_p is a test of
// each token by itself.
//
// A weight is exp(z) in fp64; within a slice of a row it is a whole number of
// 2^-43 of the slice's largest, so that the sums of LDS atomics do not depend
// on their order; slices are added up as fp64 in one order.  fp32 would draw
// another token wherever u falls within some 2^-20 of a border.
//
// Four launches:
//   bins_kernel, a workgroup per slice of a row: the slice, held in registers,
//     gives its largest logit and a histogram (tokens, weight) over bins of 1/8
//     in z, 32 down from it.  Bins are floor(8 x / T), the same numbers in
//     every slice, so the histograms of a row add up.
//   plan_kernel, one per row: adds them, and names the bins in which the cuts
//     of top-k, top-p and min-p lie.  Tokens further down than 32 weigh less
//     than 2^-44 of the largest: nothing.  Greedy rows end here.
//   list_kernel, one per slice: the tokens of those bins.
//   pick_kernel, one per row: finds K and j among them (by 1024 digits of the
//     keys' range at a time), adds up what stays per slice, and draws: the
//     slice, then the token in it.
// One row of 131072: 6.2, 7.4, 4.4 and 13 us, latencies of one workgroup in the
// second and the fourth.  256 rows of 200003 in bf16 with top-p 137 us: 72, 12,
// 30 and 30; the first two kernels over the logits (102 MB, 20 us at a large
// copy's rate) are bound by the vector units: some 30 instructions per
// logit, half of them fp64, in the first, 10 in the list.
//
// Where a slice has too many of them (a flat row), pick_kernel searches the
// whole row instead (search_row: a radix descent over the keys).  One such row
// of 131072 takes 171 us with top-k and 300 with top-p, 64 of them 241 and 327.
//
// (Two launches, whose last workgroups of a row did the second and the fourth
// kernel's work, cost one row as much and 256 rows twice: counting arrivals
// across the XCDs takes some 15 ns a workgroup whatever the counter's place.)
#include <algorithm>
#include <type_traits>

#include "batch.h"
#include "lanes.h"
#include "sample_bins.h"
#include "seq.h"

namespace tq {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kPer = 16;     // logits of a thread of the slices' kernels
constexpr int kLeastThreads = 256;  // of a slice
constexpr int kPickThreads = 1024;
constexpr int kPlanShares = 4;
constexpr int kShare = 1024;  // places of a slice in its row's list
constexpr int kMaxSlices = 65;
constexpr int kNear = 4096;  // places of the list that are kept in LDS
constexpr int kDigits = 1024;
constexpr uint64_t kOne = uint64_t(1) << 43;  // the weight of the largest logit

__device__ inline uint32_t key_of(float x) {  // 0: never drawn
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 counts as +0
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ inline float value_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key); }
// 16-bit logits as fp32 leave the lowest bits of keys alike.
template <typename T>
constexpr int kSame = sizeof(T) == 4 ? 0 : __is_same(T, bf16) ? 16 : 13;
template <int SAME>
__device__ inline uint32_t whole_key(uint32_t k) {  // of key >> SAME
  const uint32_t key = k << SAME;
  return key >> 31 ? key : key | ((1u << SAME) - 1);
}

// exp(z) for z in [-50, 0]: z = (64 k + j) ln2 / 64 + r, |r| <= ln2 / 128, exp(z) = 2^k 2^(j/64) exp(r), the last by its series
// to r^6 / 720 < 2^-54.  k ln2 / 64 is taken off in two parts, the first of 24 bits, so that its product is exact.
constexpr int kRoots = 64;
__device__ inline void fill_roots(double* roots) {
  if (threadIdx.x < kRoots) roots[threadIdx.x] = exp2((double)threadIdx.x / kRoots);
}
__device__ inline double exp_of(double z, const double* roots) {
  constexpr double kStep = 0.6931471805599453094 / kRoots, kHigh = (double)(float)kStep;
  constexpr double kLow = (kStep - kHigh) + 2.3190468138462996e-17 / kRoots;  // (the double nearest ln2 is that much short)
  constexpr double kRound = 0x1.8p52;  // a sum with it is rounded to a whole number, which its low bits hold
  const double s = __builtin_fma(z, 1.0 / kStep, kRound), n = s - kRound;
  const int i = (int)__builtin_bit_cast(uint64_t, s);
  const double r = __builtin_fma(n, -kLow, __builtin_fma(n, -kHigh, z));
  double p = __builtin_fma(r, 1.0 / 120, 1.0 / 24);
  p = __builtin_fma(r, p, 1.0 / 6);
  p = __builtin_fma(r, p, 0.5);
  p = __builtin_fma(r, p, 1.0);
  p = __builtin_fma(r, p, 1.0);
  // times 2^(i >> 6), by the exponent's bits: z above -50 keeps them in range
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, roots[i & (kRoots - 1)] * p) + ((uint64_t)(uint32_t)(i >> 6) << 52));
}

struct Scale {
  float most;
  double inv_t;
  const double* roots;
  // z of a logit above -inf
  __device__ double z(float x) const { return x == most ? 0.0 : ((double)x - (double)most) * inv_t; }
  __device__ double e(float x) const {
    const double v = z(x);
    const double e = exp_of(fmax(v, -50.0), roots);
    return v > -50.0 ? e : 0.0;  // (also where +inf makes z no number)
  }
  // units(e(x)), which of e^-50 are none.  FINITE: the largest logit is.
  template <bool FINITE = false>
  __device__ uint64_t weight(float x) const {
    return units(exp_of(fmax(FINITE ? ((double)x - (double)most) * inv_t : z(x), -50.0), roots));
  }
  // A number up to 1 as a whole number of 2^-43: the low bits of its sum with 2^52
  __device__ static uint64_t units(double e) { return __builtin_bit_cast(uint64_t, __builtin_fma(e, (double)kOne, 0x1p52)) & ((uint64_t(1) << 52) - 1); }
};

// ---- the workspace ----

struct Request {
  double inv_t, top_p, min_p;
  float per;  // bins of a unit of x
  int64_t top_k;
  bool greedy, use_k, use_p, sums;
};
struct Slice {  // a slice's largest logit and its first place
  float most;
  int at;
};
// What plan_kernel leaves for the kernels behind it.  Bins count down from that of the row's largest logit.
struct Row {
  Request q;
  float most;
  int top_bin;
  int search;       // 0: the token is there already
  int k_bin;        // the cut of top-k lies in this bin (kBins: no top-k)
  int p0, p1;       // that of top-p in one of these (p0 > p1: no top-p)
  int m0, m1;       // tokens above m0 pass min_p, below m1 none (m0 = kBins: no min-p)
  uint32_t k_count; // tokens above k_bin
  double k_mass;    // weight above k_bin; without top-k of the row
  double p_mass;    // weight above p0
  double total;     // weight of the row
};
struct Layout {
  int slices, threads;
  int64_t per;  // logits of a slice
  int64_t rows, parts, mass, count, shares, list, bytes;
};
constexpr int64_t kRows = 1024;  // of one launch
Layout layout(int64_t rows, int64_t vocab) {
  Layout l;
  rows = std::min(rows, kRows);
  // Slices of 4096 logits, since one workgroup draws in one: 16384 take its compute unit 9 us instead of 2.  More in vocabularies
  // of more than 64 slices, whose sums one wave adds.
  l.threads = kLeastThreads;
  while (vocab + 7 > (int64_t)l.threads * kPer * kMaxSlices) l.threads *= 2;
  l.per = l.threads * kPer;
  l.slices = (int)((vocab + 7 + l.per - 1) / l.per);  // (the first logit may be place 7)
  // Larger slices are fewer: places for as many as a smaller vocabulary has at most, so that a workspace serves it too.
  const int64_t most = std::min<int64_t>(kMaxSlices, (vocab + 7 + kLeastThreads * kPer - 1) / (kLeastThreads * kPer));
  const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  l.rows = 0;
  l.parts = l.rows + up(rows * (int64_t)sizeof(Row));
  l.mass = l.parts + up(rows * most * (int64_t)sizeof(Slice));
  l.count = l.mass + up(rows * most * kBins * 8);
  l.shares = l.count + up(rows * most * kBins * 4);
  l.list = l.shares + up(rows * most * 4);
  l.bytes = l.list + up(rows * most * kShare * 4);
  return l;
}
struct Space {
  Row* rows;
  Slice* parts;               // [rows][slices]
  unsigned long long* mass;   // [rows][slices][kBins], sums from the slice's first bin on
  unsigned* count;            // [rows][slices][kBins], likewise
  uint32_t* list;             // [rows][slices][kShare]: keys
  unsigned* shares;           // [rows][slices]: how many a slice has
  int slices;
};

// Places of a row are counted from the 16-byte block that its first logit lies in, so that blocks of 16 bytes are read whole
// whatever the row's alignment: logit i is place i + lead.
template <typename T>
__device__ inline int lead_of(const T* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
}
// kPer logits of a thread: groups of 16 bytes from logit `at` on, `stride` logits apart.  What lies outside [0, n) or is NaN is
// -inf.
template <typename T, int PER = kPer>
__device__ inline void load_logits(const T* row, int64_t at, int64_t stride, int64_t n, float* x) {
  constexpr int kV = 16 / sizeof(T);
  typedef Vec<T, kV> V;
#pragma unroll
  for (int g = 0; g < PER / kV; ++g, at += stride) {
    if (at >= 0 && at + kV <= n) {
      const V v = *reinterpret_cast<const V*>(row + at);
#pragma unroll
      for (int j = 0; j < kV; ++j) x[kV * g + j] = (float)v.v[j];
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) x[kV * g + j] = at + j >= 0 && at + j < n ? (float)row[at + j] : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = x[i] == x[i] ? x[i] : -INFINITY;
}
// A slice's logits spread over the workgroup, neighbours in neighbouring threads; and the logit that x[i] is.
template <typename T, int PER = kPer>
__device__ inline int64_t load_slice(const T* row, int slice, int64_t n, float* x) {
  constexpr int kV = 16 / sizeof(T);
  const int64_t at = (int64_t)slice * blockDim.x * PER + (int)threadIdx.x * kV - lead_of(row);
  load_logits<T, PER>(row, at, (int64_t)blockDim.x * kV, n, x);
  return at;
}
// The same in any order, for parts of fewer than 16 bytes per thread.
template <typename T, int PER>
__device__ inline void load_part(const T* row, int slice, int64_t n, float* x) {
  if constexpr (PER * sizeof(T) >= 16) {
    load_slice<T, PER>(row, slice, n, x);
  } else {
    const int64_t at = (int64_t)slice * blockDim.x * PER - lead_of(row) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t j = at + (int64_t)i * blockDim.x;
      x[i] = j >= 0 && j < n ? (float)row[j] : -INFINITY;
      x[i] = x[i] == x[i] ? x[i] : -INFINITY;
    }
  }
}
template <typename T>
__device__ inline int64_t logit_of(int64_t at, int i) {
  constexpr int kV = 16 / sizeof(T);
  return at + (int64_t)(i / kV) * blockDim.x * kV + i % kV;
}

__device__ inline Request request(const tq_sample_args& a, int64_t r) {
  // all asked for before the first is used (those that are not given read u)
  const float t0 = (a.temperature ? a.temperature : a.u)[r], p0 = (a.top_p ? a.top_p : a.u)[r], m0 = (a.min_p ? a.min_p : a.u)[r];
  const int32_t k0 = (a.top_k ? a.top_k : reinterpret_cast<const int32_t*>(a.u))[r];
  Request q;
  const float t = a.temperature ? t0 : 1.0f;
  q.greedy = !(t > 0.0f);
  q.inv_t = q.greedy ? 1.0 : 1.0 / (double)t;
  q.per = bins_per(q.inv_t);
  q.top_k = a.top_k ? k0 : 0;
  q.top_p = a.top_p ? (double)p0 : 1.0;
  const double m = a.min_p && !q.greedy ? (double)m0 : 0.0;
  q.min_p = m > 0.0 ? fmin(m, 1.0) : 0.0;
  q.use_k = !q.greedy && q.top_k > 0 && q.top_k < a.vocab;
  q.use_p = !q.greedy && q.top_p < 1.0;
  q.sums = !q.greedy || a.logprob;
  return q;
}

__device__ inline void finish(const tq_sample_args& a, int64_t r, int token, double z, double total) {
  a.tokens[r] = token;
  if (a.logprob) a.logprob[r] = token < 0 ? -INFINITY : (float)(z - log(total));
}

// ---- the first launch ----

struct BinsShared {
  unsigned long long mass[kBins];
  unsigned count[kBins];
  uint32_t best[kMaxWaves];
  int best_at[kMaxWaves];
  unsigned long long sum[kBins / 64];
  unsigned tokens[kBins / 64];
  double roots[kRoots];
};

// The largest of a workgroup's logits and its first place, in all threads.
__device__ inline void block_best(float* best, int* at, uint32_t* lds_best, int* lds_at) {
  const uint32_t mine = key_of(*best), most = wave_max_u32(mine);
  const int first = (int)~wave_max_u32(mine == most ? ~(uint32_t)*at : 0u);
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) lds_best[threadIdx.x >> 6] = most, lds_at[threadIdx.x >> 6] = first;
  __syncthreads();
  uint32_t key = lds_best[0];
  *at = lds_at[0];
  for (int w = 1; w < waves; ++w)
    if (lds_best[w] > key || (lds_best[w] == key && lds_at[w] < *at)) key = lds_best[w], *at = lds_at[w];
  *best = key ? value_of(key) : -INFINITY;
  __syncthreads();
}

template <typename T>
__global__ __launch_bounds__(1024) void bins_kernel(tq_sample_args a, Space ws) {
  __shared__ BinsShared sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int slice = blockIdx.x % ws.slices;
  const int64_t r = blockIdx.x / ws.slices;
  const Request q = request(a, r);
  for (int b = tid; b < kBins; b += blockDim.x) sh.mass[b] = 0, sh.count[b] = 0;
  fill_roots(sh.roots);

  float x[kPer];
  const int64_t at0 = load_slice(static_cast<const T*>(a.logits) + r * a.logit_stride, slice, a.vocab, x);
  float best = -INFINITY;
  int at = 0x7FFFFFFF;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (x[i] > best) best = x[i], at = (int)logit_of<T>(at0, i);
  block_best(&best, &at, sh.best, sh.best_at);
  if (q.sums && best > -INFINITY) {  // uniform
    const Scale sc{best, q.inv_t, sh.roots};
    const int top = bin_of(best, q.per);
    constexpr int kSide = 4;  // exponentials side by side, without branches, so that they overlap
    const auto add = [&](auto finite) __attribute__((always_inline)) {
#pragma unroll
      for (int i0 = 0; i0 < kPer; i0 += kSide) {
        uint64_t w[kSide];
        int b[kSide];
#pragma unroll
        for (int i = 0; i < kSide; ++i) w[i] = sc.weight<decltype(finite)::value>(x[i0 + i]), b[i] = top - bin_of(x[i0 + i], q.per);
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          // (64 logits in one bin queue for 128 cycles, in 16 bins for 20, in 64 for 13)
          if (x[i0 + i] > -INFINITY && (unsigned)b[i] < kBins) {
            atomicAdd(&sh.mass[b[i]], (unsigned long long)w[i]);
            if (q.use_k) atomicAdd(&sh.count[b[i]], 1u);
          }
        }
      }
    };
    if (best < INFINITY)
      add(std::true_type());
    else
      add(std::false_type());
  }
  __syncthreads();
  const int64_t part = r * ws.slices + slice;
  if (q.sums) {  // sums from the first bin on: every sum that is asked for later is one number
    uint64_t m = 0, c = 0;
    if (tid < kBins) {
      m = wave_scan((uint64_t)sh.mass[tid]);
      if (q.use_k) c = wave_scan((uint64_t)sh.count[tid]);
      if (lane == 63) sh.sum[tid >> 6] = m, sh.tokens[tid >> 6] = (unsigned)c;
    }
    __syncthreads();
    if (tid < kBins) {
      for (int w = 0; w < tid >> 6; ++w) m += sh.sum[w], c += sh.tokens[w];
      ws.mass[part * kBins + tid] = m;
      if (q.use_k) ws.count[part * kBins + tid] = (unsigned)c;
    }
  }
  if (tid == 0) ws.parts[part] = {best, at};
}

struct PlanShared {
  double roots[kRoots];
  double share_mass[kPlanShares][kBins];
  unsigned share_count[kPlanShares][kBins];
  double cum_mass[kBins];
  unsigned cum_count[kBins];
  double scale[kMaxSlices];
  int shift[kMaxSlices];
};

// kBins threads for each share of the slices
__global__ __launch_bounds__(kBins * kPlanShares) void plan_kernel(tq_sample_args a, Space ws) {
  __shared__ PlanShared sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t r = blockIdx.x;
  const Request q = request(a, r);
  fill_roots(sh.roots);
  // by every wave for itself: slices lane and lane + 64
  uint32_t key = 0;
  int at = 0x7FFFFFFF;
  Slice mine{-INFINITY, 0x7FFFFFFF};  // slice tid's
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const Slice part = lane + 64 * j < ws.slices ? ws.parts[r * ws.slices + lane + 64 * j] : Slice{-INFINITY, 0x7FFFFFFF};
    if (key_of(part.most) > key) key = key_of(part.most), at = part.at;  // (equal ones: the first slice has the first place)
    if (tid == lane + 64 * j) mine = part;
  }
  const uint32_t most = wave_max_u32(key);
  at = (int)~wave_max_u32(key == most ? ~(uint32_t)at : 0u);
  const float best = most ? value_of(most) : -INFINITY;
  __syncthreads();  // (the roots)
  if (!(best > -INFINITY)) {  // nothing to draw from
    if (tid == 0) {
      finish(a, r, -1, 0.0, 1.0);
      ws.rows[r].search = 0;
    }
    return;
  }
  const Scale sc{best, q.inv_t, sh.roots};
  const int top = bin_of(best, q.per);
  if (tid < ws.slices) {
    const bool some = mine.most > -INFINITY;
    sh.scale[tid] = some ? sc.e(mine.most) / (double)kOne : 0.0;
    sh.shift[tid] = some ? bins_below(top, bin_of(mine.most, q.per)) : kBins;
  }
  __syncthreads();
  {
    // each slice of this thread's share is asked for before the first is used (counts also where nobody wrote any: they are not
    // used then)
    double m = 0;
    unsigned c = 0;
    constexpr int kEach = (kMaxSlices + kPlanShares - 1) / kPlanShares;
    const int bin = tid & (kBins - 1), share = tid / kBins;
    const int64_t i0 = r * ws.slices * kBins;
    unsigned long long v[kEach];
    unsigned w[kEach];
    if (q.sums) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (kPlanShares * j >= ws.slices) continue;  // uniform
        const int s = min(share + kPlanShares * j, ws.slices - 1);
        const int64_t i = i0 + s * kBins + max(bin - sh.shift[s], 0);
        v[j] = ws.mass[i], w[j] = ws.count[i];
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int s = share + kPlanShares * j;
        if (s < ws.slices && bin >= sh.shift[s]) m = __builtin_fma((double)v[j], sh.scale[s], m), c += w[j];
      }
    }
    sh.share_mass[share][bin] = m, sh.share_count[share][bin] = c;
    __syncthreads();
    if (tid < kBins) {
      m = 0, c = 0;
#pragma unroll
      for (int j = 0; j < kPlanShares; ++j) m += sh.share_mass[j][tid], c += sh.share_count[j][tid];
      sh.cum_mass[tid] = m, sh.cum_count[tid] = c;
    }
  }
  __syncthreads();
  if (tid >= 64) return;
  // wave 0: first bins that reach a number
  const auto first_bin = [&](auto reached) {
    int f = kBins;
    for (int i = kBins / 64 - 1; i >= 0; --i) {
      const uint64_t ok = __ballot(reached(64 * i + lane));
      if (ok) f = 64 * i + __builtin_ctzll(ok);
    }
    return f;
  };
  const double total = sh.cum_mass[kBins - 1];
  if (q.greedy) {
    if (lane == 0) {
      finish(a, r, at, 0.0, total);
      ws.rows[r].search = 0;
    }
    return;
  }
  Row row;
  row.q = q, row.most = best, row.top_bin = top, row.search = 1, row.total = total;
  row.k_bin = kBins, row.k_count = 0, row.k_mass = total;
  row.p0 = 1, row.p1 = 0, row.p_mass = 0, row.m0 = row.m1 = kBins;
  double hi = total;
  if (q.use_k) {
    row.k_bin = first_bin([&](int b) { return sh.cum_count[b] >= (uint64_t)q.top_k; });
    if (row.k_bin < kBins) {  // (otherwise all that weigh anything stay)
      row.k_count = row.k_bin ? sh.cum_count[row.k_bin - 1] : 0;
      row.k_mass = row.k_bin ? sh.cum_mass[row.k_bin - 1] : 0.0;
      hi = sh.cum_mass[row.k_bin];
    }
  }
  if (q.use_p) {
    // what stays after top-k weighs between k_mass and hi; sums of the parts in another order differ in the last bits
    const double p = fmax(q.top_p, 0.0), g0 = p * row.k_mass * (1 - 1e-12), g1 = p * hi * (1 + 1e-12);
    row.p0 = min(first_bin([&](int b) { return sh.cum_mass[b] >= g0; }), kBins - 1);
    row.p1 = min(first_bin([&](int b) { return sh.cum_mass[b] >= g1; }), min(row.k_bin, kBins - 1));
    row.p0 = min(row.p0, row.p1);
    row.p_mass = row.p0 ? sh.cum_mass[row.p0 - 1] : 0.0;
  }
  if (q.min_p > 0.0) {
    // z = log(min_p): the difference of two logits' bins is off by one, and by two more for roundings
    const int b = (int)fmin(-log(q.min_p) * kPerUnit, 1e6);
    row.m0 = max(0, b - 3), row.m1 = b + 3;
    if (!bins_measure(best, q.per, q.inv_t)) row.m0 = 0, row.m1 = kBins;
  }
  if (lane == 0) ws.rows[r] = row;
}

// ---- the search of a whole row, by one workgroup ----

// What stays: keys above `key`, and the first `ties` (by index) of those equal to it, if their e is at least min_p.
struct Cut {
  uint32_t key;
  uint64_t ties;
  double sum;    // weight of what stays (as if every e were at least min_p)
};

struct PickShared {
  unsigned long long mass[kDigits];
  uint32_t count[kDigits];
  unsigned long long part[kMaxWaves], part2[kMaxWaves];
  uint32_t kmin, kmax;
  int digit;
  unsigned long long before_count, before_mass, digit_count, digit_mass;
  unsigned long long slice_mass[kMaxSlices], slice_ties[kMaxSlices];
  double slice_sum[kMaxSlices];
  int slice_shift[kMaxSlices];
  float slice_most[kMaxSlices];
  int flag, pick;
  int token;
  double run;
  unsigned long long tied;
  double roots[kRoots];
  uint32_t near[kNear];  // the first of the list, and their e
  double near_e[kNear];
  unsigned share[kMaxSlices + 1];  // a slice's first place in the row's list
};

// The cut at a key of which there are `equal`, each of weight w, with `sum` above it: `ties` of them, or as many as the goal
// takes.
__device__ inline Cut cut_of(uint32_t key, uint64_t ties, uint64_t equal, bool by_count, double goal, double sum, double w) {
  if (!by_count) ties = w > 0 && goal > sum ? (uint64_t)fmin(fmax(1.0, __builtin_ceil((goal - sum) / w)), 1e9) : 1;
  ties = min(ties, equal);
  return {key, ties, sum + (double)ties * w};
}

// A token's digit counted.  Equal logits (16-bit ones are many) would queue at one address: the first few different keys of a
// wave are counted by one lane each.
__device__ inline void count_digit(uint32_t key, uint32_t b, uint64_t w, PickShared& sh) {
  const int lane = threadIdx.x & 63;
  uint64_t left = __ballot(true);
#pragma unroll 1
  for (int i = 0; i < 8 && left; ++i) {
    const int who = __builtin_ctzll(left);
    const uint64_t same = __ballot(key == (uint32_t)__builtin_amdgcn_readlane((int)key, who));
    const int n = __popcll(same);
    if (lane == who) {
      atomicAdd(&sh.count[b], (uint32_t)n);
      atomicAdd(&sh.mass[b], (unsigned long long)(w * n));
    }
    left &= ~same;
    if (n < 4) break;
  }
  if (left >> lane & 1) {
    atomicAdd(&sh.count[b], 1u);
    atomicAdd(&sh.mass[b], (unsigned long long)w);
  }
}

// The beginning of the order, among the keys in [lo, hi] that `each` goes through, that reaches `tokens` tokens (by_count) or
// the weight `goal` (a fraction of 1), `above` of it already there: by 1024 digits of the keys' range at a time.
template <int SAME, typename EACH>
__device__ Cut find_cut(EACH each, uint32_t lo, uint32_t hi, const Scale& sc, bool by_count, uint64_t tokens, double goal, double above, PickShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint64_t before_count = 0, before_mass = 0, equal = 0;
  lo >>= SAME, hi >>= SAME;
  while (true) {
    int shift = 0;
    while ((hi - lo) >> shift >= kDigits) ++shift;
    for (int b = tid; b < kDigits; b += blockDim.x) sh.count[b] = 0, sh.mass[b] = 0;
    if (tid == 0) sh.digit = -1;
    __syncthreads();
    each([&](uint32_t key, uint64_t weight) {
      const uint32_t k = key >> SAME;
      if (k < lo || k > hi) return;
      count_digit(key, (k - lo) >> shift, weight, sh);
    });
    __syncthreads();
    // thread i has the digits from kDigits - 1 - per * i downwards
    const int per = kDigits / (int)blockDim.x;
    uint64_t c = 0, m = 0;
    for (int j = 0; j < per; ++j) {
      const int b = kDigits - 1 - (per * tid + j);
      c += sh.count[b], m += sh.mass[b];
    }
    const uint64_t c_in = wave_scan(c), m_in = wave_scan(m);
    if (lane == 63) sh.part[wave] = c_in, sh.part2[wave] = m_in;
    __syncthreads();
    uint64_t cb = before_count + c_in - c, mb = before_mass + m_in - m;
    for (int w = 0; w < wave; ++w) cb += sh.part[w], mb += sh.part2[w];
    for (int j = 0; j < per; ++j) {
      const int b = kDigits - 1 - (per * tid + j);
      const uint64_t ca = cb + sh.count[b], ma = mb + sh.mass[b];
      const auto reached = [&](uint64_t n, uint64_t v) { return by_count ? n >= tokens : n > 0 && above + (double)v / (double)kOne >= goal; };
      if (reached(ca, ma) && !reached(cb, mb)) {  // one digit of one thread
        sh.digit = b;
        sh.before_count = cb, sh.before_mass = mb, sh.digit_count = sh.count[b], sh.digit_mass = sh.mass[b];
      }
      cb = ca, mb = ma;
    }
    __syncthreads();
    const int digit = sh.digit;
    if (digit < 0) return {0, 0, 0};  // not reached: all of them stay (uniform)
    before_count = sh.before_count, before_mass = sh.before_mass, equal = sh.digit_count;
    const uint64_t digit_mass = sh.digit_mass;
    __syncthreads();
    hi = (uint32_t)min((uint64_t)hi, lo + ((uint64_t)(digit + 1) << shift) - 1);
    lo += (uint32_t)digit << shift;
    // one token in the digit: all from its lowest key on stay
    if (equal == 1) return {whole_key<SAME>(lo), 1, above + (double)(before_mass + digit_mass) / (double)kOne};
    if (shift == 0) break;
  }
  const uint32_t key = whole_key<SAME>(lo);
  return cut_of(key, by_count ? tokens - before_count : 0, equal, by_count, goal, above + (double)before_mass / (double)kOne,
                (double)sc.weight(value_of(key)) / (double)kOne);
}

// The same among at most 64 keys (0: none), lane i of every wave with key i and its weight: each wave compares them with a
// sixteenth of all, and the parts are added through LDS.
__device__ inline Cut small_cut(uint32_t key, uint64_t w, bool by_count, uint64_t tokens, double goal, double above, PickShared& sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kWaves = kPickThreads / 64;
  unsigned long long* masses = sh.mass;  // [kWaves][64]
  uint32_t* counts = sh.count;
  static_assert(kWaves * 64 <= kDigits, "the digits' places serve here");
  uint64_t mass = 0;
  unsigned count = 0;  // above: low half, equal: high half
#pragma unroll
  for (int i = 0; i < 64 / kWaves; ++i) {
    const int j = wave + kWaves * i;
    const uint32_t k = lane_value(key, j);
    const uint64_t v = lane_value(w, j);
    count += (k > key ? 1u : 0u) + (k == key ? 0x10000u : 0u);
    mass += k > key ? v : 0;
  }
  masses[wave * 64 + lane] = mass, counts[wave * 64 + lane] = count;
  __syncthreads();
  mass = 0, count = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) mass += masses[i * 64 + lane], count += counts[i * 64 + lane];
  __syncthreads();
  unsigned equal = count >> 16;
  count &= 0xFFFF;
  const auto reached = [&](uint64_t c, uint64_t m) { return by_count ? c >= tokens : c > 0 && above + (double)m / (double)kOne >= goal; };
  const uint64_t hit = __ballot(key != 0 && reached(count + equal, mass + w * equal) && !reached(count, mass));
  if (!hit) return {0, 0, 0};  // uniform over the workgroup
  const int who = __builtin_ctzll(hit);
  key = lane_value(key, who), count = lane_value(count, who), equal = lane_value(equal, who), mass = lane_value(mass, who);
  const double sum = above + (double)mass / (double)kOne, one = (double)lane_value(w, who) / (double)kOne;
  return cut_of(key, by_count ? tokens - count : 0, equal, by_count, goal, sum, one);
}

// Whether a logit stays; ties are for the caller to count.
struct Kept {
  Scale sc;
  Cut cut;
  double min_p;
  // 0: goes, 1: stays, 2: equal to the cut's key
  __device__ int test(uint32_t key, float x, double* e) const {
    if (key == 0 || key < cut.key) return 0;
    *e = sc.e(x);
    if (!(*e >= min_p)) return 0;
    return key == cut.key ? 2 : 1;
  }
};

// The token of [first, last) at which the running weight passes `goal` (in units of 2^-43 of the row's largest), `ties` of the
// equal ones still to come; the last one that weighs anything where it never does.  PER logits a thread.
template <typename T, int PER>
__device__ int draw(const T* row, int64_t first, int64_t last, const Kept& k, uint64_t ties, double goal, PickShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t at0 = first + (int64_t)tid * PER;
  float x[PER];
  if constexpr (PER * sizeof(T) >= 16) {
    load_logits<T, PER>(row, at0, 16 / sizeof(T), last, x);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      x[i] = at0 + i >= 0 && at0 + i < last ? (float)row[at0 + i] : -INFINITY;
      x[i] = x[i] == x[i] ? x[i] : -INFINITY;
    }
  }
  uint64_t w[PER], sum = 0, equal = 0;
  unsigned tied = 0;
  double e[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) e[i] = k.sc.e(x[i]);  // (without branches, so that they overlap)
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t key = key_of(x[i]);
    const int t = key == 0 || key < k.cut.key || !(e[i] >= k.min_p) ? 0 : key == k.cut.key ? 2 : 1;
    w[i] = t ? Scale::units(e[i]) : 0;
    if (t == 2) tied |= 1u << i, ++equal;
  }
  const uint64_t eq_in = wave_scan(equal);
  if (lane == 63) sh.part[wave] = eq_in;
  __syncthreads();
  uint64_t before = eq_in - equal;
  for (int v = 0; v < wave; ++v) before += sh.part[v];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (tied >> i & 1) {
      if (before >= ties) w[i] = 0;
      ++before;
    }
    sum += w[i];
  }
  __syncthreads();
  const uint64_t in = wave_scan(sum);
  if (lane == 63) sh.part[wave] = in;
  if (tid == 0) sh.token = -1, sh.pick = 0x7FFFFFFF;
  __syncthreads();
  uint64_t run = in - sum;
  for (int v = 0; v < wave; ++v) run += sh.part[v];
  int found = 0x7FFFFFFF, final = -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    run += w[i];
    if (w[i]) {
      final = (int)(at0 - first) + i;
      if ((double)run > goal) found = min(found, final);
    }
  }
  // threads are in the order of their logits
  const uint64_t founds = __ballot(found != 0x7FFFFFFF), finals = __ballot(final >= 0);
  if (lane == 0) {
    if (founds) atomicMin(&sh.pick, (int)lane_value((uint32_t)found, __builtin_ctzll(founds)));
    if (finals) atomicMax(&sh.token, (int)lane_value((uint32_t)final, 63 - __builtin_clzll(finals)));
  }
  __syncthreads();
  const int p = sh.pick != 0x7FFFFFFF ? sh.pick : sh.token;
  __syncthreads();
  return p < 0 ? -1 : (int)first + p;
}

// The goal of a draw from what weighs `sum`.
__device__ inline double goal_of(float u, double sum) { return !(u > 0.0f) ? 0.0 : u >= 1.0f ? INFINITY : (double)u * sum; }

// Per slice: the weight of what stays (units of 2^-43 of the row's largest) and the number equal to the cut's key.
template <typename T, int PER>
__device__ void search_row(const tq_sample_args& a, int64_t r, const Request& q, const Scale& sc, int slices, Kept* kept, PickShared& sh) {
  const T* row = static_cast<const T*>(a.logits) + r * a.logit_stride;
  const int n = (int)a.vocab;
  const auto each = [&](auto f) {
    for (int s = 0; s < slices; ++s) {
      float x[PER];
      load_part<T, PER>(row, s, n, x);
#pragma unroll 1
      for (int i = 0; i < PER; ++i)
        if (const uint32_t key = key_of(x[i])) f(key, sc.weight(x[i]));
    }
  };
  Cut cut{0, 0, 0};
  const uint32_t top = key_of(sc.most);
  double stays = -1;
  if (q.use_k) {
    cut = find_cut<kSame<T>>(each, 1u, top, sc, true, (uint64_t)q.top_k, 0.0, 0.0, sh);
    if (cut.key) stays = cut.sum;
  }
  if (q.use_p) {
    if (stays < 0) {
      uint64_t m = 0;
      each([&](uint32_t, uint64_t weight) { m += weight; });
      m = wave_total(m);
      if ((threadIdx.x & 63) == 0) sh.part[threadIdx.x >> 6] = m;
      __syncthreads();
      m = 0;
      for (int w = 0; w < (int)(blockDim.x >> 6); ++w) m += sh.part[w];
      __syncthreads();
      stays = (double)m / (double)kOne;
    }
    cut = find_cut<kSame<T>>(each, 1u, top, sc, false, 0, fmax(q.top_p, 0.0) * stays, 0.0, sh);
  }
  *kept = Kept{sc, cut, q.min_p};
  for (int s = 0; s < slices; ++s) {
    float x[PER];
    load_part<T, PER>(row, s, n, x);
    uint64_t m = 0, ties = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      double e = 0;
      const int t = kept->test(key_of(x[i]), x[i], &e);
      if (t == 1) m += Scale::units(e);
      if (t == 2) ++ties;
    }
    m = wave_total(m), ties = wave_total(ties);
    if ((threadIdx.x & 63) == 0) {
      atomicAdd(&sh.slice_mass[s], (unsigned long long)m);
      atomicAdd(&sh.slice_ties[s], (unsigned long long)ties);
    }
  }
  __syncthreads();
}

// ---- the tokens in question ----

__device__ inline bool any_cut(const Row& row) { return row.k_bin < kBins || row.p0 <= row.p1 || row.m0 < kBins; }

template <typename T>
__global__ __launch_bounds__(1024) void list_kernel(tq_sample_args a, Space ws) {
  __shared__ uint32_t keys[kShare];
  __shared__ unsigned part[kMaxWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int slice = blockIdx.x % ws.slices;
  const int64_t r = blockIdx.x / ws.slices;
  const Row row = ws.rows[r];
  if (!row.search || !any_cut(row)) return;  // uniform
  const Request& q = row.q;
  const int top = row.top_bin, k_bin = row.k_bin < kBins ? row.k_bin : -1, p0 = row.p0, p1 = row.p1, m0 = row.m0, m1 = row.m1;
  // floor(v) from top - last to top - first is v from one whole number to below another
  const int first = min(min(k_bin < 0 ? kBins : k_bin, p0 <= p1 ? p0 : kBins), m0), last = max(max(k_bin, p0 <= p1 ? p1 : -1), m0 < kBins ? m1 : -1);
  const float low = (float)(top - last), high = (float)(top - first + 1);
  float x[kPer];
  load_slice(static_cast<const T*>(a.logits) + r * a.logit_stride, slice, a.vocab, x);
  unsigned in = 0;
  const auto collect = [&](auto one_range) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float v = bin_place(x[i], q.per);
      bool ok = v >= low && v < high && x[i] > -INFINITY;
      if constexpr (!decltype(one_range)::value) {
        if (!ok) continue;
        const int b = top - bin_of(x[i], q.per);
        ok = b == k_bin || (b >= p0 && b <= p1) || (b >= m0 && b <= m1);
      }
      in |= ok ? 1u << i : 0u;
    }
  };
  // One cut: its bins are all from `first` to `last`.  (With the test of each logit's bin 256 rows of 200003 take 37 us.)
  if ((k_bin >= 0) + (p0 <= p1) + (m0 < kBins) == 1)
    collect(std::true_type());
  else
    collect(std::false_type());
  const unsigned n = __popc(in), upto = (unsigned)wave_scan((uint64_t)n);
  if (lane == 63) part[wave] = upto;
  __syncthreads();
  unsigned before = upto - n, all = 0;
  for (int w = 0; w < waves; ++w) {
    if (w < wave) before += part[w];
    all += part[w];
  }
  if (tid == 0) ws.shares[r * ws.slices + slice] = all;
  if (all == 0 || all > kShare) return;  // (too many: searched otherwise)
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (in >> i & 1) keys[before++] = key_of(x[i]);
  __syncthreads();
  for (unsigned i = tid; i < all; i += blockDim.x) ws.list[(r * ws.slices + slice) * kShare + i] = keys[i];
}

// ---- the draw ----

// kPickThreads threads, PER of a slice's logits for each.
template <typename T, int PER>
__global__ __launch_bounds__(kPickThreads) void pick_kernel(tq_sample_args a, Space ws) {
  __shared__ PickShared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int waves = kPickThreads / 64, per = PER * kPickThreads;
  const int64_t r = blockIdx.x;
  const Row row = ws.rows[r];
  if (!row.search) return;  // uniform
  const Request& q = row.q;
  const float u = a.u[r];
  fill_roots(sh.roots);
  const Scale sc{row.most, q.inv_t, sh.roots};
  const T* logits = static_cast<const T*>(a.logits) + r * a.logit_stride;
  const bool use_k = row.k_bin < kBins, use_p = row.p0 <= row.p1;
  // the slices' shares one behind the other, in LDS as far as they fit
  if (tid < ws.slices) {
    const float most = ws.parts[r * ws.slices + tid].most;
    const bool some = most > -INFINITY;
    sh.slice_shift[tid] = some ? bins_below(row.top_bin, bin_of(most, q.per)) : kBins;
    sh.slice_most[tid] = most;
    sh.slice_mass[tid] = 0, sh.slice_ties[tid] = 0;
    sh.share[tid + 1] = any_cut(row) ? ws.shares[r * ws.slices + tid] : 0;
  }
  __syncthreads();
  if (wave == 0) {  // slices 2 lane, 2 lane + 1
    const unsigned c0 = 2 * lane < ws.slices ? sh.share[2 * lane + 1] : 0, c1 = 2 * lane + 1 < ws.slices ? sh.share[2 * lane + 2] : 0;
    const uint64_t over = __ballot(c0 > kShare || c1 > kShare);
    const unsigned upto = (unsigned)wave_scan((uint64_t)c0 + c1);
    if (2 * lane < ws.slices) sh.share[2 * lane + 1] = upto - c1;
    if (2 * lane + 1 < ws.slices) sh.share[2 * lane + 2] = upto;
    if (lane == 0) sh.share[0] = 0, sh.flag = over != 0;
  }
  __syncthreads();
  const bool too_many = sh.flag;
  const unsigned n = sh.share[ws.slices];
  const uint32_t* list = ws.list + r * ws.slices * kShare;
  if (!too_many) {
    for (int s = wave; s < ws.slices; s += waves)
      for (unsigned i = sh.share[s] + lane; i < min(sh.share[s + 1], (unsigned)kNear); i += 64) {
        const uint32_t key = list[s * kShare + i - sh.share[s]];
        sh.near[i] = key, sh.near_e[i] = sc.e(value_of(key));
      }
  }
  __syncthreads();
  Kept kept{sc, {0, 0, 0}, q.min_p};
  int sure = kBins;  // tokens of the bins above it stay, and are not in question
  if (too_many) {
    search_row<T, PER>(a, r, q, sc, ws.slices, &kept, sh);
    sure = 0;
  } else {
    // this thread's of the near ones
    constexpr int kOwn = kNear / kPickThreads;
    uint32_t key[kOwn];
    uint64_t units[kOwn];
    int bin[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const unsigned i = tid + kPickThreads * j;
      key[j] = i < n ? sh.near[i] : 0;
      units[j] = i < n ? Scale::units(sh.near_e[i]) : 0;
      bin[j] = row.top_bin - bin_of(key[j] ? value_of(key[j]) : 0.0f, q.per);
    }
    // the listed tokens of the bins [b0, b1], and their weights
    const auto each_of = [&](int b0, int b1) {
      return [&, b0, b1](auto f) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
          if (key[j] && bin[j] >= b0 && bin[j] <= b1) f(key[j], units[j]);
        const auto one = [&](uint32_t key) {
          const int b = row.top_bin - bin_of(value_of(key), q.per);
          if (b >= b0 && b <= b1) f(key, sc.weight(value_of(key)));
        };
        if (n > kNear)
          for (int s = wave; s < ws.slices; s += waves)
            for (unsigned i = max(sh.share[s], (unsigned)kNear) + lane; i < sh.share[s + 1]; i += 64) one(list[s * kShare + i - sh.share[s]]);
      };
    };
    const auto key_range = [&](int b0, int b1) {  // the lowest and the highest key
      if (tid == 0) sh.kmin = 0xFFFFFFFFu, sh.kmax = 0;
      __syncthreads();
      uint32_t least = 0xFFFFFFFFu, most = 0;
      each_of(b0, b1)([&](uint32_t key, uint64_t) { least = min(least, key), most = max(most, key); });
      least = ~wave_max_u32(~least), most = wave_max_u32(most);
      if (lane == 0) atomicMin(&sh.kmin, least), atomicMax(&sh.kmax, most);
      __syncthreads();
      return make_uint2(sh.kmin, sh.kmax);
    };
    int cut_bin = kBins;
    double stays = row.k_mass;
    const bool few = n <= 64;
    const uint32_t own = few && lane < (int)n ? sh.near[lane] : 0;
    const int own_bin = own ? row.top_bin - bin_of(value_of(own), q.per) : kBins;
    const auto cut_in = [&](int b0, int b1, bool by_count, uint64_t tokens, double goal, double above) {
      if (few) {
        const uint32_t key = own_bin >= b0 && own_bin <= b1 ? own : 0;
        Cut c = small_cut(key, key ? Scale::units(sh.near_e[lane]) : 0, by_count, tokens, goal, above, sh);
        if (c.key == 0) c = {~wave_max_u32(key ? ~key : 0u), uint64_t(1) << 32, 0};
        return c;
      }
      const uint2 range = key_range(b0, b1);
      if (range.y == 0) return Cut{0xFFFFFFFFu, 0, above};  // (none)
      Cut c = find_cut<kSame<T>>(each_of(b0, b1), range.x, range.y, sc, by_count, tokens, goal, above, sh);
      if (c.key == 0) c = {range.x, uint64_t(1) << 32, 0};  // by roundings not reached: all of these
      return c;
    };
    if (use_k) {
      kept.cut = cut_in(row.k_bin, row.k_bin, true, (uint64_t)q.top_k - row.k_count, 0.0, row.k_mass);
      stays = kept.cut.sum;
      cut_bin = row.k_bin;
    }
    if (use_p) {
      // the bins from p0 on are in the list up to p1, where the cut is reached
      kept.cut = cut_in(row.p0, row.p1, false, 0, fmax(q.top_p, 0.0) * stays, row.p_mass);
      cut_bin = row.top_bin - bin_of(value_of(kept.cut.key), q.per);
    }
    sure = min(cut_bin, row.m0);
    for (int s = tid; s < ws.slices && sure > 0; s += blockDim.x) {
      const int b = min(sure, kBins) - 1 - sh.slice_shift[s];
      // (a slice whose largest weighs no unit of the row's has nothing that the draw in it could find)
      const double e = sc.e(sh.slice_most[s]);
      double m = 0;
      if (b >= 0 && Scale::units(e) > 0) m = (double)ws.mass[(r * ws.slices + s) * kBins + b] * e;
      sh.slice_sum[s] = m;
    }
    // what is in question: the cut's bin, and those of min_p above it
    const int last_bin = min(cut_bin, row.m1);
    const auto stays_at = [&](uint32_t key, double e) {  // 0, 1 or, for those equal to the cut's key, 2
      const int b = row.top_bin - bin_of(value_of(key), q.per);
      return b < sure || b > last_bin || key < kept.cut.key || !(e >= q.min_p) ? 0 : key > kept.cut.key ? 1 : 2;
    };
    if (n <= kPickThreads) {  // each thread its one
      if (tid < (int)n) {
        const int t = stays_at(sh.near[tid], sh.near_e[tid]);
        int s = 0;  // the last slice whose share begins at or before this place
        for (int step = 64; step > 0; step >>= 1)
          if (s + step < ws.slices && sh.share[s + step] <= (unsigned)tid) s += step;
        if (t == 1) atomicAdd(&sh.slice_mass[s], (unsigned long long)Scale::units(sh.near_e[tid]));
        if (t == 2) atomicAdd(&sh.slice_ties[s], 1ull);
      }
    } else {
      for (int s = wave; s < ws.slices; s += waves) {
        const unsigned first = sh.share[s], last = sh.share[s + 1];
        if (first == last) continue;
        uint64_t m = 0, ties = 0;
        for (unsigned i = first + lane; i < last; i += 64) {
          const uint32_t key = i < kNear ? sh.near[i] : list[s * kShare + i - first];
          const double e = i < kNear ? sh.near_e[i] : sc.e(value_of(key));
          const int t = stays_at(key, e);
          if (t == 1) m += Scale::units(e);
          if (t == 2) ++ties;
        }
        m = wave_total(m), ties = wave_total(ties);
        if (lane == 0) sh.slice_mass[s] = m, sh.slice_ties[s] = ties;
      }
    }
    __syncthreads();
  }

  // the draw: the slice, and the token in it.  Wave 0 has slices 2 lane and 2 lane + 1.
  if (wave == 0) {
    const double tie = kept.cut.key ? (double)sc.weight(value_of(kept.cut.key)) : 0.0;
    uint64_t t[2] = {0, 0};
    double m[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int s = 2 * lane + j;
      if (s >= ws.slices) continue;
      t[j] = sh.slice_ties[s];
      m[j] = (sure > 0 ? sh.slice_sum[s] : 0.0) + (double)sh.slice_mass[s];
    }
    const uint64_t t_in = wave_scan(t[0] + t[1]);
    uint64_t left[2];  // ties that are still to come where a slice begins
    left[0] = kept.cut.ties - min(kept.cut.ties, t_in - t[0] - t[1]);
    left[1] = left[0] - min(left[0], t[0]);
#pragma unroll
    for (int j = 0; j < 2; ++j) m[j] += (double)min(left[j], t[j]) * tie;
    const double in = wave_scan(m[0] + m[1]);
    const double goal = goal_of(u, lane_value(in, 63));
    // the first slice that weighs something and whose sum passes the goal, or the last that weighs something
    const double begin[2] = {in - m[0] - m[1], in - m[1]};
    const bool some[2] = {m[0] > 0, m[1] > 0}, over[2] = {some[0] && begin[1] > goal, some[1] && in > goal};
    const uint64_t overs = __ballot(over[0] || over[1]), somes = __ballot(some[0] || some[1]);
    const int who = overs ? __builtin_ctzll(overs) : somes ? 63 - __builtin_clzll(somes) : -1;
    if (lane == max(who, 0)) {
      const int j = overs ? !over[0] : some[1];
      sh.pick = who < 0 ? -1 : 2 * lane + j;
      sh.run = goal - begin[j], sh.tied = left[j];
    }
  }
  __syncthreads();
  const int pick = sh.pick;
  const double goal = sh.run;
  const uint64_t tied = sh.tied;
  __syncthreads();
  int token = -1;
  const int lead = lead_of(logits);
  if (pick >= 0)
    token = draw<T, PER>(logits, (int64_t)pick * per - lead, min((int64_t)a.vocab, (int64_t)(pick + 1) * per - lead), kept, tied, goal, sh);
  if (tid == 0) finish(a, r, token, token < 0 ? 0.0 : sc.z((float)logits[token]), row.total);
}

template <typename T>
hipError_t launch_t(tq_sample_args a, hipStream_t s) {
  const Layout l = layout(a.rows, a.vocab);
  char* p = static_cast<char*>(a.workspace);
  const Space ws{reinterpret_cast<Row*>(p + l.rows), reinterpret_cast<Slice*>(p + l.parts),
                 reinterpret_cast<unsigned long long*>(p + l.mass), reinterpret_cast<unsigned*>(p + l.count),
                 reinterpret_cast<uint32_t*>(p + l.list), reinterpret_cast<unsigned*>(p + l.shares), l.slices};
  const int64_t all = a.rows;
  const auto from = [](auto*& q, int64_t n) {
    if (q) q += n;
  };
  for (int64_t done = 0; done < all; done += kRows) {
    a.rows = std::min(kRows, all - done);
    const dim3 grid((unsigned)(a.rows * l.slices)), block(l.threads);
    hipLaunchKernelGGL((bins_kernel<T>), grid, block, 0, s, a, ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(plan_kernel, dim3((unsigned)a.rows), dim3(kBins * kPlanShares), 0, s, a, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.top_k || a.top_p || a.min_p) {
      hipLaunchKernelGGL((list_kernel<T>), grid, block, 0, s, a, ws);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const dim3 rows((unsigned)a.rows), pick(kPickThreads);
    if (l.per == 4 * kPickThreads)
      hipLaunchKernelGGL((pick_kernel<T, 4>), rows, pick, 0, s, a, ws);
    else if (l.per == 8 * kPickThreads)
      hipLaunchKernelGGL((pick_kernel<T, 8>), rows, pick, 0, s, a, ws);
    else
      hipLaunchKernelGGL((pick_kernel<T, 16>), rows, pick, 0, s, a, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    a.logits = static_cast<const T*>(a.logits) + kRows * a.logit_stride;
    from(a.u, kRows), from(a.temperature, kRows), from(a.top_k, kRows), from(a.top_p, kRows), from(a.min_p, kRows), from(a.tokens, kRows);
    from(a.logprob, kRows);
  }
  return hipSuccess;
}

}  // namespace

int64_t sample_workspace_bytes(int64_t rows, int64_t vocab) { return layout(rows, vocab).bytes; }

hipError_t launch_sample(const tq_sample_args& a, hipStream_t s) {
  return a.in_type == TQ_F32 ? launch_t<float>(a, s) : a.in_type == TQ_BF16 ? launch_t<bf16>(a, s) : launch_t<f16>(a, s);
}

}  // namespace tq
