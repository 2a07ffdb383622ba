// k_sample.hip -- the next token of each row of logits, from a given random
// number: temperature, top-k, top-p, min-p.
//
// The filters each keep a beginning of one order (logits descending, equal
// ones by index), so what stays after top-k and top-p is "keys above K, and
// the first j of those equal to K", found without sorting: a radix descent
// over the 32-bit keys of the logits (11 + 11 + 10 bits), counting tokens and
// adding up their weights per digit, stops at the digit where the count (or
// the weight) is reached.  min_p is a test of each token by itself.
//
// A weight is exp(z) in fp64, rounded to a multiple of 2^-43, as a whole
// number: sums are exact and the same in any order, so atomics in LDS change
// nothing, and 2^20 tokens of weight 1 still fit 64 bits.  fp32 would draw
// another token wherever u falls within some 2^-20 of a border.
//
// One workgroup per row; the row is read once for its maximum, once per digit
// and search, and for the draw (a sum per wave's share of the row, the same
// over the share that holds the drawn place, then 64 tokens at a time).
#include <algorithm>

#include "batch.h"
#include "seq.h"

namespace tq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr uint64_t kOne = uint64_t(1) << 43;  // the weight of the largest logit

__device__ inline uint32_t key_of(float x) {  // 0: never drawn
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 counts as +0
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ inline float value_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key); }

struct Scale {
  float most;
  double inv_t;
  // z of a logit above -inf
  __device__ double z(float x) const { return x == most ? 0.0 : ((double)x - (double)most) * inv_t; }
  __device__ double e(float x) const {
    const double v = z(x);
    return v > -50.0 ? exp(v) : 0.0;  // (also where +inf makes z no number)
  }
  __device__ uint64_t weight(float x) const { return (uint64_t)__builtin_rint(e(x) * (double)kOne); }
};

__device__ inline uint64_t shfl_up64(uint64_t v, int d) {
  const uint32_t lo = __shfl_up((uint32_t)v, d, 64), hi = __shfl_up((uint32_t)(v >> 32), d, 64);
  return (uint64_t)hi << 32 | lo;
}
__device__ inline uint64_t wave_scan(uint64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = shfl_up64(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ inline uint64_t wave_total(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t lo = __shfl_xor((uint32_t)v, o, 64), hi = __shfl_xor((uint32_t)(v >> 32), o, 64);
    v += (uint64_t)hi << 32 | lo;
  }
  return v;
}

// What stays: keys above `key`, and the first `ties` (by index) of those equal to it, if their e is at least min_p.
struct Cut {
  uint32_t key;
  uint64_t ties;
  uint64_t above;  // weight of the keys above
};

struct Shared {
  uint32_t count[kBins];
  unsigned long long mass[kBins];
  unsigned long long part[kWaves], part2[kWaves];
  float best[kWaves];
  int best_at[kWaves];
  uint32_t digit;
  uint32_t before_count;
  unsigned long long before_mass, digit_mass;
  uint32_t digit_count;
  int pick;
  unsigned long long pick_mass, pick_ties;
};

// The beginning of the order that has `tokens` tokens (by_count), or whose weight reaches `goal`.  The caller knows that the
// row has that many, or that much.
template <typename T>
__device__ Cut find_cut(const T* row, int n, const Scale& sc, bool by_count, uint64_t tokens, double goal, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t prefix = 0;
  uint64_t above_count = 0, above_mass = 0;
  constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
  uint32_t equal = 0;
#pragma unroll 1
  for (int level = 0; level < 3; ++level) {
    const int shift = kShift[level], bins = 1 << kBits[level];
    for (int b = tid; b < bins; b += kThreads) sh.count[b] = 0, sh.mass[b] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float x = (float)row[i];
      const uint32_t key = key_of(x);
      if (key == 0 || (level > 0 && key >> (shift + kBits[level]) != prefix)) continue;
      const uint32_t b = (key >> shift) & (bins - 1);
      atomicAdd(&sh.count[b], 1u);
      atomicAdd(&sh.mass[b], (unsigned long long)sc.weight(x));
    }
    __syncthreads();
    // thread i has the digits bins - 1 - 2i and the one below it (one digit each on the last level)
    const int per = bins / kThreads;
    uint64_t c[2] = {0, 0}, m[2] = {0, 0};
    for (int j = 0; j < per; ++j) {
      const int b = bins - 1 - (per * tid + j);
      c[j] = sh.count[b], m[j] = sh.mass[b];
    }
    const uint64_t c_in = wave_scan(c[0] + c[1], lane), m_in = wave_scan(m[0] + m[1], lane);
    if (lane == 63) sh.part[wave] = c_in, sh.part2[wave] = m_in;
    if (tid == 0) sh.digit = 0xFFFFFFFFu;
    __syncthreads();
    uint64_t cb = above_count + c_in - c[0] - c[1], mb = above_mass + m_in - m[0] - m[1];
    for (int w = 0; w < wave; ++w) cb += sh.part[w], mb += sh.part2[w];
    for (int j = 0; j < per; ++j) {
      const uint64_t ca = cb + c[j], ma = mb + m[j];
      const bool was = by_count ? cb >= tokens : cb > 0 && (double)mb >= goal;
      const bool is = by_count ? ca >= tokens : ca > 0 && (double)ma >= goal;
      if (is && !was) {  // one digit of one thread
        sh.digit = bins - 1 - (per * tid + j);
        sh.before_count = (uint32_t)cb, sh.before_mass = mb, sh.digit_count = (uint32_t)c[j];
      }
      cb = ca, mb = ma;
    }
    __syncthreads();
    if (sh.digit == 0xFFFFFFFFu) return {0, 0, 0};  // not reached: all of them (uniform)
    prefix = prefix << kBits[level] | sh.digit;
    above_count = sh.before_count, above_mass = sh.before_mass;
    equal = sh.digit_count;
    __syncthreads();
  }
  Cut cut{prefix, 1, above_mass};
  if (by_count) {
    cut.ties = tokens - above_count;
  } else {
    const uint64_t w = sc.weight(value_of(prefix));
    const double need = goal - (double)above_mass;
    if (w > 0 && need > 0) cut.ties = (uint64_t)fmax(1.0, __builtin_ceil(need / (double)w));
  }
  cut.ties = min(cut.ties, (uint64_t)equal);
  return cut;
}

// Weight of the tokens above the cut and number of those equal to it, of [first, last), by one wave.
template <typename T>
__device__ void share_sums(const T* row, int first, int last, const Scale& sc, const Cut& cut, double min_p, uint64_t* mass, uint64_t* ties) {
  const int lane = threadIdx.x & 63;
  uint64_t m = 0, t = 0;
  for (int i = first + lane; i < last; i += 64) {
    const float x = (float)row[i];
    const uint32_t key = key_of(x);
    if (key == 0 || key < cut.key) continue;
    const double e = sc.e(x);
    if (!(e >= min_p)) continue;
    if (key == cut.key)
      ++t;
    else
      m += (uint64_t)__builtin_rint(e * (double)kOne);
  }
  *mass = wave_total(m), *ties = wave_total(t);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_kernel(tq_sample_args a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t r = blockIdx.x;
  const T* row = static_cast<const T*>(a.logits) + r * a.logit_stride;
  const int n = (int)a.vocab;

  // largest logit and its first place
  float best = -INFINITY;
  int at = 0x7FFFFFFF;
  for (int i = tid; i < n; i += kThreads) {
    const float x = (float)row[i];
    if (x > best) best = x, at = i;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float ox = __shfl_xor(best, o, 64);
    const int oa = __shfl_xor(at, o, 64);
    if (ox > best || (ox == best && oa < at)) best = ox, at = oa;
  }
  if (lane == 0) sh.best[wave] = best, sh.best_at[wave] = at;
  __syncthreads();
  best = sh.best[0], at = sh.best_at[0];
  for (int w = 1; w < kWaves; ++w)
    if (sh.best[w] > best || (sh.best[w] == best && sh.best_at[w] < at)) best = sh.best[w], at = sh.best_at[w];
  __syncthreads();
  if (!(best > -INFINITY)) {  // nothing to draw from
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.logprob) a.logprob[r] = -INFINITY;
    }
    return;
  }

  const float temperature = a.temperature ? a.temperature[r] : 1.0f;
  const bool greedy = !(temperature > 0.0f);
  const Scale sc{best, greedy ? 1.0 : 1.0 / (double)temperature};
  uint64_t all = 0;  // weight of the whole row
  const int64_t top_k = a.top_k ? a.top_k[r] : 0;
  const double top_p = a.top_p ? (double)a.top_p[r] : 1.0;
  const bool use_k = !greedy && top_k > 0 && top_k < n, use_p = !greedy && top_p < 1.0;
  if (a.logprob || (use_p && !use_k)) {
    uint64_t m = 0;
    for (int i = tid; i < n; i += kThreads) {
      const float x = (float)row[i];
      if (x > -INFINITY) m += sc.weight(x);
    }
    m = wave_total(m);
    if (lane == 0) sh.part[wave] = m;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) all += sh.part[w];
    __syncthreads();
  }

  int token = at;
  if (!greedy) {
    double min_p = a.min_p ? (double)a.min_p[r] : 0.0;
    min_p = min_p > 0.0 ? fmin(min_p, 1.0) : 0.0;
    Cut cut{0, 0, 0};
    uint64_t kept = all;
    if (use_k) {
      cut = find_cut(row, n, sc, true, (uint64_t)top_k, 0.0, sh);
      if (use_p && cut.key == 0) {  // fewer tokens than top_k: all of them
        uint64_t m = 0;
        for (int i = tid; i < n; i += kThreads) {
          const float x = (float)row[i];
          if (x > -INFINITY) m += sc.weight(x);
        }
        m = wave_total(m);
        if (lane == 0) sh.part[wave] = m;
        __syncthreads();
        kept = 0;
        for (int w = 0; w < kWaves; ++w) kept += sh.part[w];
        __syncthreads();
      } else {
        kept = cut.key ? cut.above + cut.ties * sc.weight(value_of(cut.key)) : 0;
      }
    }
    if (use_p) cut = find_cut(row, n, sc, false, 0, fmax(top_p, 0.0) * (double)kept, sh);

    // the draw: the share of the row that holds the place, its share, and the token
    const uint64_t tie_weight = cut.key ? sc.weight(value_of(cut.key)) : 0;
    int first = 0, last = n;
    uint64_t before = 0, ties_left = cut.ties, goal = 0;
    for (int level = 0; level < 2; ++level) {
      const int share = ((last - first + kWaves - 1) / kWaves + 63) / 64 * 64;
      const int lo = (int)min((int64_t)last, (int64_t)first + (int64_t)wave * share), hi = (int)min((int64_t)last, (int64_t)lo + share);
      uint64_t m, t;
      share_sums(row, lo, hi, sc, cut, min_p, &m, &t);
      if (lane == 0) sh.part[wave] = m, sh.part2[wave] = t;
      __syncthreads();
      uint64_t left = ties_left, sum = before;
      if (level == 0) {
        for (int w = 0; w < kWaves; ++w) {
          const uint64_t k = min(left, (uint64_t)sh.part2[w]);
          sum += sh.part[w] + k * tie_weight;
          left -= k;
        }
        const float u = a.u[r];
        goal = !(u > 0.0f) ? 0 : u >= 1.0f ? sum - 1 : (uint64_t)((double)u * (double)sum);
        goal = min(goal, sum - 1);
        left = ties_left, sum = before;
      }
      int pick = 0;
      for (int w = 0; w < kWaves; ++w) {
        const uint64_t k = min(left, (uint64_t)sh.part2[w]);
        const uint64_t after = sum + sh.part[w] + k * tie_weight;
        pick = w;
        if (after > goal) break;
        sum = after, left -= k;
      }
      before = sum, ties_left = left;
      const int nf = (int)min((int64_t)last, (int64_t)first + (int64_t)pick * share);
      last = (int)min((int64_t)last, (int64_t)nf + share), first = nf;
      __syncthreads();
    }
    if (wave == 0) {
      for (int i = first; i < last; i += 64) {
        const int p = i + lane;
        const float x = p < last ? (float)row[p] : -INFINITY;
        const uint32_t key = key_of(x);
        const double e = key ? sc.e(x) : 0.0;
        const bool stays = key != 0 && e >= min_p;
        const uint64_t equal = __ballot(stays && key == cut.key && cut.key != 0);
        const bool tie = equal >> lane & 1 && (uint64_t)__popcll(equal & ((uint64_t(1) << lane) - 1)) < ties_left;
        uint64_t w = 0;
        if (stays && (key > cut.key || tie)) w = (uint64_t)__builtin_rint(e * (double)kOne);
        const uint64_t sum = before + wave_scan(w, lane);
        const uint64_t over = __ballot(w > 0 && sum > goal);
        if (over) {
          token = i + __builtin_ctzll(over);
          break;
        }
        before = (uint64_t)__builtin_amdgcn_readlane((int)sum, 63) & 0xFFFFFFFFu;
        before |= (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(sum >> 32), 63) << 32;
        ties_left -= min(ties_left, (uint64_t)__popcll(equal));
      }
    }
  }
  if (tid == 0) {
    a.tokens[r] = token;
    if (a.logprob) a.logprob[r] = (float)(sc.z((float)row[token]) - log((double)all / (double)kOne));
  }
}

}  // namespace

int64_t sample_workspace_bytes(int64_t rows, int64_t vocab) { return 16; }

hipError_t launch_sample(const tq_sample_args& a, hipStream_t s) {
  const dim3 grid((unsigned)a.rows), block(kThreads);
  if (a.in_type == TQ_F32)
    hipLaunchKernelGGL((sample_kernel<float>), grid, block, 0, s, a);
  else if (a.in_type == TQ_BF16)
    hipLaunchKernelGGL((sample_kernel<bf16>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sample_kernel<f16>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace tq
