// sample_bins.h -- the bins of k_sample.hip: whole numbers that grow with a
// logit, 1/8 of z wide, and the same in every slice of a row.  The arithmetic
// alone, so that the host can go through its ends too
// (tests/host/sample_bins_check.cpp).
#pragma once
#include <math.h>

#ifdef __HIPCC__
#define TQ_BOTH __host__ __device__
#else
#define TQ_BOTH
#endif

namespace tq {

constexpr int kBins = 256;  // counted down from the bin of the largest logit
constexpr int kPerUnit = 8;

// Bins of a unit of x.  Never 0, also where 1 / temperature is (then +inf * 0 would have no bin): 2^-126 takes finite logits
// into the 8 bins around 0 and +inf behind them.
TQ_BOTH inline float bins_per(double inv_t) { return (float)fmax(fmin(kPerUnit * inv_t, 0x1p100), 0x1p-126); }

// The bin of a logit that is a number: floor(8 x / T), off by one at most for the rounding of the product.  What lies further
// from 0 than kFar shares a bin (and is searched otherwise if the cuts lie there).
constexpr float kFar = 0x1p23f;
TQ_BOTH inline float bin_place(float x, float per) {
#ifdef __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_fmed3f(x * per, -kFar, kFar);
#else
  const float v = x * per;
  return v != v ? -kFar : fminf(fmaxf(v, -kFar), kFar);  // (the median of three with a NaN is the least of them)
#endif
}
TQ_BOTH inline int bin_of(float x, float per) { return (int)floorf(bin_place(x, per)); }

// Whether distances of up to kBins from the bin of `best` are distances in z: not where bins_per is held at an end, nor where
// `best`, or what lies kBins below it, shares the bins at the ends.
TQ_BOTH inline bool bins_measure(float best, float per, double inv_t) {
  return kPerUnit * inv_t <= 0x1p100 && kPerUnit * inv_t >= 0x1p-126 && best * per < kFar && best * per > 2 * kBins - kFar;
}

// How far below `top` a bin lies: 0 to kBins, the last for all that are further down.  It is an index: held from both sides.
TQ_BOTH inline int bins_below(int top, int bin) {
  const int b = top - bin;
  return b < 0 ? 0 : b > kBins ? kBins : b;
}

}  // namespace tq
