// Host-side check of the bins that the sampler's kernels index with (csrc/sample_bins.h): for every temperature above 0, its
// infinity among them, and logits from the type's lowest to +inf, the bin of a larger logit is not lower, and the distances
// that become indexes stay in [0, kBins].  Prints how many pairs were seen and how many of them break that.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "../../bit_quantized_matvec_amd/csrc/sample_bins.h"

static float from_bits(uint32_t u) {
  float f;
  memcpy(&f, &u, 4);
  return f;
}

int main() {
  // the positive floats by exponent, with four significands each, 0 and the largest; their negatives; +inf
  std::vector<float> positive;
  for (uint32_t e = 0; e < 255; ++e)
    for (uint32_t m : {0x000001u, 0x2AAAABu, 0x555555u, 0x7FFFFFu}) positive.push_back(from_bits(e << 23 | m));
  std::vector<float> logits;
  for (size_t i = positive.size(); i-- > 0;) logits.push_back(-positive[i]);
  logits.push_back(0.0f);
  logits.insert(logits.end(), positive.begin(), positive.end());
  logits.push_back(INFINITY);
  std::vector<float> temperatures(positive);
  temperatures.push_back(INFINITY);

  long seen = 0, bad = 0;
  for (float t : temperatures) {
    const float per = tq::bins_per(1.0 / (double)t);
    bad += !(per > 0.0f && per < INFINITY);
    int before = tq::bin_of(logits[0], per);
    for (float x : logits) {
      const int bin = tq::bin_of(x, per), below = bin - before;
      bad += !(bin >= -(1 << 23) && bin <= 1 << 23) || x * per != x * per || below < 0;
      const int far = tq::bins_below(bin, before);  // `before` the lower one's
      bad += far < 0 || far > tq::kBins || (below < tq::kBins && far != below) || tq::bins_below(before, bin) != 0;
      before = bin;
      ++seen;
    }
    // the largest of a row at any place: no logit below it has a negative distance
    for (size_t i = 0; i < logits.size(); i += 7)
      for (size_t j = 0; j <= i; j += 13) {
        const int d = tq::bin_of(logits[i], per) - tq::bin_of(logits[j], per);
        bad += d < 0;
        ++seen;
      }
  }
  printf("%ld %ld\n", seen, bad);
  return 0;
}
