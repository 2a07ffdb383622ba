// lists.h -- tiles of pairs sorted by expert (or of tokens by adapter), found
// from the lists of tq_expert_lists.
//
// The host does not know how many pairs an expert has.  Tile i of expert e is
// slot offsets[e] / size + e + i: slots of different experts never meet, since
// floor((o + c) / size) + 1 >= floor(o / size) + ceil(c / size), and pairs / size
// + experts + 1 of them hold every tile.  With fewer pairs than that a slot is a
// place in the sorted list, and those whose place within its expert is a
// multiple of `size` have a tile.  The last "expert" is none.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "seq.h"

namespace tq {

struct Slots {
  int64_t count;
  bool places;  // slots are places of the list
};
inline Slots list_slots(int64_t pairs, int64_t experts, int size) {
  const int64_t n = pairs / size + experts + 1;
  return pairs < n ? Slots{pairs, true} : Slots{n, false};
}

#ifdef __HIPCC__
// A tile of the pairs of one expert: places `first` .. `first + count - 1` of the sorted list.
struct Tile {
  int expert, first, count;
};

// Held in [0, pairs], whatever the list holds.
__device__ inline int offset_at(const int32_t* offsets, int e, int pairs) { return min(max(offsets[e], 0), pairs); }

// Offsets that decrease or leave [0, pairs] raise the flag.  All of them are looked at, by the launch's threads together: a
// search for a slot passes most of them by.
__device__ inline void check_offsets(const int32_t* offsets, int experts, int pairs, int32_t* flag) {
  if (!flag) return;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i <= experts; i += (int64_t)gridDim.x * blockDim.x)
    if (offsets[i] < (i > 0 ? offsets[i - 1] : 0) || offsets[i] > pairs) raise_flag(flag);
}

// The tile of `slot`, by one wave: the last expert whose first slot is at most it.
__device__ inline Tile find_tile(const int32_t* offsets, int experts, int pairs, int size, bool places, int slot, int lane) {
  int lo = 0, n = experts + 1;  // the last is none
  while (n > 1) {
    const int step = (n + 63) / 64, i = lo + lane * step;
    bool ok = false;
    if (lane * step < n) {
      const int o = offset_at(offsets, i, pairs);
      ok = (places ? o : o / size + i) <= slot;
    }
    const int last = max(1, (int)__popcll(__ballot(ok))) - 1;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const int e = __builtin_amdgcn_readfirstlane(lo);
  const int begin = offset_at(offsets, e, pairs), end = e < experts ? max(begin, offset_at(offsets, e + 1, pairs)) : pairs;
  int first;
  if (places) {
    first = slot < begin || (slot - begin) % size ? end : slot;
  } else {
    const int64_t f = begin + (int64_t)(slot - (begin / size + e)) * size;
    first = f < begin || f > end ? end : (int)f;
  }
  return {e, first, max(0, min(size, end - first))};
}
#endif

}  // namespace tq
