// lanes.h -- sums and maxima over the lanes of a wave by DPP moves, which take
// a tenth of what shuffles through LDS do: within rows of 16 lanes, then the
// rows' last lanes to the rows behind them.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#ifdef __HIPCC__
namespace tq {

template <int CTRL, int ROWS>
__device__ inline uint32_t lane_moved(uint32_t v) {  // 0 where no lane moves in
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS, typename V>
__device__ inline V lane_moved(V v) {
  static_assert(sizeof(V) == 8, "64-bit values");
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = lane_moved<CTRL, ROWS>((uint32_t)b), hi = lane_moved<CTRL, ROWS>((uint32_t)(b >> 32));
  return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
}

__device__ inline uint32_t lane_value(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
template <typename V>
__device__ inline V lane_value(V v, int lane) {
  static_assert(sizeof(V) == 8, "64-bit values");
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(V, (uint64_t)lane_value((uint32_t)(b >> 32), lane) << 32 | lane_value((uint32_t)b, lane));
}

// Sums over the lanes up to one's own: uint32_t, uint64_t or double.
template <typename V>
__device__ inline V wave_scan(V v) {
  v += lane_moved<0x111, 0xF>(v);  // row_shr:1
  v += lane_moved<0x112, 0xF>(v);
  v += lane_moved<0x114, 0xF>(v);
  v += lane_moved<0x118, 0xF>(v);
  v += lane_moved<0x142, 0xA>(v);  // row_bcast:15, to rows 1 and 3
  v += lane_moved<0x143, 0xC>(v);  // row_bcast:31, to rows 2 and 3
  return v;
}
template <typename V>
__device__ inline V wave_total(V v) {
  return lane_value(wave_scan(v), 63);
}

// The largest of a wave's values.
__device__ inline uint32_t wave_max_u32(uint32_t v) {
  v = max(v, lane_moved<0x111, 0xF>(v));
  v = max(v, lane_moved<0x112, 0xF>(v));
  v = max(v, lane_moved<0x114, 0xF>(v));
  v = max(v, lane_moved<0x118, 0xF>(v));
  v = max(v, lane_moved<0x142, 0xA>(v));
  v = max(v, lane_moved<0x143, 0xC>(v));
  return lane_value(v, 63);
}

}  // namespace tq
#endif
