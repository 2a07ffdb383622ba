// pq2_mfma.h -- operands of the int8 MFMA products of repacked pq2_0 units:
// code expansion, scale halves and raw buffer loads (k_gemm_pq2.hip,
// k_experts_pq2.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tq {

typedef int v4i __attribute__((ext_vector_type(4)));
// Native vector types (not HIP's uint4 struct) keep copies in registers.
typedef unsigned v4u __attribute__((ext_vector_type(4)));

// A code dword as 16 int8 weights of one row, times 64.
__device__ __forceinline__ v4i expand64(uint32_t d) {
  v4i a;
  a[0] = (int)((d << 6) & 0xC0C0C0C0u);
  a[1] = (int)((d << 4) & 0xC0C0C0C0u);
  a[2] = (int)((d << 2) & 0xC0C0C0C0u);
  a[3] = (int)(d & 0xC0C0C0C0u);
  return a;
}

__device__ __forceinline__ double lo_half(uint32_t p) {
  return (double)static_cast<float>(__builtin_bit_cast(_Float16, (uint16_t)(p & 0xffffu)));
}
__device__ __forceinline__ double hi_half(uint32_t p) {
  return (double)static_cast<float>(__builtin_bit_cast(_Float16, (uint16_t)(p >> 16)));
}

typedef __amdgpu_buffer_rsrc_t buf_t;
// A raw buffer resource over `bytes` bytes at p (stride 0, 32-bit data
// format word of gfx9-family targets).
__device__ __forceinline__ buf_t make_buf(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ v4u load16(buf_t r, int voff, int soff) {
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}
// Streamed once: non-temporal.
__device__ __forceinline__ v4u load16_nt(buf_t r, int voff, int soff) {
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 2));
}
__device__ __forceinline__ uint32_t load4(buf_t r, int voff, int soff) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
}

}  // namespace tq
