// lane_sums.h -- sums over the lanes of a wave and the threads of a workgroup, by moves
// within the vector registers (shared by kv_reserve.hip and kv_packed.hip).
#pragma once

#include <hip/hip_runtime.h>

namespace bcq {

// Sums of counts stop at 2^30: what a caller's arrays hold could pass 32 bits.
__device__ __forceinline__ int capped(int a, int b) {
  return (int)min((unsigned)a + (unsigned)b, 1u << 30);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int x) {  // 0 where nothing is moved to
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
// Inclusive sum over the lanes.
__device__ __forceinline__ int lane_scan(int x) {
  x = capped(x, moved<0x111, 0xf>(x));  // within 16 lanes
  x = capped(x, moved<0x112, 0xf>(x));
  x = capped(x, moved<0x114, 0xf>(x));
  x = capped(x, moved<0x118, 0xf>(x));
  x = capped(x, moved<0x142, 0xa>(x));  // the rows before
  return capped(x, moved<0x143, 0xc>(x));
}
__device__ __forceinline__ int last_lane(int x) { return __builtin_amdgcn_readlane(x, 63); }
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float x) {
  return __int_as_float(moved<CTRL, ROWS>(__float_as_int(x)));
}
__device__ __forceinline__ float lane_sum(float x) {
#pragma clang fp contract(off)
  x += moved<0x111, 0xf>(x);
  x += moved<0x112, 0xf>(x);
  x += moved<0x114, 0xf>(x);
  x += moved<0x118, 0xf>(x);
  x += moved<0x142, 0xa>(x);
  x += moved<0x143, 0xc>(x);
  return __int_as_float(last_lane(__float_as_int(x)));
}

// Inclusive sum over the workgroup's waves and the sum of all; `part` is free to be
// written.
template <int WAVES>
__device__ __forceinline__ int2 block_scan(int x, int *part) {
  const int wave = threadIdx.x >> 6;
  x = lane_scan(x);
  if ((threadIdx.x & 63) == 63) part[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int y = part[w];
    if (w < wave) before = capped(before, y);
    all = capped(all, y);
  }
  __syncthreads();
  return make_int2(capped(x, before), all);
}

}  // namespace bcq
