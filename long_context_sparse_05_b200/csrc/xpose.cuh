// Transpose-reductions over a warp: 32 values per lane reduced across the lanes, value L ending
// in lane L.
#pragma once

#include <cuda_runtime.h>

namespace csa {

// One halving step of the transpose-reduction: lanes with bit `OFF` set keep the
// upper half of their HALF live values, the others the lower half, and each
// combines what it keeps with what its partner sends.
template <bool kMax, int OFF, int HALF, int N>
__device__ __forceinline__ void xpose_step(float (&v)[N], int lane) {
  const bool hi = (lane & OFF) != 0;
#pragma unroll
  for (int i = 0; i < HALF; ++i) {
    const float send = hi ? v[i] : v[i + HALF];
    const float keep = hi ? v[i + HALF] : v[i];
    const float recv = __shfl_xor_sync(0xffffffffu, send, OFF);
    v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
  }
}

// Transpose-reduction of 32 values over the 32 lanes of a warp (31 shuffles):
// afterwards lane L holds the reduction of value L over the warp (v[0]).
template <bool kMax>
__device__ __forceinline__ void xpose_reduce32(float (&v)[32], int lane) {
  xpose_step<kMax, 16, 16>(v, lane);
  xpose_step<kMax, 8, 8>(v, lane);
  xpose_step<kMax, 4, 4>(v, lane);
  xpose_step<kMax, 2, 2>(v, lane);
  xpose_step<kMax, 1, 1>(v, lane);
}

}  // namespace csa
