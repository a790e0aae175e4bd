// Device helpers of the calls that serve a chunk of new tokens over a paged cache: which
// sequence a ragged row belongs to, and where an entry lives.
#pragma once

#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace csa {

// Sequence of ragged row r: the number of s in [1, b] with cu[s] <= r (a whole warp joins;
// 32 boundaries per step).  b when the row lies behind the last sequence.
__device__ __forceinline__ int find_seq(const int32_t* cu, int b, int r, int lane) {
  int s = 0;
  for (int base = 1; base <= b; base += kWarp) {
    const bool le = base + lane <= b && cu[base + lane] <= r;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    s += n;
    if (n < kWarp) break;   // ascending: later boundaries lie above r too
  }
  return s;
}

// Row of the pool holding entry e of sequence s, or -1 where the table or the pool has none.
__device__ __forceinline__ long long page_row(const csa_kv_cache& kv, int s, long long e) {
  if (e < 0 || e >= (long long)kv.max_pages * kPageEntries) return -1;
  const int pg = kv.block_table[(size_t)s * kv.max_pages + (size_t)(e / kPageEntries)];
  if ((unsigned)pg >= (unsigned)kv.num_pages) return -1;
  return (long long)pg * kPageEntries + (e % kPageEntries);
}

// Host: theta^(-2j/d_rope) for the d_rope / 2 rotary pairs, as powers of one root in extended
// precision (a call of pow for each pair was a microsecond of every small call).
inline void rope_frequencies(double* f, int d_rope, double theta) {
  const long double root = d_rope > 0 ? powl((long double)theta, -2.0L / d_rope) : 0.0L;
  long double x = 1.0L;
  for (int j = 0; 2 * j < d_rope; ++j, x *= root) f[j] = (double)x;
}

// The value of scale byte e: 2^(e - 127) (the byte is a float's exponent field).
__device__ __forceinline__ float scale_value(uint32_t e) { return __uint_as_float(e << 23); }

// Four E4M3 codes (one word, lowest byte first) as floats, times s.
__device__ __forceinline__ void e4m3x4_scaled(uint32_t w, float s, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * i] = v.x * s;
    f[2 * i + 1] = v.y * s;
  }
}

}  // namespace csa
