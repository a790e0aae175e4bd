// The paged latent cache: rows written into their pages (quantised where the cache is),
// read back as plain rows, and appended to the window rings.
//
// Method: the pages of "DeepSeek-V4 技术解读", section 3.2 (a classical cache of blocks of
// compressed entries, a state of the sliding window); E4M3 codes per "DeepSeek V4
// 结构速览", section "Lightning Indexer" (low-precision caches), with a power-of-two scale
// per 64 dims, so that a code is one rounding of the value and code times scale is exact in
// bf16, and the rotary dims left in bf16.
//
// Bound by memory, the quantised kernels by instruction issue as well (67 to 77 % of the slots
// active): a quantised row of 512 dims is 584 bytes (448 codes, 64 bf16 dims, 7 scale
// exponents) against 1024 in bf16.  A warp owns a row: lane l takes 16 consecutive dims, so
// 512 dims are one pass of the warp, a scale group is four neighbouring lanes (two shuffles
// for its maximum) and codes leave as 16-byte stores.  Large calls take two rows per warp,
// both loaded before the first is used, with registers held to five CTAs an SM.  262,144 rows
// of 512 (421 MB): written 84 us, read back 80 us, 5.0 and 5.3 TB/s (four rows per warp 4 and 8 us
// more, one 4 and 20); 16 rows 2.3 us, a selection of 16 x 512 rows 4.9 us.  The same rows from
// float32 145 us, to float32 154 (690 MB).  Plain rows take one warp each: bf16 98 and 96 us
// (537 MB), float32 165 and 164 (1.07 GB, 6.5 TB/s).
#include "chunk_common.cuh"

namespace csa {

namespace {

constexpr int kLcWarps = 8;

// 16 consecutive elements in registers.
template <typename T> struct Run16;
template <> struct Run16<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v[0] = reinterpret_cast<const uint4*>(p)[0];
    v[1] = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[16]) const {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Run16<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i] = v[i].x; f[4 * i + 1] = v[i].y; f[4 * i + 2] = v[i].z; f[4 * i + 3] = v[i].w;
    }
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Scale exponent of a group whose largest magnitude is `amax`: the smallest k with
// amax <= 448 2^k = 1.75 2^(k+8), from amax's exponent and whether its significand is above
// 1.75 (0x600000 of the fraction field).  Subnormal maxima fall below the lowest exponent.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kScaleExpMin, min(k, kScaleExpMax));
}

// Rows r0 .. r0 + R - 1 of the ragged rows -> their rows in the pool, or -1 (whole warp).
// Neighbouring rows mostly share a sequence, so the search runs for the first alone.
template <int R>
__device__ __forceinline__ void dest_rows(long long (&at)[R], const csa_kv_cache& kv, const RowsArgs& a,
                                          int r0, int lane) {
  int s = find_seq(a.cu, a.b, r0, lane);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    while (s < a.b && r >= a.cu[s + 1]) ++s;
    at[i] = r >= a.rows || s >= a.b || r < a.cu[s]
                ? -1 : page_row(kv, s, (long long)a.first[s] + (r - a.cu[s]));
  }
}
__device__ __forceinline__ long long dest_row(const csa_kv_cache& kv, const RowsArgs& a, int r, int lane) {
  long long at[1];
  dest_rows(at, kv, a, r, lane);
  return at[0];
}

// FP8 rows.  T: type of x.  R: rows per warp.
template <typename T, int R>
__global__ void __launch_bounds__(32 * kLcWarps, 5) write_fp8_kernel(csa_kv_cache kv, RowsArgs a) {
  const int lane = threadIdx.x & 31;
  const int r0 = (blockIdx.x * kLcWarps + (threadIdx.x >> 5)) * R;
  if (r0 >= a.rows) return;
  const int live = min(a.rows, a.cu[a.b]);   // x may end there: `rows` is only a bound
  const int nc = kv.c - kv.d_hi, S = kv_scale_stride(kv.c, kv.d_hi);
  uint8_t* codes = static_cast<uint8_t*>(kv.rows);
  __nv_bfloat16* hi = static_cast<__nv_bfloat16*>(kv.hi);
  uint8_t* scales = static_cast<uint8_t*>(kv.scales);
  long long at[R];
  // c <= 512 is one pass; wider rows take the next 512 dims in another
  for (int c0 = 0; c0 < kv.c; c0 += 512) {
    const int ch = c0 + 16 * lane;
    Run16<T> x[R];
#pragma unroll
    for (int i = 0; i < R; ++i)   // the row's values do not depend on where it goes
      if (r0 + i < live && ch < kv.c)
        x[i].load(reinterpret_cast<const T*>(a.x) + (long long)(r0 + i) * a.x_stride + ch);
    if (c0 == 0) dest_rows(at, kv, a, r0, lane);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (at[i] < 0) continue;    // uniform over the warp
      float f[16];
      if (ch < kv.c) {
        x[i].get(f);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = 0.f;
      }
      float am = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) am = fmaxf(am, fabsf(f[e]));   // NaN never wins
      // 64 dims = 4 lanes, and a group never straddles the bf16 dims (nc % 64 == 0)
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      if (ch < nc) {
        const int k = scale_exp(am);
        const float inv = __uint_as_float((uint32_t)(127 - k) << 23);   // 2^-k, a normal number
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(
              make_float2(f[4 * q] * inv, f[4 * q + 1] * inv), __NV_SATFINITE, __NV_E4M3);
          const uint32_t h2 = __nv_cvt_float2_to_fp8x2(
              make_float2(f[4 * q + 2] * inv, f[4 * q + 3] * inv), __NV_SATFINITE, __NV_E4M3);
          w[q] = lo | (h2 << 16);
        }
        *reinterpret_cast<uint4*>(codes + at[i] * nc + ch) = make_uint4(w[0], w[1], w[2], w[3]);
        if ((lane & 3) == 0) scales[at[i] * S + ch / kScaleGroup] = (uint8_t)(k + 127);
      } else if (ch < kv.c) {
        store8(hi + at[i] * kv.d_hi + (ch - nc), f);
        store8(hi + at[i] * kv.d_hi + (ch - nc) + 8, f + 8);
      }
    }
  }
}

// Plain rows: x (type T) into rows of type U, chunks of 8 elements.  ring > 0: into slot
// (first + j) % ring of the sequence's ring instead of a page, the last `ring` rows only.
template <typename T, typename U>
__global__ void __launch_bounds__(32 * kLcWarps) write_plain_kernel(csa_kv_cache kv, RowsArgs a,
                                                                    int ring) {
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kLcWarps + (threadIdx.x >> 5);
  if (r >= a.rows) return;
  long long at;
  if (ring > 0) {
    const int s = find_seq(a.cu, a.b, r, lane);
    if (s >= a.b || r < a.cu[s] || r < a.cu[s + 1] - ring) return;
    const long long u = (long long)a.first[s] + (r - a.cu[s]);
    if (u < 0) return;
    at = (long long)s * ring + u % ring;
  } else {
    at = dest_row(kv, a, r, lane);
    if (at < 0) return;
  }
  const T* src = reinterpret_cast<const T*>(a.x) + (long long)r * a.x_stride;
  U* dst = static_cast<U*>(kv.rows) + at * kv.c;
  for (int ch = lane; ch < kv.c / 8; ch += 32) {
    float f[8];
    load8(src + 8 * ch, f);
    store8(dst + 8 * ch, f);
  }
}

// Slot (s, j) of the rows read -> its row in the pool, or -1.
__device__ __forceinline__ long long slot_row(const csa_kv_cache& kv, const int32_t* idx,
                                              const int32_t* count, int k, long long slot,
                                              long long slots) {
  if (slot >= slots) return -1;
  const int s = (int)(slot / k), j = (int)(slot - (long long)s * k);
  if (count && j >= count[s]) return -1;
  return page_row(kv, s, idx ? (long long)idx[slot] : (long long)j);
}

template <typename U, int R>
__global__ void __launch_bounds__(32 * kLcWarps, 5) read_fp8_kernel(csa_kv_cache kv, const int32_t* idx,
                                                                 const int32_t* count, int k,
                                                                 long long slots, U* out) {
  const int lane = threadIdx.x & 31;
  const long long s0 = ((long long)blockIdx.x * kLcWarps + (threadIdx.x >> 5)) * R;
  if (s0 >= slots) return;
  const int nc = kv.c - kv.d_hi, S = kv_scale_stride(kv.c, kv.d_hi);
  const uint8_t* codes = static_cast<const uint8_t*>(kv.rows);
  const __nv_bfloat16* hi = static_cast<const __nv_bfloat16*>(kv.hi);
  const uint8_t* scales = static_cast<const uint8_t*>(kv.scales);
  long long at[R];
#pragma unroll
  for (int i = 0; i < R; ++i) at[i] = slot_row(kv, idx, count, k, s0 + i, slots);
  for (int c0 = 0; c0 < kv.c; c0 += 512) {
    const int ch = c0 + 16 * lane;
    if (ch >= kv.c) break;
    uint4 v[R], v2[R];
    uint32_t e[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (at[i] < 0) continue;
      if (ch < nc) {
        v[i] = *reinterpret_cast<const uint4*>(codes + at[i] * nc + ch);
        e[i] = scales[at[i] * S + ch / kScaleGroup];
      } else {
        const uint4* p = reinterpret_cast<const uint4*>(hi + at[i] * kv.d_hi + (ch - nc));
        v[i] = p[0];
        v2[i] = p[1];
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (s0 + i >= slots) break;
      float f[16];
      if (at[i] < 0) {
#pragma unroll
        for (int x = 0; x < 16; ++x) f[x] = 0.f;
      } else if (ch < nc) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        const float sc = scale_value(e[i]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float g[4];
          e4m3x4_scaled(w[x], sc, g);
          f[4 * x] = g[0]; f[4 * x + 1] = g[1]; f[4 * x + 2] = g[2]; f[4 * x + 3] = g[3];
        }
      } else {
        Run16<__nv_bfloat16> r;
        r.v[0] = v[i]; r.v[1] = v2[i];
        r.get(f);
      }
      U* dst = out + (s0 + i) * kv.c + ch;
      store8(dst, f);
      store8(dst + 8, f + 8);
    }
  }
}

template <typename T, typename U>
__global__ void __launch_bounds__(32 * kLcWarps) read_plain_kernel(csa_kv_cache kv,
                                                                   const int32_t* idx,
                                                                   const int32_t* count, int k,
                                                                   long long slots, U* out) {
  const int lane = threadIdx.x & 31;
  const long long slot = (long long)blockIdx.x * kLcWarps + (threadIdx.x >> 5);
  if (slot >= slots) return;
  const long long at = slot_row(kv, idx, count, k, slot, slots);
  U* dst = out + slot * kv.c;
  for (int ch = lane; ch < kv.c / 8; ch += 32) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (at >= 0) load8(static_cast<const T*>(kv.rows) + at * kv.c + 8 * ch, f);
    store8(dst + 8 * ch, f);
  }
}

inline unsigned blocks(long long rows, int per_warp) {
  return (unsigned)((rows + (long long)kLcWarps * per_warp - 1) / ((long long)kLcWarps * per_warp));
}

// Rows enough that two per warp still give every SM a few waves of warps.
inline bool many(long long rows) { return rows >= 148LL * 64 * 4; }

template <typename T>
void write_t(const csa_kv_cache& kv, const RowsArgs& a, cudaStream_t st) {
  const int thr = 32 * kLcWarps;
  if (kv.dtype == CSA_FP8_E4M3) {
    constexpr int R = 2;
    if (many(a.rows)) write_fp8_kernel<T, R><<<blocks(a.rows, R), thr, 0, st>>>(kv, a);
    else write_fp8_kernel<T, 1><<<blocks(a.rows, 1), thr, 0, st>>>(kv, a);
  } else if (kv.dtype == CSA_BF16) {
    write_plain_kernel<T, __nv_bfloat16><<<blocks(a.rows, 1), thr, 0, st>>>(kv, a, 0);
  } else {
    write_plain_kernel<T, float><<<blocks(a.rows, 1), thr, 0, st>>>(kv, a, 0);
  }
}

template <typename U>
void read_t(const csa_kv_cache& kv, const int32_t* idx, const int32_t* count, int k,
            long long slots, U* out, cudaStream_t st) {
  const int thr = 32 * kLcWarps;
  if (kv.dtype == CSA_FP8_E4M3) {
    if (many(slots)) read_fp8_kernel<U, 2><<<blocks(slots, 2), thr, 0, st>>>(kv, idx, count, k, slots, out);
    else read_fp8_kernel<U, 1><<<blocks(slots, 1), thr, 0, st>>>(kv, idx, count, k, slots, out);
  } else if (kv.dtype == CSA_BF16) {
    read_plain_kernel<__nv_bfloat16, U><<<blocks(slots, 1), thr, 0, st>>>(kv, idx, count, k, slots, out);
  } else {
    read_plain_kernel<float, U><<<blocks(slots, 1), thr, 0, st>>>(kv, idx, count, k, slots, out);
  }
}

}  // namespace

csa_status launch_cache_write(const csa_kv_cache& kv, int x_dtype, const RowsArgs& a, cudaStream_t st) {
  if (x_dtype == CSA_F32) write_t<float>(kv, a, st);
  else write_t<__nv_bfloat16>(kv, a, st);
  CSA_CHECK_LAUNCH();
  return CSA_OK;
}

csa_status launch_cache_read(const csa_kv_cache& kv, const int32_t* idx, const int32_t* count, int b,
                             int k, int out_dtype, void* out, cudaStream_t st) {
  const long long slots = (long long)b * k;
  if (slots > 0x7fffffffLL * kLcWarps) return CSA_ERR_UNSUPPORTED;
  if (out_dtype == CSA_F32) read_t<float>(kv, idx, count, k, slots, static_cast<float*>(out), st);
  else read_t<__nv_bfloat16>(kv, idx, count, k, slots, static_cast<__nv_bfloat16*>(out), st);
  CSA_CHECK_LAUNCH();
  return CSA_OK;
}

csa_status launch_window_append(int dtype, int c, int n_w, void* win, const RowsArgs& a,
                                cudaStream_t st) {
  csa_kv_cache kv{};
  kv.dtype = dtype; kv.c = c; kv.rows = win;
  const int thr = 32 * kLcWarps;
  if (dtype == CSA_F32)
    write_plain_kernel<float, float><<<blocks(a.rows, 1), thr, 0, st>>>(kv, a, n_w);
  else
    write_plain_kernel<__nv_bfloat16, __nv_bfloat16><<<blocks(a.rows, 1), thr, 0, st>>>(kv, a, n_w);
  CSA_CHECK_LAUNCH();
  return CSA_OK;
}

}  // namespace csa
