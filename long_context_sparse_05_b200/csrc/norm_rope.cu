// RMSNorm and rotation of the query heads and the latent row of each token, in one pass.
//
// Method: "DeepSeek V4 结构速览", section "HCA（c128a 路线）" (RMSNorm per head, RoPE on the
// last dims); the rotation and its float64 angle are the compressor's.
//
// Every element is read once and written once (2 x 2 bytes in bf16), and the arithmetic per row
// is one sum of squares and a scaling, which at this byte rate nearly fills the issue slots (76 %
// of them active, DRAM 55 %).  A warp owns whole rows (a head, or the latent row), kept in registers between the sum and the store: chunks of 8 elements, chunk
// lane + 32 i.  The rotary angles depend on the token only: the warp forms each pair's sine
// and cosine once per token (a float64 angle and one sincosf per lane) in its own piece of
// shared memory and every row of the token takes them from there.  Long inputs take four
// consecutive rows per warp, all loaded before the first is summed, with registers held to
// four CTAs an SM; short ones (too few rows for that to fill the SMs) take one.  4096 tokens
// of 64 heads of 512 (545 MB): 109 to 114 us, 4.8 to 5.0 TB/s (beside 109: one row per warp 137 us,
// two 114, four without the register bound 117); 16 tokens: 3.2 us.  Index queries, 64 heads of
// 128, leave half of a warp's lanes idle: 78 us for 136 MB.  float32: 252 us for 1.09 GB at 512
// dims (four rows just pass the 64 registers: 276 bytes a thread are spilled), 84 us for 273 MB
// at 128.

#include "chunk_common.cuh"

namespace csa {

namespace {

constexpr int kNrWarps = 8;

template <typename T> struct Chunk8;
template <> struct Chunk8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <> struct Chunk8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ static __forceinline__ void store(float* p, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// NV: chunks of 8 elements per lane (d <= 256 NV).  R: rows per warp.
template <typename T, int NV, int R>
__global__ void __launch_bounds__(32 * kNrWarps, NV <= 2 ? 4 : 1) norm_rope_kernel(NormRopeArgs a) {
  __shared__ float2 s_rot[kNrWarps][kMaxRopePairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nq = a.q ? a.H : 0;
  const int per = nq + (a.kv ? 1 : 0);            // rows per token: the heads, then the latent row
  const int total = a.N * per;
  const int r0 = (blockIdx.x * kNrWarps + warp) * R;
  if (r0 >= total) return;
  const int nchunk = a.d >> 3, rope0 = a.d - a.d_rope;
  Chunk8<T> x[R][NV];
  const int tok0 = r0 / per, hd0 = r0 - tok0 * per;
  int tok = tok0, hd = hd0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const T* src = hd < nq ? reinterpret_cast<const T*>(a.q) + tok * a.q_stride + (long long)hd * a.d
                           : reinterpret_cast<const T*>(a.kv) + tok * a.kv_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int ch = lane + 32 * j;
      if (ch < nchunk) x[i][j].load(src + 8 * ch);
      else x[i][j].zero();
    }
    if (r0 + i + 1 < total && ++hd == per) { hd = 0; ++tok; }   // past the end: the last row again
  }
  // sums of squares of all rows, then their reductions side by side
  float inv[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float ss = 0.f;
    if (a.norm) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float f[8];
        x[i][j].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
      }
    }
    inv[i] = ss;
  }
  if (a.norm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < R; ++i) inv[i] += __shfl_xor_sync(0xffffffffu, inv[i], o);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) inv[i] = a.norm ? 1.f / sqrtf(inv[i] / (float)a.d + a.eps) : 1.f;
  tok = tok0;
  hd = hd0;
  int rot_tok = -1;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (r0 + i >= total) break;
    if (a.d_rope > 0 && tok != rot_tok) {         // uniform over the warp
      rot_tok = tok;
      __syncwarp();
      const double t = (double)a.pos[rot_tok];
      for (int j = lane; 2 * j < a.d_rope; j += 32) {
        float sn, cs;
        rope_angle(t * a.inv_freq[j], &sn, &cs);
        s_rot[warp][j] = make_float2(sn, cs);
      }
      __syncwarp();
    }
    const bool is_q = hd < nq;
    const float* gain = is_q ? a.q_gain : a.kv_gain;
    T* dst = is_q ? reinterpret_cast<T*>(a.q_out) + ((long long)tok * a.H + hd) * a.d
                  : reinterpret_cast<T*>(a.kv_out) + (long long)tok * a.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int ch = lane + 32 * j;
      if (ch >= nchunk) continue;
      float f[8];
      x[i][j].get(f);
      if (gain) {
        const float4 g0 = *reinterpret_cast<const float4*>(gain + 8 * ch);
        const float4 g1 = *reinterpret_cast<const float4*>(gain + 8 * ch + 4);
        f[0] *= g0.x; f[1] *= g0.y; f[2] *= g0.z; f[3] *= g0.w;
        f[4] *= g1.x; f[5] *= g1.y; f[6] *= g1.z; f[7] *= g1.w;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv[i];
      if (a.d_rope > 0 && 8 * ch + 8 > rope0) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int u = 8 * ch + e - rope0;
          if (u >= 0) {
            const float2 sc = s_rot[warp][u >> 1];
            const float x0 = f[e], x1 = f[e + 1];
            f[e] = fmaf(x0, sc.y, -x1 * sc.x);
            f[e + 1] = fmaf(x0, sc.x, x1 * sc.y);
          }
        }
      }
      Chunk8<T>::store(dst + 8 * ch, f);
    }
    if (++hd == per) { hd = 0; ++tok; }
  }
}

template <typename T, int NV>
csa_status launch_nv(const NormRopeArgs& a, long long rows, cudaStream_t st) {
  // four rows per warp once one row each would give the 148 SMs more than two full waves
  constexpr int R = NV <= 2 ? 4 : 2;
  if (rows >= 148LL * 64 * 2) {
    const unsigned grid = (unsigned)((rows + kNrWarps * R - 1) / (kNrWarps * R));
    norm_rope_kernel<T, NV, R><<<grid, 32 * kNrWarps, 0, st>>>(a);
  } else {
    const unsigned grid = (unsigned)((rows + kNrWarps - 1) / kNrWarps);
    norm_rope_kernel<T, NV, 1><<<grid, 32 * kNrWarps, 0, st>>>(a);
  }
  CSA_CHECK_LAUNCH();
  return CSA_OK;
}

template <typename T>
csa_status launch_t(const NormRopeArgs& a, long long rows, cudaStream_t st) {
  if (a.d <= 256) return launch_nv<T, 1>(a, rows, st);
  if (a.d <= 512) return launch_nv<T, 2>(a, rows, st);
  if (a.d <= 1024) return launch_nv<T, 4>(a, rows, st);
  return launch_nv<T, 8>(a, rows, st);
}

}  // namespace

csa_status launch_norm_rope(NormRopeArgs& a, int dtype, double theta, cudaStream_t st) {
  rope_frequencies(a.inv_freq, a.d_rope, theta);
  const long long rows = (long long)a.N * ((a.q ? a.H : 0) + (a.kv ? 1 : 0));
  if (rows > 0x7fffffffLL - 64) return CSA_ERR_UNSUPPORTED;
  return dtype == CSA_F32 ? launch_t<float>(a, rows, st) : launch_t<__nv_bfloat16>(a, rows, st);
}

}  // namespace csa
