// Attention of a chunk of new tokens over a paged cache, on CUDA cores: any head count and
// head dim, float32 or bf16, plain or FP8 rows.  It serves the small fp32 configuration and
// every shape the tensor-core kernel does not cover.
//
// Method: "DeepSeek Technical Reports", sections DSA and CSA; "DeepSeek V4 结构速览",
// sections "CSA（c4a 路线）" and "HCA（c128a 路线）": selected (or all visible) entries, then
// the sliding window, K = V, a sink per head in the denominator.
//
// One CTA per (token, head), one pass over the token's rows in tiles of 64: a warp per row
// forms the logit (lanes over the dims: coalesced), the running maximum and sum of the
// softmax carry over the tiles, and the threads accumulate the weighted rows: up to 128
// channels, several threads share a channel, each with every G-th row, in a register (64
// channels: 4 rows at a time); more channels, a thread takes some of them, in shared memory.
// The second reading of a tile's rows comes from L1 / L2.  Latency bound at the sizes it is
// for: 98 tokens of 4 heads of 64 dims, 32 rows each, 8.8 us.  Every head reads its rows again:
// 16 tokens of 512 chosen bf16 rows and the window take 238 us at 16 heads of 512 dims and 1,004
// at 128 (64 heads on the tensor cores: 25).
#include "chunk_common.cuh"

namespace csa {

namespace {

constexpr int kCsThreads = 256;
constexpr int kCsRows = 64;

// Element `e` of a pool row (FP8: codes, then the bf16 dims) or of a raw row.
template <typename T, bool FP8>
__device__ __forceinline__ float pool_elem(const csa_kv_cache& kv, long long row, int e, int nc, int S) {
  if (!FP8) return to_f32(static_cast<const T*>(kv.rows)[row * kv.c + e]);
  if (e >= nc)
    return to_f32(static_cast<const __nv_bfloat16*>(kv.hi)[row * kv.d_hi + (e - nc)]);
  return e4m3_to_f32(static_cast<const uint8_t*>(kv.rows)[row * nc + e]) *
         scale_value(static_cast<const uint8_t*>(kv.scales)[row * S + e / kScaleGroup]);
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(kCsThreads) chunk_simt_kernel(ChunkArgs a, csa_kv_cache kv) {
  extern __shared__ float sm[];
  float* s_q = sm;                       // [d] the head, scaled
  float* s_o = s_q + a.d;                // [d] running output
  float* s_l = s_o + a.d;                // [kCsRows] logits, then probabilities
  long long* s_row = reinterpret_cast<long long*>(s_l + kCsRows);   // [kCsRows]
  const int tok = blockIdx.x, h = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = find_seq(a.cu_q, a.b, tok, lane);
  if (s >= a.b || tok < a.cu_q[s]) return;          // behind the last sequence
  const int p0 = a.pos0[s], i0 = a.cu_q[s];
  const long long t = (long long)p0 + (tok - i0);
  const long long cap = (long long)kv.max_pages * kPageEntries;
  long long ns = a.idx ? (long long)a.count[tok] : (t + 1) / a.m;
  ns = t < 0 ? 0 : min(ns, a.idx ? (long long)a.k : cap);
  const int nsel = (int)max(0LL, ns);
  const long long w0 = max(0LL, t - a.n_w + 1);
  const int nwin = t >= 0 ? (int)(t - w0 + 1) : 0;
  const int R = nsel + nwin;
  const int nc = kv.c - kv.d_hi, S = FP8 ? kv_scale_stride(kv.c, kv.d_hi) : 0;
  const T* win = static_cast<const T*>(a.win);
  const T* nwr = static_cast<const T*>(a.new_win);

  const T* q = static_cast<const T*>(a.q) + ((long long)tok * a.H + h) * a.d;
  for (int e = threadIdx.x; e < a.d; e += kCsThreads) {
    s_q[e] = to_f32(q[e]) * a.scale;
    s_o[e] = 0.f;
  }
  float M = -INFINITY, l = 0.f;          // running maximum and sum, the same in every thread
  // few channels: thread (grp, ch) adds rows grp, grp + G, ... of channel ch in `part`
  const int G = a.d <= kCsThreads / 2 ? kCsThreads / a.d : 1;
  const int grp = threadIdx.x / a.d, ch = threadIdx.x - grp * a.d;
  float part = 0.f;
  for (int base = 0; base < R; base += kCsRows) {
    const int nr = min(kCsRows, R - base);
    __syncthreads();                     // the previous tile has been read; s_q is in place
    if (threadIdx.x < nr) {
      // >= 0: row of the pool; -1: none; -2 - x: row x of the rings; below -2^40: of new_win
      const int pos = base + threadIdx.x;
      long long code;
      if (pos < nsel) {
        code = page_row(kv, s, a.idx ? (long long)a.idx[(long long)tok * a.k + pos] : (long long)pos);
      } else {
        const long long u = w0 + (pos - nsel);
        code = u >= p0 ? -(1LL << 40) - 2 - (i0 + (u - p0)) : -2 - ((long long)s * a.n_w + u % a.n_w);
      }
      s_row[threadIdx.x] = code;
    }
    __syncthreads();
    for (int r = warp; r < nr; r += kCsThreads / 32) {
      const long long code = s_row[r];
      float dot = 0.f;
      if (code >= 0) {
        for (int e = lane; e < a.d; e += 32)
          dot = fmaf(s_q[e], pool_elem<T, FP8>(kv, code, e, nc, S), dot);
      } else if (code != -1) {
        const T* row = code < -(1LL << 40) ? nwr + (-(code + (1LL << 40)) - 2) * a.d : win + (-code - 2) * a.d;
        for (int e = lane; e < a.d; e += 32) dot = fmaf(s_q[e], to_f32(row[e]), dot);
      }
      dot = warp_sum(dot);
      if (lane == 0) s_l[r] = code == -1 ? -INFINITY : dot;
    }
    __syncthreads();
    float tm = -INFINITY;
    for (int r = lane; r < nr; r += 32) tm = fmaxf(tm, s_l[r]);
    const float Mn = fmaxf(M, warp_max(tm));
    const float ref = Mn == -INFINITY ? 0.f : Mn;       // nothing but masked rows so far
    const float al = M == -INFINITY ? 0.f : expf(M - ref);
    __syncthreads();                     // every warp has read the logits
    if (threadIdx.x < nr) s_l[threadIdx.x] = expf(s_l[threadIdx.x] - ref);
    __syncthreads();
    float ps = 0.f;
    for (int r = lane; r < nr; r += 32) ps += s_l[r];
    l = l * al + warp_sum(ps);
    M = Mn;
    auto value = [&](int r, int e) {
      const long long code = s_row[r];
      if (code >= 0) return pool_elem<T, FP8>(kv, code, e, nc, S);
      if (code == -1) return 0.f;
      return to_f32(code < -(1LL << 40) ? nwr[(-(code + (1LL << 40)) - 2) * a.d + e] : win[(-code - 2) * a.d + e]);
    };
    if (G > 1) {
      part *= al;
      if (grp < G)
        for (int r = grp; r < nr; r += G) part = fmaf(s_l[r], value(r, ch), part);
    } else {
      for (int e = threadIdx.x; e < a.d; e += kCsThreads) {
        float acc = s_o[e] * al;
        for (int r = 0; r < nr; ++r) acc = fmaf(s_l[r], value(r, e), acc);
        s_o[e] = acc;
      }
    }
  }
  if (G > 1) {                           // the groups' parts, in order
    for (int g = 0; g < G; ++g) {
      __syncthreads();
      if (grp == g) s_o[ch] += part;
    }
  }
  __syncthreads();
  // the sink joins the denominator; with neither rows nor a sink the output is zero
  const float sink = a.sink[h];
  const float top = fmaxf(M, sink);
  const float wr = M == -INFINITY ? 0.f : expf(M - top);
  const float den = l * wr + (sink == top && top != -INFINITY ? 1.f : sink == -INFINITY ? 0.f : expf(sink - top));
  const float inv = den > 0.f || den != den ? wr / den : 0.f;
  T* o = static_cast<T*>(a.out) + ((long long)tok * a.H + h) * a.d;
  const int rope0 = a.d - a.d_rope_out;
  for (int e = threadIdx.x; e < rope0 + a.d_rope_out / 2; e += kCsThreads) {
    if (e < rope0) {
      o[e] = from_f32<T>(s_o[e] * inv);
    } else {
      const int j = e - rope0, c0 = rope0 + 2 * j;
      float sn, cs;
      rope_angle((double)t * pow(a.theta, -2.0 * (double)j / (double)a.d_rope_out), &sn, &cs);
      const float x0 = s_o[c0] * inv, x1 = s_o[c0 + 1] * inv;
      o[c0] = from_f32<T>(inv_rope_elem(x0, x1, c0, a.d, a.d_rope_out, sn, cs));
      o[c0 + 1] = from_f32<T>(inv_rope_elem(x1, x0, c0 + 1, a.d, a.d_rope_out, sn, cs));
    }
  }
  if (a.lse && threadIdx.x == 0) a.lse[(long long)tok * a.H + h] = den > 0.f || den != den ? top + logf(den) : -INFINITY;
}

}  // namespace

csa_status launch_chunk_attn_simt(const ChunkArgs& a, const csa_kv_cache& kv, int dtype,
                                  cudaStream_t st) {
  if (a.H > 65535) return CSA_ERR_UNSUPPORTED;
  const size_t smem = (size_t)(2 * a.d + kCsRows) * 4 + kCsRows * 8 + 8;
  if (smem > 200 * 1024) return CSA_ERR_UNSUPPORTED;
  const bool fp8 = kv.dtype == CSA_FP8_E4M3;
  auto kern = dtype == CSA_F32 ? (fp8 ? chunk_simt_kernel<float, true> : chunk_simt_kernel<float, false>)
                               : (fp8 ? chunk_simt_kernel<__nv_bfloat16, true>
                                      : chunk_simt_kernel<__nv_bfloat16, false>);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return CSA_ERR_CUDA;
  kern<<<dim3((unsigned)a.N, (unsigned)a.H), kCsThreads, smem, st>>>(a, kv);
  CSA_CHECK_LAUNCH();
  return CSA_OK;
}

}  // namespace csa
