// Host side of the calls that serve a chunk of new tokens over a paged latent cache
// (include/csa.h): argument checks and kernel selection.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

using namespace csa;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool plain_type(int dt) { return dt == CSA_F32 || dt == CSA_BF16; }
inline int elem_bytes(int dt) { return dt == CSA_F32 ? 4 : 2; }

// Shape and pointers of a paged cache.
bool cache_ok(const csa_kv_cache* kv) {
  if (!kv || kv->num_pages < 1 || kv->max_pages < 1 || !kv->rows || !kv->block_table) return false;
  if (kv->max_pages > 0x7fffffff / kPageEntries) return false;   // entries are int32
  if (!aligned16(kv->rows)) return false;
  if (plain_type(kv->dtype)) return kv->c >= 8 && kv->c % 8 == 0 && kv->d_hi == 0;
  if (kv->dtype != CSA_FP8_E4M3) return false;
  if (kv->d_hi < 0 || kv->d_hi % 16 || kv->c - kv->d_hi < kScaleGroup ||
      (kv->c - kv->d_hi) % kScaleGroup)
    return false;
  if (!kv->scales || !aligned16(kv->scales)) return false;
  return kv->d_hi == 0 || (kv->hi && aligned16(kv->hi));
}

// Rows of n elements of type dt, `stride` elements apart, each starting on 16 bytes.
bool rows_ok(const void* x, int dt, int64_t stride, int64_t n) {
  return x && aligned16(x) && stride >= n && (stride * elem_bytes(dt)) % 16 == 0;
}

bool chunk_shape_ok(const csa_attn_params* p, const csa_kv_cache* kv, bool selected) {
  if (!p || !cache_ok(kv)) return false;
  if (p->H < 1 || p->d < 8 || p->d % 8 || p->n_w < 0 || p->m < 1) return false;
  if (!plain_type(p->dtype) || kv->c != p->d) return false;
  if (kv->dtype != p->dtype && kv->dtype != CSA_FP8_E4M3) return false;
  if (p->d_rope_out < 0 || p->d_rope_out % 2 || p->d_rope_out > p->d) return false;
  if (p->d_rope_out > 0 && !(p->rope_theta > 0.0)) return false;
  return !selected || p->k >= 1;
}

}  // namespace

extern "C" {

csa_status csa_cache_write(const csa_kv_cache* kv, int x_dtype, const void* x, int64_t x_stride,
                           const int32_t* cu_rows, const int32_t* first, int b, int rows,
                           cudaStream_t stream) {
  if (!cache_ok(kv) || !plain_type(x_dtype) || b < 0 || rows < 0) return CSA_ERR_INVALID_ARG;
  if (b == 0 || rows == 0) return CSA_OK;
  if (!cu_rows || !first || !rows_ok(x, x_dtype, x_stride, kv->c)) return CSA_ERR_INVALID_ARG;
  return launch_cache_write(*kv, x_dtype, RowsArgs{x, x_stride, cu_rows, first, b, rows}, stream);
}

csa_status csa_cache_read(const csa_kv_cache* kv, const int32_t* idx, const int32_t* count, int b,
                          int k, int out_dtype, void* out, cudaStream_t stream) {
  if (!cache_ok(kv) || !plain_type(out_dtype) || b < 0 || k < 0) return CSA_ERR_INVALID_ARG;
  if (b == 0 || k == 0) return CSA_OK;
  if (!out || !aligned16(out)) return CSA_ERR_INVALID_ARG;
  return launch_cache_read(*kv, idx, count, b, k, out_dtype, out, stream);
}

csa_status csa_window_append(int dtype, int c, int n_w, void* win, const void* x, int64_t x_stride,
                             const int32_t* cu_rows, const int32_t* first, int b, int rows,
                             cudaStream_t stream) {
  if (!plain_type(dtype) || c < 8 || c % 8 || n_w < 1 || b < 0 || rows < 0) return CSA_ERR_INVALID_ARG;
  if (b == 0 || rows == 0) return CSA_OK;
  if (!win || !aligned16(win) || !cu_rows || !first || !rows_ok(x, dtype, x_stride, c))
    return CSA_ERR_INVALID_ARG;
  return launch_window_append(dtype, c, n_w, win, RowsArgs{x, x_stride, cu_rows, first, b, rows},
                              stream);
}

csa_status csa_qk_norm_rope(const csa_norm_rope_params* p, const void* q, int64_t q_stride,
                            const float* q_gain, const void* kv, int64_t kv_stride,
                            const float* kv_gain, const int32_t* pos, int N, void* q_out,
                            void* kv_out, cudaStream_t stream) {
  if (!p || !plain_type(p->dtype) || p->H < 1 || p->d < 8 || p->d % 8) return CSA_ERR_INVALID_ARG;
  if (p->d_rope < 0 || p->d_rope % 2 || p->d_rope > p->d) return CSA_ERR_INVALID_ARG;
  if (p->d_rope > 0 && !(p->rope_theta > 0.0)) return CSA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || N < 0) return CSA_ERR_INVALID_ARG;
  if (!p->apply_norm && (q_gain || kv_gain)) return CSA_ERR_INVALID_ARG;
  if (p->d > 2048 || p->d_rope > 2 * kMaxRopePairs) return CSA_ERR_UNSUPPORTED;
  if (N == 0 || (!q && !kv)) return CSA_OK;
  if (q && (!q_out || !aligned16(q_out) || !rows_ok(q, p->dtype, q_stride, (int64_t)p->H * p->d)))
    return CSA_ERR_INVALID_ARG;
  if (kv && (!kv_out || !aligned16(kv_out) || !rows_ok(kv, p->dtype, kv_stride, p->d)))
    return CSA_ERR_INVALID_ARG;
  if ((q_gain && !aligned16(q_gain)) || (kv_gain && !aligned16(kv_gain))) return CSA_ERR_INVALID_ARG;
  if (p->d_rope > 0 && !pos) return CSA_ERR_INVALID_ARG;
  NormRopeArgs a{};
  a.q = q; a.kv = kv; a.q_out = q_out; a.kv_out = kv_out; a.q_stride = q_stride;
  a.kv_stride = kv_stride; a.q_gain = q_gain; a.kv_gain = kv_gain; a.pos = pos; a.H = p->H;
  a.d = p->d; a.d_rope = p->d_rope; a.N = N; a.norm = p->apply_norm ? 1 : 0; a.eps = p->eps;
  return launch_norm_rope(a, p->dtype, p->rope_theta, stream);
}

size_t csa_chunk_attn_workspace_size(const csa_attn_params* p, const csa_kv_cache* kv, int b, int N,
                                     int L_max) {
  if (!p || !kv || b <= 0 || N <= 0 || L_max < 1 || p->m < 1) return 0;
  if (!chunk_tc_supported(p->H, p->d, p->dtype, p->d_rope_out, *kv)) return 0;
  return chunk_tc_workspace_bytes(p->n_w, p->m, p->k, N, L_max);
}

size_t csa_chunk_attn_workspace_bound(const csa_attn_params* p, const csa_kv_cache* kv, int b, int N,
                                      int L_max) {
  if (!p || !kv || b <= 0 || N <= 0 || L_max < 1 || p->m < 1) return 0;
  if (!chunk_tc_supported(p->H, p->d, p->dtype, p->d_rope_out, *kv)) return 0;
  return chunk_tc_workspace_bound(p->n_w, p->m, p->k, N, L_max);
}

int csa_chunk_attn_launch_count(const csa_attn_params* p, const csa_kv_cache* kv, int b, int N,
                                int L_max) {
  if (!p || !kv || b <= 0 || N <= 0 || L_max < 1 || p->m < 1) return 0;
  if (!chunk_tc_supported(p->H, p->d, p->dtype, p->d_rope_out, *kv)) return 1;
  return chunk_tc_launch_count(p->n_w, p->m, p->k, N, L_max);
}

csa_status csa_selftest_chunk_give_up(int role) {
  return chunk_tc_give_up(role) ? CSA_OK : CSA_ERR_INVALID_ARG;
}

csa_status csa_chunk_attn(const csa_attn_params* p, const csa_kv_cache* kv, const void* q,
                          const int32_t* cu_q, const int32_t* pos0, const int32_t* idx,
                          const int32_t* count, const void* win, const void* new_win,
                          const float* sink, int b, int N, int L_max, void* out, float* lse,
                          void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!chunk_shape_ok(p, kv, idx != nullptr)) return CSA_ERR_INVALID_ARG;
  if (b < 0 || N < 0 || L_max < 1) return CSA_ERR_INVALID_ARG;
  // a selection needs k and count, dense attention neither (k = 0 tells the two apart in
  // the workspace size, where no pointer does)
  if ((idx != nullptr) != (p->k > 0) || (idx != nullptr) != (count != nullptr)) return CSA_ERR_INVALID_ARG;
  if (b == 0 || N == 0) return CSA_OK;
  if (!q || !cu_q || !pos0 || !sink || !out) return CSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out)) return CSA_ERR_INVALID_ARG;
  if (p->n_w > 0 && (!win || !new_win || !aligned16(win) || !aligned16(new_win)))
    return CSA_ERR_INVALID_ARG;
  ChunkArgs a{};
  a.q = q; a.cu_q = cu_q; a.pos0 = pos0; a.idx = idx; a.count = count; a.win = win;
  a.new_win = new_win; a.sink = sink; a.out = out; a.lse = lse; a.b = b; a.N = N; a.H = p->H;
  a.d = p->d; a.n_w = p->n_w; a.m = p->m; a.k = p->k; a.L_max = L_max;
  a.d_rope_out = p->d_rope_out; a.scale = p->scale; a.theta = p->rope_theta;
  if (chunk_tc_supported(p->H, p->d, p->dtype, p->d_rope_out, *kv)) {
    const csa_status st = launch_chunk_attn_tc(a, *kv, ws, ws_bytes, stream);
    if (st != CSA_ERR_UNSUPPORTED) return st;
  }
  return launch_chunk_attn_simt(a, *kv, p->dtype, stream);
}

}  // extern "C"
