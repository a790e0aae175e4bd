"""The cache's write kernels on the CPU: their source compiled for the host, a warp's lanes as
threads.  The rows written lie at the very end of a mapping whose next page may not be touched, so
that a read past the last sequence's rows, up to the call's bound, ends the program."""

import os
import re
import subprocess

import numpy as np
import pytest

from oracle import chunk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_sparse_05_b200", "csrc")

PRELUDE = r"""
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <pthread.h>
#include <sys/mman.h>
#include <thread>
#include <vector>
#include <cuda_runtime_api.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_fp4.h>
using std::max;
using std::min;
#undef __launch_bounds__
#define __launch_bounds__(...)
struct Dim { unsigned x; };
thread_local Dim threadIdx, blockIdx, blockDim;
inline void __syncthreads() { std::abort(); }    // (no kernel here has one)
static uint32_t g_slot[32];
static pthread_barrier_t g_bar;
static uint32_t exchange(uint32_t v, int from) {
  const int lane = threadIdx.x & 31;
  g_slot[lane] = v;
  pthread_barrier_wait(&g_bar);
  const uint32_t r = g_slot[from];
  pthread_barrier_wait(&g_bar);
  return r;
}
template <class T> T __shfl_xor_sync(unsigned, T v, int o) {
  uint32_t u;
  std::memcpy(&u, &v, 4);
  u = exchange(u, (threadIdx.x & 31) ^ o);
  std::memcpy(&v, &u, 4);
  return v;
}
static unsigned __ballot_sync(unsigned, bool p) {
  unsigned r = 0;
  g_slot[threadIdx.x & 31] = p;
  pthread_barrier_wait(&g_bar);
  for (int i = 0; i < 32; ++i) r |= g_slot[i] << i;
  pthread_barrier_wait(&g_bar);
  return r;
}
static int __popc(unsigned x) { return __builtin_popcount(x); }
static uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
static float __uint_as_float(uint32_t u) { float f; std::memcpy(&f, &u, 4); return f; }
extern "C" cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
"""

MAIN = r"""
using namespace csa;
template <class F> static void grid(unsigned blocks, F f) {
  for (unsigned b = 0; b < blocks; ++b)
    for (unsigned w = 0; w < 8; ++w) {
      std::vector<std::thread> lanes;
      for (unsigned l = 0; l < 32; ++l)
        lanes.emplace_back([=] { threadIdx.x = 32 * w + l; blockIdx.x = b; f(); });
      for (auto& t : lanes) t.join();
    }
}
// argv: input file (float32 rows), output file, c, d_hi, cache type, x type, rows a warp, bound, ring
int main(int, char** v) {
  const int c = atoi(v[3]), d_hi = atoi(v[4]), fmt = atoi(v[5]), xt = atoi(v[6]), R = atoi(v[7]);
  const int bound = atoi(v[8]), ring = atoi(v[9]), n = 5;
  pthread_barrier_init(&g_bar, nullptr, 32);
  std::vector<float> in((size_t)n * c);
  FILE* f = fopen(v[1], "rb");
  if (fread(in.data(), 4, in.size(), f) != in.size()) return 1;
  fclose(f);
  const size_t bytes = in.size() * (xt == CSA_F32 ? 4 : 2), page = 4096;
  const size_t span = (bytes + page - 1) / page * page;
  char* m = (char*)mmap(nullptr, span + page, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
  mprotect(m + span, page, PROT_NONE);
  char* x = m + span - bytes;
  for (size_t i = 0; i < in.size(); ++i) {
    if (xt == CSA_F32) ((float*)x)[i] = in[i];
    else ((__nv_bfloat16*)x)[i] = __float2bfloat16_rn(in[i]);
  }
  const size_t slots = kPageEntries;
  std::vector<char> rows(slots * c * 4), hi(slots * 512 * 2), sc(slots * 64);
  const int32_t cu[4] = {0, 2, 2, n}, first[3] = {3, 0, 100}, bt[3] = {0, 0, 0};
  csa_kv_cache kv{};
  kv.dtype = fmt; kv.c = c; kv.d_hi = d_hi; kv.num_pages = 1; kv.max_pages = 1;
  kv.rows = rows.data(); kv.hi = hi.data(); kv.scales = sc.data(); kv.block_table = bt;
  const RowsArgs a{x, c, cu, first, 3, bound};
  grid((bound + 8 * R - 1) / (8 * R), [=] {
    if (fmt == CSA_FP8_E4M3) {
      if (xt == CSA_F32) R == 2 ? write_fp8_kernel<float, 2>(kv, a) : write_fp8_kernel<float, 1>(kv, a);
      else R == 2 ? write_fp8_kernel<__nv_bfloat16, 2>(kv, a) : write_fp8_kernel<__nv_bfloat16, 1>(kv, a);
    } else if (xt == CSA_F32) {
      write_plain_kernel<float, float>(kv, a, ring);
    } else {
      write_plain_kernel<__nv_bfloat16, __nv_bfloat16>(kv, a, ring);
    }
  });
  f = fopen(v[2], "wb");
  fwrite(rows.data(), 1, rows.size(), f);
  fclose(f);
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src = open(os.path.join(CSRC, "latent_cache.cu")).read()
    src = re.sub(r"<<<.*?>>>", "", src, flags=re.S)      # (the launchers are not called)
    (d / "rows.cpp").write_text(PRELUDE + src + MAIN)
    exe = d / "rows"
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-pthread", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", "/usr/local/cuda/include", str(d / "rows.cpp"), "-o", str(exe)], check=True, timeout=300)
    return exe


@pytest.mark.parametrize("fmt,d_hi,x_dtype,R,ring", [
    (2, 64, 1, 1, 0), (2, 64, 1, 2, 0), (2, 64, 0, 1, 0), (2, 64, 0, 2, 0),
    (1, 0, 1, 1, 0), (0, 0, 0, 1, 0), (1, 0, 1, 1, 128), (0, 0, 0, 1, 16),
])
@pytest.mark.parametrize("bound", [5, 6, 40])
def test_rows_behind_the_last_sequence_are_not_read(program, tmp_path, fmt, d_hi, x_dtype, R, ring, bound):
    c = 512
    x = np.random.default_rng(1).standard_normal((5, c)).astype(np.float32)
    x = (x.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)    # bf16 values
    x.tofile(tmp_path / "x")
    r = subprocess.run([str(program), str(tmp_path / "x"), str(tmp_path / "o"), str(c), str(d_hi), str(fmt),
                        str(x_dtype), str(R), str(bound), str(ring)], timeout=120)
    assert r.returncode == 0, "a row behind the last sequence was read" if r.returncode < 0 else r.returncode
    if ring:
        return
    out = np.fromfile(tmp_path / "o", np.uint8)
    # entries 3, 4 of sequence 0 and 100 .. 102 of sequence 2, whose tables share the page
    for row, entry in zip(range(5), (3, 4, 100, 101, 102)):
        if fmt == 2:
            w = c - d_hi
            assert np.array_equal(out[entry * w:(entry + 1) * w], chunk.quant_row(x[row].astype(np.float64), d_hi)[0])
        else:
            w = c * (4 if fmt == 0 else 2)
            want = x[row].view(np.uint32) >> 16 if fmt == 1 else x[row].view(np.uint32)
            assert np.array_equal(out[entry * w:(entry + 1) * w], want.astype(np.uint16 if fmt == 1 else np.uint32).view(np.uint8))
