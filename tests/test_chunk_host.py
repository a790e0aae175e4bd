"""Host side of the chunk calls, without a GPU: struct layouts against the header, and argument
errors that come back before any launch (fake pointers are never dereferenced)."""

import ctypes
import os
import subprocess
import sys
import tempfile

import pytest
import torch

from long_context_sparse_05_b200 import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
F = 1 << 20          # an aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    from long_context_sparse_05_b200 import build
    build.build()


def test_struct_layouts_match_c():
    structs = {"csa_kv_cache": L.KVCache, "csa_norm_rope_params": L.NormRopeParams}
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "csa.h"', "int main(void){"]
    for cname, py in structs.items():
        prog.append('printf("%s %%zu\\n", sizeof(%s));' % (cname, cname))
        for fname, _ in py._fields_:
            prog.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (cname, fname, cname, fname))
    prog.append("return 0;}")
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write("\n".join(prog))
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-I",
                               "/usr/local/cuda/include", c, "-o", exe])
        got = dict(x.split() for x in subprocess.check_output([exe], text=True).split("\n") if x)
    for cname, py in structs.items():
        assert int(got[cname]) == ctypes.sizeof(py), cname
        for fname, _ in py._fields_:
            assert int(got["%s.%s" % (cname, fname)]) == getattr(py, fname).offset, (cname, fname)


def cache(**over):
    v = dict(dtype=L.CSA_FP8_E4M3, c=512, d_hi=64, num_pages=4, max_pages=2, rows=F, hi=F, scales=F,
             block_table=F)
    v.update(over)
    return L.KVCache(**v)


BAD_CACHES = [dict(num_pages=0), dict(max_pages=0), dict(max_pages=1 << 24), dict(rows=None),
              dict(rows=F + 8), dict(block_table=None), dict(d_hi=8), dict(d_hi=-64), dict(d_hi=512),
              dict(c=500), dict(hi=None), dict(hi=F + 2), dict(scales=None), dict(scales=F + 4),
              dict(dtype=L.CSA_NVFP4), dict(dtype=9), dict(dtype=L.CSA_BF16),   # d_hi of a plain cache
              dict(dtype=L.CSA_BF16, d_hi=0, c=12), dict(dtype=L.CSA_F32, d_hi=0, c=0)]


@pytest.mark.parametrize("over", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(over):
    lib, kv = L.lib(), cache(**over)
    r = ctypes.byref(kv)
    assert lib.csa_cache_write(r, L.CSA_BF16, F, 512, F, F, 1, 4, None) == INVALID
    assert lib.csa_cache_read(r, F, F, 1, 4, L.CSA_BF16, F, None) == INVALID
    p = L.AttnParams(H=64, d=512, n_w=128, scale=1.0, m=4, k=8, dtype=L.CSA_BF16)
    assert lib.csa_chunk_attn(ctypes.byref(p), r, F, F, F, F, F, F, F, F, 1, 4, 64, F, F, F, 1 << 30,
                              None) == INVALID


def test_cache_write_refusals():
    w, kv = L.lib().csa_cache_write, ctypes.byref(cache())
    good = [kv, L.CSA_BF16, F, 512, F, F, 1, 4, None]
    for at, bad in ((1, L.CSA_FP8_E4M3), (2, None), (2, F + 8), (3, 511), (3, 516), (3, -512), (4, None),
                    (5, None), (6, -1), (7, -1)):
        args = list(good)
        args[at] = bad
        assert w(*args) == INVALID, (at, bad)
    assert w(None, *good[1:]) == INVALID
    assert w(kv, L.CSA_BF16, None, 0, None, None, 0, 4, None) == OK       # no sequences
    assert w(kv, L.CSA_BF16, None, 0, None, None, 3, 0, None) == OK       # no rows


def test_cache_read_refusals():
    r, kv = L.lib().csa_cache_read, ctypes.byref(cache())
    good = [kv, F, F, 1, 4, L.CSA_F32, F, None]
    for at, bad in ((3, -1), (4, -1), (5, L.CSA_FP8_E4M3), (6, None), (6, F + 4)):
        args = list(good)
        args[at] = bad
        assert r(*args) == INVALID, (at, bad)
    assert r(kv, None, None, 0, 4, L.CSA_F32, None, None) == OK
    assert r(kv, None, None, 4, 0, L.CSA_F32, None, None) == OK


def test_window_append_refusals():
    w = L.lib().csa_window_append
    good = [L.CSA_BF16, 512, 128, F, F, 512, F, F, 1, 4, None]
    for at, bad in ((0, L.CSA_FP8_E4M3), (1, 4), (1, 20), (2, 0), (3, None), (3, F + 2), (4, None), (4, F + 2),
                    (5, 8), (5, 513), (6, None), (7, None), (8, -1), (9, -1)):
        args = list(good)
        args[at] = bad
        assert w(*args) == INVALID, (at, bad)
    assert w(L.CSA_BF16, 512, 128, None, None, 0, None, None, 0, 0, None) == OK


def test_norm_rope_refusals():
    f = L.lib().csa_qk_norm_rope

    def call(q=F, qs=64 * 512, qg=F, kv=F, ks=512, kg=F, pos=F, N=4, qo=F, ko=F, **over):
        v = dict(H=64, d=512, d_rope=64, rope_theta=1e4, eps=1e-6, apply_norm=1, dtype=L.CSA_BF16)
        v.update(over)
        p = L.NormRopeParams(**v)
        return f(ctypes.byref(p), q, qs, qg, kv, ks, kg, pos, N, qo, ko, None)

    for bad in (dict(H=0), dict(d=4), dict(d=20), dict(d_rope=7), dict(d_rope=-2), dict(d_rope=514),
                dict(rope_theta=0.0), dict(rope_theta=-1.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(dtype=L.CSA_FP8_E4M3), dict(apply_norm=0), dict(N=-1), dict(q=F + 2), dict(qs=512),
                dict(qs=64 * 512 + 4), dict(kv=F + 8), dict(ks=256), dict(qo=None), dict(ko=None),
                dict(qo=F + 2), dict(qg=F + 4), dict(pos=None)):
        assert call(**bad) == INVALID, bad
    assert call(d=4096, qs=64 * 4096, ks=4096) == UNSUPPORTED
    assert call(d_rope=256) == UNSUPPORTED
    assert call(N=0) == OK
    assert call(q=None, kv=None, qo=None, ko=None) == OK
    assert f(None, F, 512, None, F, 512, None, F, 1, F, F, None) == INVALID


def test_chunk_attn_refusals():
    lib, f = L.lib(), L.lib().csa_chunk_attn
    names = ["q", "cu_q", "pos0", "idx", "count", "win", "new_win", "sink"]

    def call(b=1, N=4, L_max=64, out=F, lse=F, ws=F, ws_bytes=1 << 30, kv=None, **over):
        v = dict(H=64, d=512, n_w=128, scale=1.0, m=4, k=8, dtype=L.CSA_BF16)
        ptr = {n: F for n in names}
        for k, x in over.items():
            (ptr if k in ptr else v)[k] = x
        p = L.AttnParams(**v)
        return f(ctypes.byref(p), ctypes.byref(kv or cache()), *[ptr[n] for n in names], b, N, L_max, out,
                 lse, ws, ws_bytes, None)

    for bad in (dict(H=0), dict(d=4), dict(d=256), dict(n_w=-1), dict(m=0), dict(dtype=L.CSA_FP8_E4M3),
                dict(d_rope_out=3), dict(d_rope_out=-2), dict(d_rope_out=514), dict(d_rope_out=64),  # theta 0
                dict(b=-1), dict(N=-1), dict(L_max=0), dict(k=0), dict(k=-1), dict(idx=None), dict(count=None),
                dict(idx=None, count=None),                     # dense with k > 0
                dict(q=None), dict(q=F + 2), dict(cu_q=None), dict(pos0=None), dict(sink=None), dict(out=None),
                dict(out=F + 8), dict(win=None), dict(new_win=None), dict(win=F + 2), dict(new_win=F + 2),
                dict(kv=cache(dtype=L.CSA_F32, d_hi=0))):        # an fp32 cache under bf16 queries
        assert call(**bad) == INVALID, bad
    assert call(N=0) == OK and call(b=0) == OK
    p = L.AttnParams(H=64, d=512, n_w=128, scale=1.0, m=4, k=8, dtype=L.CSA_BF16)
    kv = cache()
    for a in ((0, 4, 64), (1, 0, 64), (1, 4, 0)):
        assert lib.csa_chunk_attn_workspace_size(ctypes.byref(p), ctypes.byref(kv), *a) == 0
    assert lib.csa_chunk_attn_workspace_size(None, None, 1, 1, 1) == 0


def test_binding_checks_types_places_and_sizes():
    with pytest.raises(L.CsaError):
        L.kv_cache(L.CSA_NVFP4, 512, 0, torch.zeros(256, 512), None, None, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(L.CsaError):      # not whole pages
        L.kv_cache(L.CSA_F32, 8, 0, torch.zeros(255, 8), None, None, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(L.CsaError):      # CPU tensors
        L.kv_cache(L.CSA_F32, 8, 0, torch.zeros(256, 8), None, None, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(L.CsaError):      # scales of a plain cache
        L.kv_cache(L.CSA_F32, 8, 0, torch.zeros(256, 8), None, torch.zeros(256, 8), torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(L.CsaError):
        L.csa_window_append(L.CSA_F32, 8, 4, torch.zeros(1, 4, 8), torch.zeros(2, 8), None, None, 1, 2)
    with pytest.raises(L.CsaError):
        L.csa_window_append(L.CSA_FP8_E4M3, 8, 4, None, None, None, None, 1, 2)


@pytest.mark.parametrize("m", [1, 4])
def test_workspace_of_the_longest_positions(m):
    """A bound of 2^31 - 1 positions (or one that only says "any") splits like one a tile shorter."""
    lib, kv = L.lib(), cache()
    p = L.AttnParams(H=64, d=512, n_w=128, scale=1.0, m=m, k=0, dtype=L.CSA_BF16)
    far = 2 ** 31 - 1
    for N in (1, 8, 150):
        size, launches = [[f(ctypes.byref(p), ctypes.byref(kv), 1, N, x) for x in (far, far - 128 * m)]
                          for f in (lib.csa_chunk_attn_workspace_size, lib.csa_chunk_attn_launch_count)]
        assert size[0] == size[1] > 0 and launches == [2, 2], (N, size, launches)


@pytest.mark.parametrize("k,m,n_w", [(0, 128, 128), (0, 4, 128), (512, 4, 128), (0, 4, 0), (4096, 4, 300)])
def test_workspace_bound_covers_every_smaller_call(k, m, n_w):
    """One workspace for a program's largest batch and context serves its smaller calls."""
    lib, kv = L.lib(), cache()
    p = L.AttnParams(H=64, d=512, n_w=n_w, scale=1.0, m=m, k=k, dtype=L.CSA_BF16)
    args = ctypes.byref(p), ctypes.byref(kv), 1
    for N, L_max in ((1, 1), (1, 1 << 14), (16, 1 << 15), (150, 1 << 15), (296, 1 << 15), (5000, 1 << 14)):
        bound = lib.csa_chunk_attn_workspace_bound(*args, N, L_max)
        # a context for each number of tiles: E entries, from 0 to the last
        most = max(lib.csa_chunk_attn_workspace_size(*args, n, x)
                   for n in range(1, min(N, 300) + 1)
                   for x in ([L_max] if k else [*range(1, L_max, 128 * m), L_max]))
        assert bound == most, (N, L_max, bound, most)
    for far in (1 << 24, 2 ** 31 - 1):               # too many tiles to try each: still a bound
        bound = lib.csa_chunk_attn_workspace_bound(*args, 296, far)
        assert all(lib.csa_chunk_attn_workspace_size(*args, n, x) <= bound
                   for n in range(1, 297) for x in (far, far // 2, far // 3, far // 1000))


def test_workspace_bound_of_nothing():
    f = L.lib().csa_chunk_attn_workspace_bound
    p = L.AttnParams(H=64, d=512, n_w=128, scale=1.0, m=4, k=0, dtype=L.CSA_BF16)
    for a in ((0, 4, 64), (1, 0, 64), (1, 4, 0)):
        assert f(ctypes.byref(p), ctypes.byref(cache()), *a) == 0
    assert f(None, None, 1, 1, 1) == 0
    p.H = 32                                         # the CUDA-core kernel takes none
    assert f(ctypes.byref(p), ctypes.byref(cache()), 1, 8, 1 << 20) == 0


def test_give_up_refusals():
    f = L.lib().csa_selftest_chunk_give_up
    assert f(0) == INVALID and f(4) == INVALID and f(-1) == INVALID


def test_the_package_imports_on_a_torch_without_cuda():
    """Such a build lacks the private CUDA functions of torch._C; the calls then say what is missing."""
    code = """
import torch
for n in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, n)
torch.cuda.is_available = torch.cuda.is_initialized = lambda: False
import long_context_sparse_05_b200 as csa
t = torch.zeros(1, 4, 8)
try:
    csa.csa_window_append(csa.CSA_F32, 8, 4, t, t[0], t, t, 1, 2)
except csa.CsaError as e:
    print("refused:", e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("refused:") and "CUDA" in r.stdout
