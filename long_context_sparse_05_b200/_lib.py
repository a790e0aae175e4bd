"""ctypes binding of libcsa.so (the C ABI in include/csa.h).

Argument marshalling only: torch tensors become device pointers, Python
numbers become C scalars, the stream defaults to torch's current stream.
Every computation happens in the CUDA library; if it is missing or fails to
load, every call raises.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

CSA_F32, CSA_BF16, CSA_FP8_E4M3, CSA_NVFP4 = 0, 1, 2, 3
DTYPE = {"f32": CSA_F32, "bf16": CSA_BF16, "fp8": CSA_FP8_E4M3, "nvfp4": CSA_NVFP4}

c_int, c_float, c_double, c_size_t, c_void_p = (ctypes.c_int, ctypes.c_float, ctypes.c_double,
                                                 ctypes.c_size_t, ctypes.c_void_p)


class CsaError(RuntimeError):
    pass


class CompressParams(ctypes.Structure):
    _fields_ = [("m", c_int), ("overlap", c_int), ("c", c_int), ("d_rope", c_int),
                ("rope_theta", c_double), ("eps", c_float), ("apply_norm", c_int),
                ("in_dtype", c_int), ("out_dtype", c_int), ("out_entry_offset", c_int)]


class IndexParams(ctypes.Structure):
    _fields_ = [("H_I", c_int), ("d_I", c_int), ("m", c_int), ("qk_dtype", c_int),
                ("score_dtype", c_int)]


class AttnParams(ctypes.Structure):
    _fields_ = [("H", c_int), ("d", c_int), ("n_w", c_int), ("scale", c_float), ("m", c_int),
                ("k", c_int), ("dtype", c_int), ("d_rope_out", c_int), ("rope_theta", c_double)]


class DecodeParams(ctypes.Structure):
    _fields_ = [("b", c_int), ("L", c_int), ("m", c_int), ("c", c_int), ("H", c_int),
                ("c_I", c_int), ("H_I", c_int), ("d_rope", c_int), ("d_rope_I", c_int),
                ("rope_theta", c_double), ("eps", c_float), ("k", c_int), ("n_w", c_int),
                ("scale", c_float), ("kv_dtype", c_int), ("idx_dtype", c_int), ("hca", c_int),
                ("E_cap", c_int), ("mode", c_int), ("P", c_int), ("inv_rope", c_int)]


CSA_MODE_FULL, CSA_MODE_REUSE, CSA_MODE_REINDEX = 0, 1, 2


_DECODE_TENSORS = ["C_a", "Z_a", "C_b", "Z_b", "B_a", "B_b", "CI_a", "ZI_a", "CI_b", "ZI_b",
                   "BI_a", "BI_b", "kv_cache", "kI_cache", "kI_scales", "kv_win", "q", "q_I", "w",
                   "sink", "out", "lse", "idx_out", "count_out", "idx_in", "count_in", "pool",
                   "pool_count"]


class DecodeTensors(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in _DECODE_TENSORS]


class PagedParams(ctypes.Structure):
    _fields_ = [("b", c_int), ("m", c_int), ("c", c_int), ("H", c_int), ("c_I", c_int),
                ("H_I", c_int), ("d_rope", c_int), ("d_rope_I", c_int), ("rope_theta", c_double),
                ("eps", c_float), ("k", c_int), ("n_w", c_int), ("scale", c_float),
                ("kv_dtype", c_int), ("idx_dtype", c_int), ("hca", c_int), ("max_pages", c_int),
                ("num_pages", c_int), ("L_max", c_int), ("inv_rope", c_int)]


_PAGED_TENSORS = ["kv_pages", "kI_pages", "kI_scales", "block_table", "win", "tail_C_a",
                  "tail_Z_a", "tail_C_b", "tail_Z_b", "tail_CI_a", "tail_ZI_a", "tail_CI_b",
                  "tail_ZI_b", "pos", "new_C_a", "new_Z_a", "new_C_b", "new_Z_b", "new_CI_a",
                  "new_ZI_a", "new_CI_b", "new_ZI_b", "new_win", "B_a", "B_b", "BI_a", "BI_b",
                  "q", "q_I", "w", "sink", "out", "lse", "idx_out", "count_out"]


class PagedTensors(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in _PAGED_TENSORS]


PAGE_ENTRIES = 256


class PrefillParams(ctypes.Structure):
    _fields_ = [("b", c_int), ("n", c_int), ("m", c_int), ("c", c_int), ("H", c_int),
                ("c_I", c_int), ("H_I", c_int), ("d_rope", c_int), ("d_rope_I", c_int),
                ("rope_theta", c_double), ("eps", c_float), ("k", c_int), ("n_w", c_int),
                ("scale", c_float), ("kv_dtype", c_int), ("idx_dtype", c_int),
                ("score_dtype", c_int), ("inv_rope", c_int)]


_PREFILL_TENSORS = ["C_a", "Z_a", "C_b", "Z_b", "B_a", "B_b", "CI_a", "ZI_a", "CI_b", "ZI_b",
                    "BI_a", "BI_b", "kv_win", "q", "q_I", "w", "sink", "kv_cache", "kI_cache",
                    "kI_scales", "out", "lse", "idx_out", "count_out"]


class PrefillTensors(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in _PREFILL_TENSORS]


class KVCache(ctypes.Structure):
    """csa_kv_cache; made by kv_cache(), which keeps the arrays alive."""
    _fields_ = [("dtype", c_int), ("c", c_int), ("d_hi", c_int), ("num_pages", c_int),
                ("max_pages", c_int), ("rows", c_void_p), ("hi", c_void_p), ("scales", c_void_p),
                ("block_table", c_void_p)]


class NormRopeParams(ctypes.Structure):
    _fields_ = [("H", c_int), ("d", c_int), ("d_rope", c_int), ("rope_theta", c_double),
                ("eps", c_float), ("apply_norm", c_int), ("dtype", c_int)]


SCALE_GROUP = 64   # dims sharing one scale of an FP8 cache row

_lib = None

_SIGS = {
    "csa_status_string": (ctypes.c_char_p, [c_int]),
    "csa_version": (c_int, []),
    "csa_device_error": (c_int, [c_void_p]),
    "csa_selftest_bounded_wait": (c_int, [c_int, c_void_p]),
    "csa_compress": (c_int, [ctypes.POINTER(CompressParams)] + [c_void_p] * 6 +
                     [c_int] * 5 + [c_void_p, c_void_p, c_void_p]),
    "csa_quantize": (c_int, [c_int, c_int, c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "csa_index_scores": (c_int, [ctypes.POINTER(IndexParams)] + [c_void_p] * 6 + [c_int] * 4 +
                         [c_void_p, c_void_p]),
    "csa_topk": (c_int, [c_void_p, c_int, c_void_p, c_int, c_int, c_int, c_int, c_int, c_void_p,
                         c_void_p, c_void_p, c_size_t, c_void_p]),
    "csa_topk_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "csa_pool_topk": (c_int, [ctypes.POINTER(IndexParams)] + [c_void_p] * 6 + [c_int] * 4 +
                      [c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_size_t,
                       c_void_p]),
    "csa_pool_topk_workspace_size": (c_size_t, [ctypes.POINTER(IndexParams), c_int, c_int, c_int,
                                                c_int]),
    "csa_out_proj": (c_int, [c_void_p, c_void_p] + [c_int] * 5 + [c_void_p, c_void_p, c_size_t,
                                                                 c_void_p]),
    "csa_out_proj_workspace_size": (c_size_t, [c_int] * 5),
    "csa_sparse_attn": (c_int, [ctypes.POINTER(AttnParams), c_void_p, c_void_p, c_int, c_void_p,
                                c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int,
                                c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "csa_sparse_attn_workspace_size": (c_size_t, [ctypes.POINTER(AttnParams), c_int, c_int, c_int]),
    "csa_sparse_attn_noalloc": (c_int, [ctypes.POINTER(AttnParams), c_void_p, c_void_p, c_int,
                                        c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p,
                                        c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "csa_decode": (c_int, [ctypes.POINTER(DecodeParams), ctypes.POINTER(DecodeTensors), c_void_p,
                           c_size_t, c_void_p]),
    "csa_decode_workspace_size": (c_size_t, [ctypes.POINTER(DecodeParams)]),
    "csa_prefill": (c_int, [ctypes.POINTER(PrefillParams), ctypes.POINTER(PrefillTensors),
                            c_void_p, c_size_t, c_void_p]),
    "csa_prefill_workspace_size": (c_size_t, [ctypes.POINTER(PrefillParams)]),
    "csa_decode_launch_count": (c_int, [ctypes.POINTER(DecodeParams)]),
    "csa_decode_paged": (c_int, [ctypes.POINTER(PagedParams), ctypes.POINTER(PagedTensors),
                                 c_void_p, c_size_t, c_void_p]),
    "csa_decode_paged_workspace_size": (c_size_t, [ctypes.POINTER(PagedParams)]),
    "csa_decode_paged_launch_count": (c_int, [ctypes.POINTER(PagedParams)]),
    "csa_prefill_launch_count": (c_int, [ctypes.POINTER(PrefillParams)]),
    "csa_cp_candidates": (c_int, [c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_int,
                                  c_void_p, c_void_p, c_void_p]),
    "csa_cp_merge_workspace_size": (c_size_t, [c_int, c_int, c_int]),
    "csa_cp_merge": (c_int, [c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p,
                             c_void_p, c_size_t, c_void_p]),
    "csa_cache_write": (c_int, [ctypes.POINTER(KVCache), c_int, c_void_p, ctypes.c_int64, c_void_p,
                                c_void_p, c_int, c_int, c_void_p]),
    "csa_cache_read": (c_int, [ctypes.POINTER(KVCache), c_void_p, c_void_p, c_int, c_int, c_int,
                               c_void_p, c_void_p]),
    "csa_window_append": (c_int, [c_int, c_int, c_int, c_void_p, c_void_p, ctypes.c_int64, c_void_p,
                                  c_void_p, c_int, c_int, c_void_p]),
    "csa_qk_norm_rope": (c_int, [ctypes.POINTER(NormRopeParams), c_void_p, ctypes.c_int64, c_void_p,
                                 c_void_p, ctypes.c_int64, c_void_p, c_void_p, c_int, c_void_p,
                                 c_void_p, c_void_p]),
    "csa_chunk_attn": (c_int, [ctypes.POINTER(AttnParams), ctypes.POINTER(KVCache)] +
                       [c_void_p] * 8 + [c_int] * 3 + [c_void_p] * 3 + [c_size_t, c_void_p]),
    "csa_chunk_attn_workspace_size": (c_size_t, [ctypes.POINTER(AttnParams),
                                                 ctypes.POINTER(KVCache), c_int, c_int, c_int]),
    "csa_chunk_attn_workspace_bound": (c_size_t, [ctypes.POINTER(AttnParams),
                                                  ctypes.POINTER(KVCache), c_int, c_int, c_int]),
    "csa_selftest_chunk_give_up": (c_int, [c_int]),
    "csa_chunk_attn_launch_count": (c_int, [ctypes.POINTER(AttnParams), ctypes.POINTER(KVCache),
                                            c_int, c_int, c_int]),
    "csa_cp_pack_rows": (c_int, [c_void_p, c_int, c_int, c_int, c_int, c_int, c_void_p, c_void_p,
                                 c_int, c_int, c_void_p, c_void_p]),
}


def lib():
    """The loaded CUDA library; raises if it is missing (no CPU fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise CsaError("libcsa.so is not built (%s); run "
                           "`python -m long_context_sparse_05_b200.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if x.device.type != "cuda":
            raise CsaError("tensor arguments must be CUDA tensors (got %s)" % x.device)
        if not x.is_contiguous():
            raise CsaError("tensor arguments must be contiguous")
        return x.data_ptr()
    return int(x)


def _stream(s):
    if s is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, torch.cuda.Stream):
        return s.cuda_stream
    return int(s)


def _check(status):
    if status != 0:
        raise CsaError(lib().csa_status_string(status).decode())


def csa_device_error(stream=None):
    """Synchronise and read/clear the device error word (0 = no bounded wait gave up)."""
    return int(lib().csa_device_error(_stream(stream)))


def csa_selftest_bounded_wait(limit_us, stream=None):
    _check(lib().csa_selftest_bounded_wait(limit_us, _stream(stream)))


def csa_selftest_chunk_give_up(role):
    """The next csa_chunk_attn of this thread acts as if a wait of the role (1..3) had given up."""
    _check(lib().csa_selftest_chunk_give_up(role))


def csa_status_string(status):
    return lib().csa_status_string(status).decode()


def csa_compress(p, C_a, Z_a, B_a, C_b, Z_b, B_b, b, n, entry_begin, entry_count,
                 out_entries_per_seq, out, out_scales=None, stream=None):
    _check(lib().csa_compress(ctypes.byref(p), _ptr(C_a), _ptr(Z_a), _ptr(B_a), _ptr(C_b),
                              _ptr(Z_b), _ptr(B_b), b, n, entry_begin, entry_count,
                              out_entries_per_seq, _ptr(out), _ptr(out_scales), _stream(stream)))


def csa_quantize(in_dtype, out_dtype, x, rows, d, codes, scales, stream=None):
    _check(lib().csa_quantize(in_dtype, out_dtype, _ptr(x), rows, d, _ptr(codes), _ptr(scales),
                              _stream(stream)))


def csa_index_scores(p, q_I, q_scales, w, k_I, k_scales, q_pos, b, T, E_cap, E, scores,
                     stream=None):
    _check(lib().csa_index_scores(ctypes.byref(p), _ptr(q_I), _ptr(q_scales), _ptr(w), _ptr(k_I),
                                  _ptr(k_scales), _ptr(q_pos), b, T, E_cap, E, _ptr(scores),
                                  _stream(stream)))


def csa_topk(scores, score_dtype, q_pos, m, b, T, E, k, idx, count, ws=None, ws_bytes=0,
             stream=None):
    _check(lib().csa_topk(_ptr(scores), score_dtype, _ptr(q_pos), m, b, T, E, k, _ptr(idx),
                          _ptr(count), _ptr(ws), ws_bytes, _stream(stream)))


def csa_topk_workspace_size(score_dtype, b, T, E, k):
    return int(lib().csa_topk_workspace_size(score_dtype, b, T, E, k))


def csa_pool_topk_workspace_size(p, b, T, P, k):
    return int(lib().csa_pool_topk_workspace_size(ctypes.byref(p), b, T, P, k))


def csa_pool_topk(p, q_I, q_scales, w, k_I, k_scales, q_pos, b, T, E_cap, E, pool, pool_count,
                  P, k, idx, count, ws, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().csa_pool_topk(ctypes.byref(p), _ptr(q_I), _ptr(q_scales), _ptr(w), _ptr(k_I),
                               _ptr(k_scales), _ptr(q_pos), b, T, E_cap, E, _ptr(pool),
                               _ptr(pool_count), P, k, _ptr(idx), _ptr(count), _ptr(ws), ws_bytes,
                               _stream(stream)))


def csa_out_proj_workspace_size(T, H, d, g, d_g):
    return int(lib().csa_out_proj_workspace_size(T, H, d, g, d_g))


def csa_out_proj(o, W, T, H, d, g, d_g, y, ws=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(lib().csa_out_proj(_ptr(o), _ptr(W), T, H, d, g, d_g, _ptr(y), _ptr(ws), ws_bytes,
                              _stream(stream)))


def csa_sparse_attn_workspace_size(p, b, T, E_cap):
    return int(lib().csa_sparse_attn_workspace_size(ctypes.byref(p), b, T, E_cap))


def csa_sparse_attn(p, q, kv_comp, E_cap, idx, count, kv_win, n, q_pos, sink, b, T, out, lse=None,
                    ws=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    _check(lib().csa_sparse_attn(ctypes.byref(p), _ptr(q), _ptr(kv_comp), E_cap, _ptr(idx),
                                 _ptr(count), _ptr(kv_win), n, _ptr(q_pos), _ptr(sink), b, T,
                                 _ptr(out), _ptr(lse), _ptr(ws), ws_bytes, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20


def csa_sparse_attn_noalloc(p, q, kv_comp, E_cap, idx, count, kv_win, n, q_pos, sink, b, T, out,
                            lse=None, stream=None):
    """csa_sparse_attn without a workspace: the library's fixed scratch array is used."""
    _check(lib().csa_sparse_attn_noalloc(ctypes.byref(p), _ptr(q), _ptr(kv_comp), E_cap, _ptr(idx),
                                         _ptr(count), _ptr(kv_win), n, _ptr(q_pos), _ptr(sink), b,
                                         T, _ptr(out), _ptr(lse), _stream(stream)))


def _fill(struct_cls, names, tensors):
    s = struct_cls()
    for n in names:
        setattr(s, n, _ptr(tensors.get(n)))
    return s


def csa_decode_workspace_size(p):
    return int(lib().csa_decode_workspace_size(ctypes.byref(p)))


def csa_decode(p, tensors, ws, ws_bytes=None, stream=None):
    """tensors: dict with the csa_decode_tensors field names (missing -> NULL)."""
    x = _fill(DecodeTensors, _DECODE_TENSORS, tensors)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().csa_decode(ctypes.byref(p), ctypes.byref(x), _ptr(ws), ws_bytes, _stream(stream)))


def csa_prefill_workspace_size(p):
    return int(lib().csa_prefill_workspace_size(ctypes.byref(p)))


def csa_prefill(p, tensors, ws, ws_bytes=None, stream=None):
    x = _fill(PrefillTensors, _PREFILL_TENSORS, tensors)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().csa_prefill(ctypes.byref(p), ctypes.byref(x), _ptr(ws), ws_bytes,
                             _stream(stream)))



def csa_decode_launch_count(p):
    return int(lib().csa_decode_launch_count(ctypes.byref(p)))


def csa_prefill_launch_count(p):
    return int(lib().csa_prefill_launch_count(ctypes.byref(p)))


def csa_decode_paged_workspace_size(p):
    return int(lib().csa_decode_paged_workspace_size(ctypes.byref(p)))


def csa_decode_paged_launch_count(p):
    return int(lib().csa_decode_paged_launch_count(ctypes.byref(p)))


def csa_decode_paged(p, tensors, ws, ws_bytes=None, stream=None):
    """tensors: dict with the csa_paged_tensors field names (missing -> NULL)."""
    x = _fill(PagedTensors, _PAGED_TENSORS, tensors)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().csa_decode_paged(ctypes.byref(p), ctypes.byref(x), _ptr(ws), ws_bytes,
                                  _stream(stream)))


# ---------------------------------------------------------------- context-parallel decode

def csa_cp_candidates(scores, E_local, idx, count, b, k, entry_offset, cand_scores, cand_idx,
                      stream=None):
    _check(lib().csa_cp_candidates(_ptr(scores), E_local, _ptr(idx), _ptr(count), b, k,
                                   entry_offset, _ptr(cand_scores), _ptr(cand_idx),
                                   _stream(stream)))


def csa_cp_merge_workspace_size(G, b, k):
    return int(lib().csa_cp_merge_workspace_size(G, b, k))


def csa_cp_merge(cand_scores, cand_idx, G, b, k, idx, count, rows_idx, ws, ws_bytes, stream=None):
    _check(lib().csa_cp_merge(_ptr(cand_scores), _ptr(cand_idx), G, b, k, _ptr(idx), _ptr(count),
                              _ptr(rows_idx), _ptr(ws), ws_bytes, _stream(stream)))


def csa_cp_pack_rows(kv_local, E_cap_local, E_local, entry_offset, c, kv_dtype, idx, count, b, k,
                     rows, stream=None):
    _check(lib().csa_cp_pack_rows(_ptr(kv_local), E_cap_local, E_local, entry_offset, c, kv_dtype,
                                  _ptr(idx), _ptr(count), b, k, _ptr(rows), _stream(stream)))


# ---------------------------------------------------------------- chunks over a paged cache

_ELEM = {CSA_F32: torch.float32, CSA_BF16: torch.bfloat16, CSA_FP8_E4M3: torch.uint8}


def _plain(dtype):
    """torch type of a csa_dtype of plain elements."""
    if dtype not in (CSA_F32, CSA_BF16):
        raise CsaError("expected CSA_F32 or CSA_BF16 (got %s)" % dtype)
    return _ELEM[dtype]


_BYTES = (torch.uint8, torch.float8_e4m3fn)


def _place(stream):
    """(current device, stream) of a call: torch's current stream there unless one is given."""
    if not torch.cuda.is_initialized() and not torch.cuda.is_available():
        raise CsaError("tensor arguments must be CUDA tensors, and there is no CUDA device")
    dev = torch.cuda.current_device()
    if stream is None:
        # (taken here: a build of torch without CUDA lacks it, and imports this file all the same)
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != dev:
        raise CsaError("the stream is on %s, not on the current device" % stream.device)
    return dev, _stream(stream)


def _bad(x, dtype, what, numel, dev):
    if not x.is_cuda:
        return "tensor arguments must be CUDA tensors (%s is on %s)" % (what, x.device)
    if x.dtype is not dtype and not (dtype is torch.uint8 and x.dtype in _BYTES):
        return "%s must be %s (got %s)" % (what, dtype, x.dtype)
    if x.get_device() != dev:
        return "%s is on %s, not on the current device" % (what, x.device)
    if not x.is_contiguous():
        return "%s must be contiguous" % what
    if x.numel() < numel:
        return "%s holds %d elements, %d are needed" % (what, x.numel(), numel)
    return None


def _arg(x, dtype, what, numel, dev):
    """Address of a contiguous CUDA tensor of the given type and at least numel elements on
    device dev; None stays None."""
    if x is None:
        return None
    # (a CPU tensor's device number is -1)
    if x.dtype is dtype and x.get_device() == dev and x.is_contiguous() and x.numel() >= numel:
        return x.data_ptr()
    why = _bad(x, dtype, what, numel, dev)
    if why:
        raise CsaError(why)
    return x.data_ptr()


def _strided(x, dtype, n, rows, what, dev):
    """(address, elements between rows) of a CUDA tensor of at least `rows` rows of n elements
    whose first dimension may be strided."""
    if x is None:
        return None, 0
    if x.is_contiguous():
        if x.dim() < 2 or x.shape[0] < rows or x.numel() != x.shape[0] * n:
            raise CsaError("%s must hold %d rows of %d elements (got %s)" % (what, rows, n, tuple(x.shape)))
        return _arg(x, dtype, what, 0, dev), n
    if x.dim() < 2 or x.shape[0] < rows or x.numel() != x.shape[0] * n:
        raise CsaError("%s must hold %d rows of %d elements (got %s)" % (what, rows, n, tuple(x.shape)))
    if not x[0].is_contiguous():
        raise CsaError("%s: the elements of a row must be contiguous" % what)
    why = _bad(x[0], dtype, what, 0, dev)
    if why:
        raise CsaError(why)
    # a single row has no distance to the next: torch may report any
    return x.data_ptr(), x.stride(0) if x.shape[0] > 1 else n


def kv_cache(dtype, c, d_hi, rows, hi, scales, block_table):
    """csa_kv_cache over torch tensors (rows; or E4M3 codes, bf16 dims and scale exponents),
    which the returned object keeps alive.  The number of pages is the rows' number over
    PAGE_ENTRIES."""
    if dtype not in _ELEM:
        raise CsaError("a cache is F32, BF16 or FP8_E4M3")
    width = c - d_hi if dtype == CSA_FP8_E4M3 else c
    if width < 1 or rows.numel() % (width * PAGE_ENTRIES) or rows.numel() == 0:
        raise CsaError("rows must be whole pages of %d rows of %d elements" % (PAGE_ENTRIES, width))
    pages = rows.numel() // (width * PAGE_ENTRIES)
    n = pages * PAGE_ENTRIES
    if block_table.dim() != 2:
        raise CsaError("block_table must be [b][max_pages]")
    if dtype != CSA_FP8_E4M3 and (hi is not None or scales is not None):
        raise CsaError("hi and scales belong to an FP8 cache")
    stride = ((c - d_hi) // SCALE_GROUP + 7) // 8 * 8
    dev = rows.get_device()
    if dev < 0:
        raise CsaError("tensor arguments must be CUDA tensors (rows is on %s)" % rows.device)
    kv = KVCache(dtype=dtype, c=c, d_hi=d_hi, num_pages=pages, max_pages=block_table.shape[1],
                 rows=_arg(rows, _ELEM[dtype], "rows", 0, dev),
                 hi=_arg(hi, torch.bfloat16, "hi", n * d_hi, dev),
                 scales=_arg(scales, torch.uint8, "scales", n * stride, dev),
                 block_table=_arg(block_table, torch.int32, "block_table", 0, dev))
    kv._tensors = (rows, hi, scales, block_table)
    kv._place = (dev, block_table.shape[0])
    return kv


def alloc_kv_cache(dtype, c, d_hi, num_pages, block_table, device="cuda"):
    """A paged cache of num_pages pages of zeros for the given block table."""
    n = num_pages * PAGE_ENTRIES
    if dtype != CSA_FP8_E4M3:
        return kv_cache(dtype, c, 0, torch.zeros((n, c), dtype=_ELEM[dtype], device=device), None,
                        None, block_table)
    stride = ((c - d_hi) // SCALE_GROUP + 7) // 8 * 8
    return kv_cache(dtype, c, d_hi, torch.zeros((n, c - d_hi), dtype=torch.uint8, device=device),
                    torch.zeros((n, d_hi), dtype=torch.bfloat16, device=device) if d_hi else None,
                    torch.zeros((n, stride), dtype=torch.uint8, device=device), block_table)


def _kv(kv, b, dev):
    """The cache, on device dev, whose block table must have a row for each of b sequences."""
    if kv._place[0] != dev:
        raise CsaError("the cache is on device %d, not on the current one" % kv._place[0])
    if kv._place[1] < b:
        raise CsaError("block_table has %d rows for %d sequences" % (kv._place[1], b))
    return ctypes.byref(kv)


def csa_cache_write(kv, x_dtype, x, cu_rows, first, b, rows, stream=None):
    """x: [rows][c], rows possibly strided (a slice of a wider tensor)."""
    dev, st = _place(stream)
    p, stride = _strided(x, _plain(x_dtype), kv.c, rows, "x", dev)
    _check(lib().csa_cache_write(_kv(kv, b, dev), x_dtype, p, stride,
                                 _arg(cu_rows, torch.int32, "cu_rows", b + 1, dev),
                                 _arg(first, torch.int32, "first", b, dev), b, rows, st))


def csa_cache_read(kv, idx, count, b, k, out_dtype, out, stream=None):
    dev, st = _place(stream)
    _check(lib().csa_cache_read(_kv(kv, b, dev), _arg(idx, torch.int32, "idx", b * k, dev),
                                _arg(count, torch.int32, "count", b, dev), b, k, out_dtype,
                                _arg(out, _plain(out_dtype), "out", b * k * kv.c, dev), st))


def csa_window_append(dtype, c, n_w, win, x, cu_rows, first, b, rows, stream=None):
    dev, st = _place(stream)
    p, stride = _strided(x, _plain(dtype), c, rows, "x", dev)
    _check(lib().csa_window_append(dtype, c, n_w, _arg(win, _plain(dtype), "win", b * n_w * c, dev), p,
                                   stride, _arg(cu_rows, torch.int32, "cu_rows", b + 1, dev),
                                   _arg(first, torch.int32, "first", b, dev), b, rows, st))


def csa_qk_norm_rope(p, q, q_gain, kv, kv_gain, pos, N, q_out, kv_out, stream=None):
    """q: [N][H][d] and kv: [N][d], tokens possibly strided; either may be None."""
    dev, st = _place(stream)
    dt, d = _plain(p.dtype), p.d
    qp, qs = _strided(q, dt, p.H * d, N, "q", dev)
    kp, ks = _strided(kv, dt, d, N, "kv", dev)
    _check(lib().csa_qk_norm_rope(ctypes.byref(p), qp, qs, _arg(q_gain, torch.float32, "q_gain", d, dev),
                                  kp, ks, _arg(kv_gain, torch.float32, "kv_gain", d, dev),
                                  _arg(pos, torch.int32, "pos", N, dev), N,
                                  _arg(q_out, dt, "q_out", N * p.H * d, dev),
                                  _arg(kv_out, dt, "kv_out", N * d, dev), st))


def csa_chunk_attn_workspace_size(p, kv, b, N, L_max):
    return int(lib().csa_chunk_attn_workspace_size(ctypes.byref(p), ctypes.byref(kv), b, N, L_max))


def csa_chunk_attn_workspace_bound(p, kv, b, N, L_max):
    """Bytes for every call with up to b sequences, N rows and L_max positions."""
    return int(lib().csa_chunk_attn_workspace_bound(ctypes.byref(p), ctypes.byref(kv), b, N, L_max))


def csa_chunk_attn_launch_count(p, kv, b, N, L_max):
    return int(lib().csa_chunk_attn_launch_count(ctypes.byref(p), ctypes.byref(kv), b, N, L_max))


def csa_chunk_attn(p, kv, q, cu_q, pos0, idx, count, win, new_win, sink, b, N, L_max, out, lse=None,
                   ws=None, ws_bytes=None, stream=None):
    dev, st = _place(stream)
    dt, d = _plain(p.dtype), p.d
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    n = N * p.H * d
    i32, f32 = torch.int32, torch.float32
    _check(lib().csa_chunk_attn(ctypes.byref(p), _kv(kv, b, dev), _arg(q, dt, "q", n, dev),
                                _arg(cu_q, i32, "cu_q", b + 1, dev), _arg(pos0, i32, "pos0", b, dev),
                                _arg(idx, i32, "idx", N * p.k, dev), _arg(count, i32, "count", N, dev),
                                _arg(win, dt, "win", b * p.n_w * d, dev),
                                _arg(new_win, dt, "new_win", N * d, dev),
                                _arg(sink, f32, "sink", p.H, dev), b, N, L_max,
                                _arg(out, dt, "out", n, dev), _arg(lse, f32, "lse", N * p.H, dev),
                                _arg(ws, ws.dtype if ws is not None else None, "ws", 0, dev), ws_bytes, st))
