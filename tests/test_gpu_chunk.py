"""The calls that serve a chunk of new tokens over a paged cache, against the float64 oracle.

Tolerances, derived before the first run:
 * Cache writes and reads are exact: a code is one rounding of a value scaled by a power of
   two, and what it stands for is a bf16 value.
 * Norm and rotation: a bf16 result is off by at most half a step (2^-8 of its value); the
   float32 arithmetic before it by (d/32 + 16) 2^-24 (a lane's d/32 terms of the sum of
   squares, five shuffles, root, division, two products) of the value, and by 2^-21 of the
   pair's |x0| + |x1| for a rotated one (the reduced angle, up to pi, is rounded to float32:
   2^-23; its sine and cosine to 2^-23 again; two products and a sum).
 * Attention: with l the logits and A = sum_r w_r |row_r| the weighted magnitudes (both from
   the oracle), rounding the logits by dl moves the output by at most 2 dl A and the lse by dl.
   dl <= scale |q|.|row| 2^-14 covers 512 float32 accumulations with an error of a whole
   last place each (2^-23); small head dims lie far below.  The accumulation over R rows adds
   R 2^-23 A, the exponentials 2^-21 A.  In bf16 each weight is rounded (2^-8) and so is the
   result (2^-8): 2^-8 (A + |o|).  The inverse rotation mixes a pair: its A is the pair's sum,
   and the angle adds 2^-21 of it.
"""

import math

import numpy as np
import pytest
import torch

from long_context_sparse_05_b200 import _lib as L
from oracle import chunk, csa

from helpers import f64

pytestmark = pytest.mark.gpu

PE = L.PAGE_ENTRIES
THETA, EPS = 10000.0, 1e-6
TDT = {L.CSA_F32: torch.float32, L.CSA_BF16: torch.bfloat16}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(lens):
    return [0] + np.cumsum(lens).tolist()


def randn(seed, shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def table(entries, seed=0, extra=1, max_pages=None):
    """(pages, block table) of sequences with the given entries, pages shuffled."""
    need = [-(-e // PE) for e in entries]
    total = sum(need) + extra
    perm = np.random.default_rng(seed).permutation(total)
    bt = np.full((len(entries), max_pages or max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = perm[at:at + n]
        at += n
    return total, bt


def place(bt, s, e):
    return int(bt[s, e // PE]) * PE + e % PE


# ----------------------------------------------------------------------------- norm, rotation

@pytest.mark.parametrize("dtype,N,H,d,d_rope,gain,strided,norm", [
    (L.CSA_BF16, 1, 64, 512, 64, True, False, 1),
    (L.CSA_BF16, 5, 64, 512, 64, False, True, 1),
    (L.CSA_BF16, 331, 64, 512, 64, True, True, 1),     # several rows per warp, tokens straddle warps
    (L.CSA_BF16, 17, 64, 128, 64, False, False, 0),    # index queries: rotation alone
    (L.CSA_F32, 33, 4, 64, 16, True, False, 1),
    (L.CSA_F32, 9, 3, 40, 6, True, True, 1),           # rotary dims starting inside a chunk of 8
    (L.CSA_F32, 2, 1, 8, 8, False, False, 1),
    (L.CSA_F32, 3, 2, 2048, 128, True, False, 1),
    (L.CSA_BF16, 4, 2, 1000, 0, True, False, 1),
])
def test_norm_rope(dtype, N, H, d, d_rope, gain, strided, norm):
    dt = TDT[dtype]
    if strided:
        buf = randn(1, (N, (H + 1) * d + 16), dt)
        q, kv = buf[:, : H * d].view(N, H, d), buf[:, H * d:(H + 1) * d]
    else:
        q, kv = randn(1, (N, H, d), dt), randn(2, (N, d), dt)
    qg = (1 + 0.2 * randn(3, (d,))) if gain else None
    kg = (1 + 0.2 * randn(4, (d,))) if gain else None
    pos = [(i * 7919 + 3) % (1 << 20) for i in range(N)]
    qo, ko = torch.empty((N, H, d), dtype=dt, device="cuda"), torch.empty((N, d), dtype=dt, device="cuda")
    p = L.NormRopeParams(H=H, d=d, d_rope=d_rope, rope_theta=THETA, eps=EPS, apply_norm=norm, dtype=dtype)
    L.csa_qk_norm_rope(p, q, qg, kv, kg, i32(pos), N, qo, ko)
    rows = sorted(set([0, N - 1, N // 2] + list(range(min(N, 6)))))
    for out, x, g in ((qo, q, qg), (ko[:, None], kv[:, None], kg)):
        for n in rows:
            xr = f64(x[n])
            y0 = chunk.norm_rope(xr, None if g is None else f64(g), np.zeros(len(xr)), 0, THETA, EPS, bool(norm))
            ref = csa.rope_partial(y0, np.full(len(xr), float(pos[n])), d_rope, THETA)
            tol = (d / 32 + 16) * 2.0 ** -24 * np.abs(ref)
            if d_rope:
                pair = np.abs(y0[:, d - d_rope:]).reshape(len(xr), -1, 2).sum(-1)
                tol[:, d - d_rope:] += np.repeat(pair, 2, axis=1) * ((d / 32 + 16) * 2.0 ** -24 + 2.0 ** -21)
            if dtype == L.CSA_BF16:
                tol += 2.0 ** -8 * np.abs(ref)
            err = np.abs(f64(out[n]) - ref)
            assert np.all(err <= tol + 1e-37), (n, float(np.max(err / (tol + 1e-37))))


def test_norm_rope_one_side_and_in_place():
    N, H, d = 6, 64, 512
    q, kv = randn(5, (N, H, d), torch.bfloat16), randn(6, (N, d), torch.bfloat16)
    pos = i32([5] * N)
    p = L.NormRopeParams(H=H, d=d, d_rope=64, rope_theta=THETA, eps=EPS, apply_norm=1, dtype=L.CSA_BF16)
    qo, ko = torch.empty_like(q), torch.empty_like(kv)
    L.csa_qk_norm_rope(p, q, None, kv, None, pos, N, qo, ko)
    q1, k1 = torch.empty_like(q), torch.empty_like(kv)
    L.csa_qk_norm_rope(p, q, None, None, None, pos, N, q1, None)
    L.csa_qk_norm_rope(p, None, None, kv, None, pos, N, None, k1)
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    L.csa_qk_norm_rope(p, q, None, kv, None, pos, N, q, kv)
    assert torch.equal(q, qo) and torch.equal(kv, ko)


# ----------------------------------------------------------------------------- the cache

def cache_of(fmt, c, d_hi, total, bt, fill=None):
    kv = L.alloc_kv_cache(fmt, c, d_hi, total, torch.from_numpy(bt).cuda())
    if fill is not None:
        for t in kv._tensors[:3]:
            if t is not None:
                t.view(torch.uint8).fill_(fill)
    return kv


@pytest.mark.parametrize("fmt,x_dtype,c,d_hi,lens,first", [
    (L.CSA_FP8_E4M3, L.CSA_BF16, 512, 64, [1] * 5, [0, 255, 256, 700, 511]),
    (L.CSA_FP8_E4M3, L.CSA_BF16, 512, 64, [300, 0, 1, 517, 0], [250, 3, 255, 1, 0]),
    (L.CSA_FP8_E4M3, L.CSA_F32, 512, 64, [33, 2], [0, 254]),
    (L.CSA_FP8_E4M3, L.CSA_BF16, 64, 0, [7], [3]),
    (L.CSA_FP8_E4M3, L.CSA_F32, 1104, 16, [5, 3], [254, 0]),      # more than one pass, odd widths
    (L.CSA_FP8_E4M3, L.CSA_BF16, 512, 64, [39000, 77], [0, 9]),   # several rows per warp
    (L.CSA_BF16, L.CSA_BF16, 512, 0, [3, 270], [255, 0]),
    (L.CSA_BF16, L.CSA_F32, 40, 0, [3, 1], [0, 2]),
    (L.CSA_F32, L.CSA_F32, 8, 0, [2, 300], [1, 0]),
    (L.CSA_F32, L.CSA_BF16, 64, 0, [4], [254]),
])
def test_cache_write_and_read(fmt, x_dtype, c, d_hi, lens, first):
    b, n = len(lens), sum(lens)
    total, bt = table([f + l for f, l in zip(first, lens)], seed=3, extra=2)
    kv = cache_of(fmt, c, d_hi, total, bt, fill=0xA5)
    before = [None if t is None else t.clone() for t in kv._tensors[:3]]
    x = randn(7, (n + 3, c), TDT[x_dtype])
    x[:, ::5] *= 30.0                                  # groups of very different sizes
    x[0, : min(c, 64)] = 0.0
    if fmt == L.CSA_FP8_E4M3 and n > 2:
        x[1, 0], x[1, 1] = 448.0, -448.0 * 2.0 ** -30
        x[2, 0] = 1.0e-42 if x_dtype == L.CSA_F32 else 2.0 ** -130
    cu = starts(lens)
    # rows counted beyond the last sequence's are not written
    L.csa_cache_write(kv, x_dtype, x, i32(cu), i32(first), b, n + 3)
    torch.cuda.synchronize()
    xs = f64(x)
    arrs = [None if t is None else t.cpu() for t in kv._tensors[:3]]
    touched = set()
    rng = np.random.default_rng(0)
    for s in range(b):
        js = range(lens[s]) if lens[s] <= 600 else sorted(set([0, 1, lens[s] - 1]) | set(rng.integers(0, lens[s], 60).tolist()))
        touched |= {place(bt, s, first[s] + j) for j in range(lens[s])}
        for j in js:
            at, row = place(bt, s, first[s] + j), xs[cu[s] + j]
            if fmt == L.CSA_FP8_E4M3:
                codes, hi, exps = chunk.quant_row(row, d_hi)
                assert np.array_equal(arrs[0][at].numpy(), codes), (s, j)
                assert np.array_equal(arrs[2][at].numpy()[: len(exps)], exps), (s, j)
                if d_hi:
                    assert np.array_equal(f64(arrs[1][at]), hi)
            else:
                assert torch.equal(arrs[0][at].cuda(), x[cu[s] + j].to(TDT[fmt]))
    # every other row as it was, and the spare scale bytes too
    rest = torch.ones(total * PE, dtype=torch.bool)
    rest[torch.tensor(sorted(touched), dtype=torch.long)] = False
    for t, t0 in zip(arrs, before):
        if t is not None:
            assert torch.equal(t.view(torch.uint8)[rest], t0.cpu().view(torch.uint8)[rest])
    if fmt == L.CSA_FP8_E4M3:
        ng = (c - d_hi) // 64
        assert torch.all(arrs[2][:, ng:] == 0xA5)
    # read back: selected entries in any order, a repeated one, ones outside, and whole ranges
    kmax = max(max(first[s] + lens[s] for s in range(b)), 4) + 2
    k = min(kmax, 300)
    idx = rng.integers(-2, kmax, (b, k)).astype(np.int32)
    idx[0, :4] = [first[0], first[0], 2 ** 31 - 1, -2 ** 31]
    count = np.array([k - (s % 3) for s in range(b)], dtype=np.int32)
    for out_dtype in (L.CSA_F32, L.CSA_BF16):
        for sel in (idx, None):
            out = torch.full((b, k, c), float("nan"), dtype=TDT[out_dtype], device="cuda")
            L.csa_cache_read(kv, None if sel is None else i32(sel.tolist()), i32(count.tolist()), b, k,
                             out_dtype, out)
            for s in range(b):
                for j in list(range(6)) + [k // 2, k - 2, k - 1]:
                    e = int(sel[s, j]) if sel is not None else j
                    held = 0 <= e < bt.shape[1] * PE and j < count[s] and bt[s, e // PE] >= 0
                    if not held:
                        assert torch.all(out[s, j] == 0), (s, j, e)
                        continue
                    at = place(bt, s, e)
                    if at not in touched:
                        continue               # filler bytes: not numbers to compare
                    if fmt == L.CSA_FP8_E4M3:
                        hi = f64(arrs[1][at]) if d_hi else np.zeros(0)
                        ref = chunk.dequant_row(arrs[0][at].numpy(), hi, arrs[2][at].numpy()[: (c - d_hi) // 64])
                        assert np.array_equal(f64(out[s, j]), ref), (s, j, e)
                    else:
                        assert torch.equal(out[s, j], arrs[0][at].cuda().to(TDT[out_dtype]))


def test_cache_write_strided_rows_and_specials():
    c, d_hi = 512, 64
    total, bt = table([20], seed=1)
    wide = randn(8, (20, 2 * c + 8), torch.bfloat16)
    wide[0, c], wide[0, c + 1] = float("nan"), 3.0
    wide[1, c + 64], wide[1, c + 65] = float("inf"), -float("inf")
    wide[2, c:c + 64] = float("nan")
    x = wide[:, c:2 * c]
    kv = cache_of(L.CSA_FP8_E4M3, c, d_hi, total, bt)
    L.csa_cache_write(kv, L.CSA_BF16, x, i32([0, 20]), i32([0]), 1, 20)
    out = torch.empty((1, 20, c), dtype=torch.bfloat16, device="cuda")
    L.csa_cache_read(kv, None, None, 1, 20, L.CSA_BF16, out)
    for j in range(20):
        codes, hi, exps = chunk.quant_row(f64(x[j]), d_hi)
        assert np.array_equal(kv._tensors[0][place(bt, 0, j)].cpu().numpy(), codes), j
        np.testing.assert_array_equal(f64(out[0, j]), chunk.dequant_row(codes, hi, exps))


def test_cache_skips_pages_and_entries_outside():
    """A table entry outside the pool, entries past the table and before 0: nothing is written
    there, nothing is read."""
    c = 64
    bt = np.array([[0, 7, 1], [-1, 2, -5]], dtype=np.int32)     # 7 and the negatives: no page
    kv = cache_of(L.CSA_BF16, c, 0, 4, bt)
    x = torch.ones((1600, c), dtype=torch.bfloat16, device="cuda")
    L.csa_cache_write(kv, L.CSA_BF16, x, i32([0, 800, 1600]), i32([0, -20]), 2, 1600)
    rows = kv._tensors[0].view(4, PE, c)
    assert torch.all(rows[0] == 1) and torch.all(rows[1] == 1) and torch.all(rows[2] == 1)
    assert torch.all(rows[3] == 0)
    out = torch.full((2, 900, c), 9.0, dtype=torch.bfloat16, device="cuda")
    L.csa_cache_read(kv, None, None, 2, 900, L.CSA_BF16, out)
    ok = torch.zeros((2, 900), dtype=torch.bool)
    ok[0, :256] = ok[0, 512:768] = ok[1, 256:512] = True
    assert torch.equal((out[:, :, 0] == 1).cpu(), ok) and torch.all(out[~ok.cuda()] == 0)


@pytest.mark.parametrize("dtype,c,n_w", [(L.CSA_BF16, 512, 128), (L.CSA_F32, 64, 16), (L.CSA_BF16, 8, 1)])
def test_window_append(dtype, c, n_w):
    """The rings after a chunk are what appending token by token leaves, whatever its length."""
    lens, first = [1, 3 * n_w + 5, 0, n_w, 7], [5, 1000, 3, 0, n_w - 1]
    b, n = len(lens), sum(lens)
    win = randn(1, (b, n_w, c), TDT[dtype])
    x = randn(2, (n + 2, c + 8), TDT[dtype])[:, :c]
    want = win.clone()
    cu = starts(lens)
    for s in range(b):
        for j in range(lens[s]):
            want[s, (first[s] + j) % n_w] = x[cu[s] + j]
    L.csa_window_append(dtype, c, n_w, win, x, i32(cu), i32(first), b, n + 2)
    assert torch.equal(win, want)


# ----------------------------------------------------------------------------- attention

class Case:
    """A ragged chunk over a paged cache with everything random, and its oracle."""

    def __init__(self, lens, ctx, H, d, m, k, n_w, dtype, fmt, d_hi=0, d_rope_out=0, seed=0,
                 sink=None, pad=2, counts=None, hole=False, qscale=1.0, rscale=1.0, zero_group=False,
                 nan_rest=False, dup=False):
        self.__dict__.update(lens=lens, ctx=ctx, H=H, d=d, m=m, k=k, n_w=n_w, dtype=dtype, fmt=fmt,
                             d_hi=d_hi)
        b, n = len(lens), sum(lens)
        dt = TDT[dtype]
        self.b, self.N, self.cu = b, n + pad, starts(lens)
        ents = [(p + l) // m for p, l in zip(ctx, lens)]
        total, self.bt = table(ents, seed=seed)
        if hole and self.bt.shape[1] > 1:
            self.bt[0, 0] = total + 3                # a page outside the pool
        self.kv = cache_of(fmt, d, d_hi, total, self.bt)
        rows = randn(seed + 1, (total * PE, d)) * rscale
        if zero_group:
            rows[::3, :64] = 0.0                     # groups of zeros: the lowest scale
        if fmt == L.CSA_FP8_E4M3:
            flat = L.alloc_kv_cache(fmt, d, d_hi, total, i32([list(range(total))]))
            flat.rows, flat.hi, flat.scales = self.kv.rows, self.kv.hi, self.kv.scales
            L.csa_cache_write(flat, L.CSA_F32, rows, i32([0, total * PE]), i32([0]), 1, total * PE)
        else:
            self.kv._tensors[0].copy_(rows)
        if nan_rest:
            # every row that no token may see: NaN
            seen = torch.zeros(total * PE, dtype=torch.bool)
            for s, e in enumerate(ents):
                for x in range(e):
                    if 0 <= self.bt[s, x // PE] < total:
                        seen[place(self.bt, s, x)] = True
            hid = (~seen).cuda()
            if fmt == L.CSA_FP8_E4M3:
                self.kv._tensors[0][hid] = 0x7F
                self.kv._tensors[1][hid] = float("nan")
                self.kv._tensors[2][hid] = 0xFF
            else:
                self.kv._tensors[0][hid] = float("nan")
        self.q = (randn(seed + 2, (self.N, H, d)) * qscale).to(dt)
        self.win = randn(seed + 3, (b, max(n_w, 1), d), dt)
        self.new_win = randn(seed + 4, (self.N, d), dt)
        if rscale != 1.0:
            self.win *= rscale
            self.new_win *= rscale
        if nan_rest:
            for s in range(b):                       # ring slots before the sequence's first token
                for u in range(ctx[s] - max(n_w, 1), min(0, ctx[s])):
                    self.win[s, u % max(n_w, 1)] = float("nan")
            self.new_win[self.cu[-1]:] = float("nan")
            self.q[self.cu[-1]:] = float("nan")
        self.sink = randn(seed + 5, (H,)) if sink is None else torch.full((H,), sink, device="cuda")
        self.idx = self.count = None
        if k:
            rng = np.random.default_rng(seed)
            idx, count = np.full((self.N, k), -1, dtype=np.int32), np.zeros(self.N, dtype=np.int32)
            for s in range(b):
                for i in range(lens[s]):
                    E = (ctx[s] + i + 1) // m
                    r = self.cu[s] + i
                    c = min(E, k) if counts is None else min(counts, k)
                    pick = np.sort(rng.choice(E, min(E, c), replace=False)) if E else np.zeros(0, int)
                    if dup and len(pick) > 2:
                        pick[1] = pick[0]            # an entry named twice counts twice
                        pick[-1] = 2 ** 31 - 1       # and one far outside the table
                    idx[r, :len(pick)] = pick
                    count[r] = c
            self.idx, self.count = i32(idx.tolist()), i32(count.tolist())
        self.L_max = max(p + l for p, l in zip(ctx, lens))
        self.p = L.AttnParams(H=H, d=d, n_w=n_w, scale=1.0 / math.sqrt(d), m=m, k=k, dtype=dtype,
                              d_rope_out=d_rope_out, rope_theta=THETA)
        self.out = torch.full((self.N, H, d), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((self.N, H), 7.0, device="cuda")
        nb = L.csa_chunk_attn_workspace_size(self.p, self.kv, b, self.N, self.L_max)
        self.ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        L.csa_chunk_attn(self.p, self.kv, self.q, i32(self.cu), i32(self.ctx), self.idx, self.count,
                         self.win if self.n_w else None, self.new_win if self.n_w else None, self.sink,
                         self.b, self.N, self.L_max, self.out, self.lse, self.ws, stream=stream)
        torch.cuda.synchronize()
        assert L.csa_device_error() == 0
        return self

    def entry(self, s, e):
        pg = int(self.bt[s, e // PE])
        if not 0 <= pg < self.kv.num_pages:
            return None
        at = pg * PE + e % PE
        if self.fmt != L.CSA_FP8_E4M3:
            return self.rows64[at]
        return self.rows64[at]

    def values(self):
        """The pool's rows as float64."""
        a = self.kv._tensors
        if self.fmt != L.CSA_FP8_E4M3:
            return f64(a[0])
        out = torch.empty((1, self.kv.num_pages * PE, self.d), dtype=torch.float32, device="cuda")
        flat = L.alloc_kv_cache(self.fmt, self.d, self.d_hi, 1, i32([list(range(self.kv.num_pages))]))
        flat.num_pages, flat.rows, flat.hi, flat.scales = (self.kv.num_pages, self.kv.rows,
                                                           self.kv.hi, self.kv.scales)
        L.csa_cache_read(flat, None, None, 1, self.kv.num_pages * PE, L.CSA_F32, out)
        return f64(out[0])

    def check(self, tokens=None):
        self.rows64 = self.values()
        q, win, nw, sink = f64(self.q), f64(self.win), f64(self.new_win), f64(self.sink)
        out, lse = f64(self.out), f64(self.lse)
        d, r_out = self.d, self.p.d_rope_out
        bf = self.dtype == L.CSA_BF16
        for s in range(self.b):
            picks = range(self.lens[s]) if tokens is None else sorted(
                {0, self.lens[s] - 1} | set(np.linspace(0, self.lens[s] - 1, tokens).astype(int))) if self.lens[s] else []
            for i in picks:
                row = self.cu[s] + i
                sel = None
                if self.k:
                    sel = self.idx[row].cpu().numpy()[: int(self.count[row])]
                t, rows = chunk.chunk_rows(s, i, self.entry, sel, self.ctx[s], self.cu[s], self.m,
                                           self.bt.shape[1] * PE, win, nw, self.n_w)
                o, l, A = chunk.attend(q[row], rows, sink, self.p.scale)
                R = np.asarray(rows) if rows else np.zeros((1, d))
                dl = self.p.scale * (np.abs(q[row]) @ np.abs(R).T).max(axis=1) * 2.0 ** -14
                n = len(rows)
                tol = A * (2 * dl[:, None] + n * 2.0 ** -23 + 2.0 ** -21)
                if bf:
                    tol += 2.0 ** -8 * A
                if r_out:
                    o = csa.inverse_rope(o, t, r_out, THETA)
                    pair = tol[:, d - r_out:].reshape(self.H, -1, 2).sum(-1)
                    mag = A[:, d - r_out:].reshape(self.H, -1, 2).sum(-1) * 2.0 ** -21
                    tol[:, d - r_out:] = np.repeat(pair + mag, 2, axis=1)
                if bf:
                    tol += 2.0 ** -8 * np.abs(o)
                err = np.abs(out[row] - o)
                assert np.all(err <= tol + 1e-30), (s, i, t, float(np.max(err / (tol + 1e-30))))
                fin = np.isfinite(l)
                assert np.array_equal(lse[row][~fin], l[~fin])
                ltol = dl + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(fin, l, 0))
                assert np.all(np.abs(lse[row] - np.where(fin, l, 0))[fin] <= ltol[fin]), (s, i)
        # rows behind the last sequence stay as they were
        assert torch.all(self.out[self.cu[-1]:] == 7.0) and torch.all(self.lse[self.cu[-1]:] == 7.0)


SMALL = dict(H=4, d=64, m=4, n_w=16, dtype=L.CSA_F32, fmt=L.CSA_F32)
TC = dict(H=64, d=512, n_w=128, dtype=L.CSA_BF16)


@pytest.mark.parametrize("k", [0, 16])
@pytest.mark.parametrize("over", [
    dict(), dict(H=3, d=40, n_w=5), dict(H=1, d=8, n_w=0), dict(dtype=L.CSA_BF16, fmt=L.CSA_BF16, d_rope_out=16),
    dict(fmt=L.CSA_FP8_E4M3, d=128, d_hi=64, d_rope_out=64),
    dict(dtype=L.CSA_BF16, fmt=L.CSA_FP8_E4M3, d=80, d_hi=16, m=128, n_w=128),
])
def test_chunk_attn_any_shape(k, over):
    cfg = dict(SMALL, **over)
    Case([5, 0, 1, 33], [0, 9, 1027, 300], k=k, seed=11, **cfg).run().check()


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
@pytest.mark.parametrize("lens,ctx,m,k,d_rope_out", [
    ([1], [0], 4, 0, 0),                                  # the very first token: a window of one row
    ([1, 1, 1], [511, 5000, 2], 4, 512, 64),              # single tokens, selections cut by E(t) and k
    ([1, 1], [128 * 700 + 17, 128 * 300 - 1], 128, 0, 64),  # long dense rows, split over CTAs
    ([7, 0, 130, 1], [1000, 4, 0, 40000], 4, 512, 64),    # ragged, an empty sequence, a fresh prompt
    ([40, 3], [128 * 256 - 20, 128 * 40], 128, 0, 0),     # visible entries cross a page inside the chunk
    ([200, 101], [3000, 0], 4, 37, 64),                   # a selection of an odd length
])
def test_chunk_attn_tensor_core(fmt, d_hi, lens, ctx, m, k, d_rope_out):
    Case(lens, ctx, m=m, k=k, fmt=fmt, d_hi=d_hi, d_rope_out=d_rope_out, seed=21, **TC).run().check(tokens=6)


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
@pytest.mark.parametrize("cfg", [
    dict(n_w=0, k=64, counts=0),                    # no row at all: zeros, the sink as lse
    dict(n_w=0, k=64, counts=0, sink=-math.inf),    # nor a sink: lse -inf
    dict(n_w=0, k=0),                               # E(t) = 0 for the first tokens
    dict(n_w=1, k=64),
    dict(n_w=300, k=64),                            # a window of more than two tiles
    dict(n_w=128, k=64, sink=-math.inf),
    dict(n_w=128, k=64, sink=200.0),                # a sink far above every logit
    dict(n_w=128, k=64, sink=-200.0),
    dict(n_w=128, k=700, hole=True),                # selected entries on a page outside the pool
    dict(n_w=0, k=64, hole=True, ctx=[900, 40]),    # every selected entry outside: weights of nothing
    dict(n_w=128, k=300, counts=300, ctx=[400, 0]),  # count beyond the valid entries: -1 padding inside
    dict(n_w=128, k=512, qscale=30.0),              # one row takes nearly all the weight
])
def test_chunk_attn_masks_and_edges(fmt, d_hi, cfg):
    c = dict(TC, lens=[5, 3], ctx=[2500, 1], m=4, seed=31, fmt=fmt, d_hi=d_hi)
    c.update(cfg)
    Case(**c).run().check()


def test_chunk_attn_small_shape_edges():
    for cfg in (dict(n_w=0, k=16, counts=0), dict(n_w=0, k=16, counts=0, sink=-math.inf),
                dict(n_w=16, k=0, sink=-math.inf), dict(n_w=0, k=0), dict(n_w=3, k=16, hole=True),
                dict(n_w=16, k=16, sink=90.0), dict(n_w=0, k=8, hole=True)):
        c = dict(SMALL, lens=[5, 3], ctx=[2500, 1], seed=41)
        c.update(cfg)
        Case(**c).run().check()


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
@pytest.mark.parametrize("cfg", [
    dict(lens=[303], ctx=[2600], k=700, qscale=20.0),             # many tiles in one CTA, maxima that rise
    dict(lens=[200, 130], ctx=[4000, 17], k=0),                   # whole tiles, partial ones, two windows
    dict(lens=[303], ctx=[2600], k=0, qscale=20.0, n_w=5),
    dict(lens=[303], ctx=[2400], k=650, hole=True),               # tiles without a row before the first with one
    dict(lens=[303], ctx=[2400], k=0, hole=True, sink=-math.inf, n_w=0),
    dict(lens=[150, 160], ctx=[3000, 900], k=300, nan_rest=True),
    dict(lens=[150, 160], ctx=[3000, 60], k=0, nan_rest=True, n_w=130),
    dict(lens=[40], ctx=[5000], k=0, nan_rest=True),              # the same with the rows split over CTAs
    dict(lens=[301], ctx=[1500], k=300, rscale=2.0 ** 30, qscale=2.0 ** -30),   # scales beyond f16
    dict(lens=[301], ctx=[1500], k=300, zero_group=True),
    dict(lens=[9], ctx=[1500], k=300, zero_group=True, rscale=2.0 ** -20, qscale=2.0 ** 20),
    dict(lens=[301, 20], ctx=[1500, 90], k=64, dup=True),
    dict(lens=[7], ctx=[1500], k=200, dup=True),
    dict(lens=[160, 140], ctx=[128 * 70, 128 * 3], k=0, m=128),
])
def test_chunk_attn_many_tiles(fmt, d_hi, cfg):
    c = dict(TC, m=4, seed=51, fmt=fmt, d_hi=d_hi, d_rope_out=64)
    c.update(cfg)
    Case(**c).run().check(tokens=5)


@pytest.mark.parametrize("fmt,d_hi,shape", [(L.CSA_BF16, 0, "tc"), (L.CSA_FP8_E4M3, 64, "tc"), (L.CSA_F32, 0, "small")])
def test_chunk_attn_counts_out_of_range(fmt, d_hi, shape):
    """A negative count selects nothing, one above k all k slots."""
    cfg = dict(TC, m=4) if shape == "tc" else dict(SMALL)
    cfg["fmt"] = fmt
    c = Case([4], [900], k=32, d_hi=d_hi, seed=61, **cfg)
    want = c.count.clone()
    c.count[0], c.count[1] = -7, 32 + 1000
    c.run()
    c.count = want
    c.count[0], c.count[1] = 0, 32
    c.check()


@pytest.mark.parametrize("cfg", [
    dict(TC, fmt=L.CSA_BF16, lens=[5, 3], ctx=[2500, 900]),          # split over several CTAs
    dict(TC, fmt=L.CSA_BF16, lens=[300], ctx=[2500]),                # not split
    dict(TC, fmt=L.CSA_FP8_E4M3, d_hi=64, lens=[300], ctx=[2500]),
    dict(SMALL, lens=[5, 3], ctx=[2500, 900]),
])
def test_chunk_attn_a_head_of_infinities(cfg):
    """Head 0's logits are all -inf: its sink takes all, and the other heads are untouched."""
    c = Case(**dict(cfg, m=4, k=0, seed=81))
    if c.fmt == L.CSA_FP8_E4M3:
        c.kv._tensors[0].view(-1, c.d - c.d_hi)[:, 0] = 0x38         # 1.0
    else:
        c.kv._tensors[0].view(-1, c.d)[:, 0] = 1.0
    c.win[..., 0] = 1.0
    c.new_win[..., 0] = 1.0
    finite = c.q.clone()
    c.q[:, 0, 0] = -math.inf
    c.run()
    out, lse, n = c.out.clone(), c.lse.clone(), c.cu[-1]
    assert torch.all(out[:n, 0] == 0)
    s = c.sink[0].item()
    assert torch.all((lse[:n, 0] - s).abs() <= 2.0 ** -20 + 2.0 ** -22 * abs(s))
    c.q = finite
    c.run()
    c.out[:, 1:], c.lse[:, 1:] = out[:, 1:], lse[:, 1:]
    c.check(tokens=5)


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
@pytest.mark.parametrize("cfg", [
    dict(lens=[310, 140], ctx=[700, 0], n_w=300, k=64),              # whole tiles of new rows, then a part
    dict(lens=[450], ctx=[77], n_w=256, k=0),                        # part of the first from the rings
    dict(lens=[128], ctx=[0], n_w=128, k=16, pad=0),                 # one token with a whole tile
    dict(lens=[127], ctx=[1], n_w=128, k=16, pad=0),                 # fewer rows than a tile
    dict(lens=[60, 200, 60], ctx=[0, 5, 900], n_w=129, k=64),
    dict(lens=[400], ctx=[0], n_w=128, k=64, counts=0),              # the window alone
])
def test_chunk_attn_windows_of_new_rows(fmt, d_hi, cfg):
    c = dict(TC, m=4, seed=91, fmt=fmt, d_hi=d_hi, nan_rest=True, d_rope_out=64)
    c.update(cfg)
    Case(**c).run().check(tokens=12)


def _one_by_one(c, n_least):
    """Each sequence of a case by itself, in a call of at least n_least rows (so that neither is
    split): the same output, bit for bit."""
    out, lse = c.out.clone(), c.lse.clone()
    bt = i32(c.bt.tolist())
    for s in range(c.b):
        lo, hi = c.cu[s], c.cu[s + 1]
        n = max(hi - lo, n_least)
        kv = L.kv_cache(c.fmt, c.d, c.d_hi, *c.kv._tensors[:3], bt[s:s + 1].contiguous())

        def part(x):
            y = torch.zeros((n,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
            y[:hi - lo] = x[lo:hi]
            return y

        o = torch.empty((n,) + tuple(out.shape[1:]), dtype=out.dtype, device="cuda")
        e = torch.empty((n, c.H), device="cuda")
        assert L.csa_chunk_attn_workspace_size(c.p, kv, 1, n, c.L_max) == 0
        L.csa_chunk_attn(c.p, kv, part(c.q), i32([0, hi - lo]), i32([c.ctx[s]]),
                         part(c.idx) if c.k else None, part(c.count) if c.k else None,
                         c.win[s:s + 1].contiguous(), part(c.new_win), c.sink, 1, n, c.L_max, o, e, None)
        torch.cuda.synchronize()
        assert torch.equal(out[lo:hi], o[:hi - lo]) and torch.equal(lse[lo:hi], e[:hi - lo]), s


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
@pytest.mark.parametrize("lens,ctx,k", [
    ([1, 37, 300, 29, 61], [70001, 0, 131, 3000, 25500], 0),         # one long token, many short
    ([0, 200, 0, 3, 160, 0], [9, 5000, 0, 40, 0, 77], 0),            # sequences without tokens
    ([5] * 63 + [9], list(range(0, 64 * 300, 300)), 0),              # as many as are ordered
    ([7] * 65, list(range(0, 65 * 300, 300)), 0),                    # one more
    ([300, 200], [4000, 0], 64),
    ([149, 148, 1], [0, 0, 0], 0),                                   # equal ones
])
def test_chunk_attn_shared_out(fmt, d_hi, lens, ctx, k):
    c = Case(lens, ctx, m=4, k=k, seed=101, fmt=fmt, d_hi=d_hi, d_rope_out=64, **TC).run()
    assert c.N >= 296 and torch.all(c.out[c.cu[-1]:] == 7.0)
    _one_by_one(c, 296)


def test_chunk_attn_shared_out_long_lists():
    """147 tokens of 3,200 tiles (nearly all on pages outside the pool) and 1,300 of one: a CTA
    would take more items than its list holds."""
    m, e = 4096, 3200 * 128
    t = e * m
    c = Case([147, 1300], [0, 0], m=4, k=0, seed=111, fmt=L.CSA_BF16, **TC)
    bt = torch.full((2, e // PE), -1, dtype=torch.int32, device="cuda")
    bt[0, 0], bt[0, -1], bt[1, 0] = 1, 0, 1
    c.bt, c.kv = bt.cpu().numpy(), L.kv_cache(c.fmt, c.d, c.d_hi, *c.kv._tensors[:3], bt)
    c.p.m, c.ctx, c.L_max = m, [t, 0], t + 147
    c.run()
    _one_by_one(c, 296)
    assert torch.all(torch.isfinite(c.out[:c.cu[-1]].float()))


def test_captured_shares_follow_the_lengths():
    """A replay shares its items out by the lengths it then finds."""
    c = Case([200, 130], [2900, 50], m=4, k=0, seed=121, fmt=L.CSA_BF16, **TC)
    cu, pos0 = i32([0, 200, 330]), i32([2900, 50])

    def call():
        L.csa_chunk_attn(c.p, c.kv, c.q, cu, pos0, None, None, c.win, c.new_win, c.sink, 2, c.N,
                         c.L_max, c.out, c.lse, c.ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens, ctx in (([200, 130], [2900, 50]), ([30, 300], [2900, 0]), ([0, 310], [7, 20])):
        cu.copy_(i32(starts(lens)))
        pos0.copy_(i32(ctx))
        c.out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        got, glse = c.out.clone(), c.lse.clone()
        c.out.fill_(3.0)
        call()
        torch.cuda.synchronize()
        assert L.csa_device_error() == 0
        assert torch.equal(got, c.out) and torch.equal(glse, c.lse)
        c.lens, c.ctx, c.cu = lens, ctx, starts(lens)
        assert torch.all(c.out[c.cu[-1]:] == 3.0)
        c.out[c.cu[-1]:], c.lse[c.cu[-1]:] = 7.0, 7.0
        c.check(tokens=4)


@pytest.mark.parametrize("b", [33, 1100])
def test_chunk_attn_many_sequences(b):
    """More sequences than one step of the search, and than shared memory holds."""
    rng = np.random.default_rng(b)
    lens = [int(x) for x in rng.integers(0, 3, b)]
    ctx = [int(x) for x in rng.integers(0, 600, b)]
    c = Case(lens, ctx, m=4, k=0, fmt=L.CSA_BF16, seed=71, **TC).run()
    c.rows64 = c.values()
    full = c.b
    # a sample of the sequences
    keep = [s for s in range(full) if lens[s]][:: max(1, full // 12)]
    q, win, nw, sink = f64(c.q), f64(c.win), f64(c.new_win), f64(c.sink)
    for s in keep:
        for i in range(lens[s]):
            _, rows = chunk.chunk_rows(s, i, c.entry, None, ctx[s], c.cu[s], 4, c.bt.shape[1] * PE, win, nw, 128)
            o, l, A = chunk.attend(q[c.cu[s] + i], rows, sink, c.p.scale)
            # the weights' and the result's bf16 rounding, 2^-8 each, and the logits' error
            # (2 A scale |q|.|row| 2^-14, below 2^-8 A at these sizes)
            assert np.all(np.abs(f64(c.out[c.cu[s] + i]) - o) <= 2.0 ** -8 * (2 * A + np.abs(o)))


def test_cache_and_attention_past_32_bits():
    """Pages whose rows start beyond 2^31 elements (4 GiB of bf16): written, read, attended to."""
    pages = (1 << 31) // (512 * PE) + 3
    kv_rows = torch.empty((pages * PE, 512), dtype=torch.bfloat16, device="cuda")
    bt = i32([[pages - 1, pages - 2, 0]])
    kv = L.kv_cache(L.CSA_BF16, 512, 0, kv_rows, None, None, bt)
    x = randn(1, (600, 512), torch.bfloat16)
    L.csa_cache_write(kv, L.CSA_BF16, x, i32([0, 600]), i32([0]), 1, 600)
    assert torch.equal(kv_rows[(pages - 1) * PE:], x[:256])
    out = torch.empty((1, 600, 512), dtype=torch.bfloat16, device="cuda")
    L.csa_cache_read(kv, None, None, 1, 600, L.CSA_BF16, out)
    assert torch.equal(out[0], x)
    # the same rows in a small pool give the same attention, bit for bit
    small = L.kv_cache(L.CSA_BF16, 512, 0, torch.zeros((3 * PE, 512), dtype=torch.bfloat16, device="cuda"), None,
                       None, i32([[2, 0, 1]]))
    L.csa_cache_write(small, L.CSA_BF16, x, i32([0, 600]), i32([0]), 1, 600)
    p = L.AttnParams(H=64, d=512, n_w=128, scale=1.0 / math.sqrt(512), m=4, k=0, dtype=L.CSA_BF16)
    res = []
    for c in (kv, small):
        for n in (5, 310):                           # split rows, and one CTA a token
            q, nw, win = (randn(2, (n, 64, 512), torch.bfloat16), randn(3, (n, 512), torch.bfloat16),
                          randn(4, (1, 128, 512), torch.bfloat16))
            o = torch.empty_like(q)
            ws = torch.empty(max(16, L.csa_chunk_attn_workspace_size(p, c, 1, n, 2400)), dtype=torch.uint8,
                             device="cuda")
            L.csa_chunk_attn(p, c, q, i32([0, n]), i32([2400 - n]), None, None, win, nw, randn(5, (64,)), 1, n,
                             2400, o, None, ws)
            res.append(o)
    assert torch.equal(res[0], res[2]) and torch.equal(res[1], res[3])


def test_chunk_attn_workspace_is_checked():
    c = Case([3], [5000], m=4, k=512, fmt=L.CSA_BF16, seed=81, **TC)
    need = L.csa_chunk_attn_workspace_size(c.p, c.kv, c.b, c.N, c.L_max)
    assert need > 0 and L.csa_chunk_attn_launch_count(c.p, c.kv, c.b, c.N, c.L_max) == 2
    args = (c.p, c.kv, c.q, i32(c.cu), i32(c.ctx), c.idx, c.count, c.win, c.new_win, c.sink, c.b, c.N, c.L_max,
            c.out, c.lse)
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 16, dtype=torch.uint8, device="cuda")[4:]):
        with pytest.raises(L.CsaError):
            L.csa_chunk_attn(*args, ws)
    with pytest.raises(L.CsaError):                  # a type, a size, a table too short, a place
        L.csa_chunk_attn(*args[:2], c.q.float(), *args[3:], c.ws)
    with pytest.raises(L.CsaError):
        L.csa_chunk_attn(*args[:2], c.q[:-1], *args[3:], c.ws)
    with pytest.raises(L.CsaError):
        L.csa_cache_read(c.kv, None, None, 2, 4, L.CSA_BF16, torch.empty((2, 4, 512), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(L.CsaError):
        L.csa_cache_read(c.kv, None, None, 1, 4, L.CSA_BF16, torch.empty((1, 4, 512), dtype=torch.bfloat16))
    assert torch.all(c.out == 7.0)


def _steps(c):
    """The five calls on one case's tensors (outputs of the case's shapes)."""
    def run():
        L.csa_qk_norm_rope(c.np_, c.q, None, c.new_win, None, c.pos, c.N, c.q2, c.w2)
        L.csa_cache_write(c.kv, L.CSA_BF16, c.rows_in, c.wcu, c.wfirst, c.b, c.rows_in.shape[0])
        L.csa_chunk_attn(c.p, c.kv, c.q2, c.dcu, c.dctx, None, None, c.win, c.w2, c.sink, c.b, c.N, c.L_max, c.out,
                         c.lse, c.ws)
        L.csa_window_append(L.CSA_BF16, c.d, c.n_w, c.win2, c.w2, c.dcu, c.dctx, c.b, c.N)
        L.csa_cache_read(c.kv, None, None, c.b, 64, L.CSA_BF16, c.back)
    return run


def _step_case(seed, fmt, d_hi):
    c = Case([5, 33], [1000, 40], m=4, k=0, fmt=fmt, d_hi=d_hi, d_rope_out=64, seed=seed, **TC)
    c.np_ = L.NormRopeParams(H=64, d=512, d_rope=64, rope_theta=THETA, eps=EPS, apply_norm=1, dtype=L.CSA_BF16)
    c.pos = i32([1000 + i for i in range(5)] + [40 + i for i in range(33)] + [0] * (c.N - 38))
    c.q2, c.w2, c.win2 = torch.zeros_like(c.q), torch.zeros_like(c.new_win), c.win.clone()
    c.rows_in = randn(seed + 9, (12, 512), torch.bfloat16)
    c.wcu, c.wfirst = i32([0, 4, 12]), i32([246, 10])
    c.dcu, c.dctx = i32(c.cu), i32(c.ctx)
    c.back = torch.zeros((2, 64, 512), dtype=torch.bfloat16, device="cuda")
    return c


def _results(c):
    return [x.clone() for x in (c.q2, c.w2, c.out, c.lse, c.win2, c.back)]


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
def test_captured_calls_follow_their_tensors(fmt, d_hi):
    """A captured sequence of the calls, replayed on other values in the same tensors, gives what
    the calls give on those values."""
    a, b = _step_case(91, fmt, d_hi), _step_case(92, fmt, d_hi)
    run = _steps(a)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    names = ("q", "new_win", "win", "win2", "sink", "rows_in", "pos", "dcu", "dctx", "wcu", "wfirst")
    b.dcu, b.dctx = i32([0, 30, 38]), i32([77, 1300])          # other lengths and positions too
    b.wfirst = i32([3, 300])
    for n in names:
        getattr(a, n).copy_(getattr(b, n))
    # the other case's pages and table
    for x, y in zip(a.kv._tensors, b.kv._tensors):
        if x is not None:
            x.copy_(y)
    for x in (a.out, a.lse):
        x.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    got = _results(a)
    _steps(b)()
    torch.cuda.synchronize()
    for x, y in zip(got, _results(b)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
def test_two_streams_at_once(fmt, d_hi):
    """Two independent sequences of the calls on two streams, many times over, and the same on one
    stream: the same bits (no state shared between calls)."""
    a, b = _step_case(101, fmt, d_hi), _step_case(102, fmt, d_hi)
    want = []
    for c in (a, b):
        _steps(c)()
        torch.cuda.synchronize()
        want.append(_results(c))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for c, s in ((a, s1), (b, s2)):
            with torch.cuda.stream(s):
                _steps(c)()
    torch.cuda.synchronize()
    assert L.csa_device_error() == 0
    for c, w in zip((a, b), want):
        for x, y in zip(_results(c), w):
            assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", [L.CSA_BF16, L.CSA_FP8_E4M3])
@pytest.mark.parametrize("m,n", [(4, 700), (128, 1500)])
def test_a_sequence_served_in_chunks(fmt, m, n):
    """A prompt brought in chunks of every size, its entries compressed, written to pages and
    attended to chunk by chunk, against one dense call over the whole sequence.

    Tolerance: both calls round their weights (2^-8) and results (2^-8) to bf16, so they differ by
    at most twice 2^-8 (A + |o|) with A = sum w |row| <= max |row| over the sequence's rows; the
    float32 parts are far below.  A is taken from the whole call's rows."""
    d, H, n_w = 512, 64, 128
    raw = {k: randn(i, (1, n, d), torch.bfloat16) for i, k in enumerate(("C", "Z"))}
    Bp = randn(7, (m, d))
    E = n // m
    cp = L.CompressParams(m=m, overlap=0, c=d, d_rope=64, rope_theta=THETA, eps=EPS, apply_norm=1,
                          in_dtype=L.CSA_BF16, out_dtype=L.CSA_BF16, out_entry_offset=0)
    ent = torch.zeros((1, E, d), dtype=torch.bfloat16, device="cuda")
    L.csa_compress(cp, raw["C"], raw["Z"], Bp, None, None, None, 1, n, 0, E, E, ent)
    qraw, kraw = randn(8, (n, H, d), torch.bfloat16), raw["C"][0]
    nrm = L.NormRopeParams(H=H, d=d, d_rope=64, rope_theta=THETA, eps=EPS, apply_norm=1, dtype=L.CSA_BF16)
    sink = randn(9, (H,))
    pages = -(-E // PE) + 1
    bt = i32([[(3 * j + 1) % pages if pages % 3 else j for j in range(-(-E // PE))]])
    kv = L.alloc_kv_cache(fmt, d, 64 if fmt == L.CSA_FP8_E4M3 else 0, pages, bt)
    win = torch.zeros((1, n_w, d), dtype=torch.bfloat16, device="cuda")
    p = L.AttnParams(H=H, d=d, n_w=n_w, scale=1.0 / math.sqrt(d), m=m, k=0, dtype=L.CSA_BF16, d_rope_out=64,
                     rope_theta=THETA)
    q_all, w_all = torch.empty_like(qraw), torch.empty_like(kraw)
    outs, lses, at = [], [], 0
    for size in (1, 2, 37, 128, 300, n):
        size = min(size, n - at)
        if not size:
            break
        pos = torch.arange(at, at + size, dtype=torch.int32, device="cuda")
        q, w = q_all[at:at + size], w_all[at:at + size]
        L.csa_qk_norm_rope(nrm, qraw[at:at + size], None, kraw[at:at + size], None, pos, size, q, w)
        e0, e1 = at // m, (at + size) // m           # the entries this chunk completes
        if e1 > e0:
            L.csa_cache_write(kv, L.CSA_BF16, ent[0, e0:e1], i32([0, e1 - e0]), i32([e0]), 1, e1 - e0)
        o, l = torch.empty_like(q), torch.empty((size, H), device="cuda")
        ws = torch.empty(max(16, L.csa_chunk_attn_workspace_size(p, kv, 1, size, at + size)), dtype=torch.uint8,
                         device="cuda")
        L.csa_chunk_attn(p, kv, q, i32([0, size]), i32([at]), None, None, win, w, sink, 1, size, at + size, o, l, ws)
        L.csa_window_append(L.CSA_BF16, d, n_w, win, w, i32([0, size]), i32([at]), 1, size)
        outs.append(o)
        lses.append(l)
        at += size
    # the whole sequence at once, over the rows the cache stands for
    rows = torch.empty((1, E, d), dtype=torch.bfloat16, device="cuda")
    L.csa_cache_read(kv, None, None, 1, E, L.CSA_BF16, rows)
    if fmt == L.CSA_BF16:
        assert torch.equal(rows, ent)
    out, lse = torch.empty((1, n, H, d), dtype=torch.bfloat16, device="cuda"), torch.empty((1, n, H), device="cuda")
    wsz = L.csa_sparse_attn_workspace_size(p, 1, n, E)
    L.csa_sparse_attn(p, q_all[None], rows, E, None, None, w_all[None].contiguous(), n,
                      torch.arange(n, dtype=torch.int32, device="cuda")[None], sink, 1, n, out, lse,
                      torch.empty(max(16, wsz), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert L.csa_device_error() == 0
    A = max(float(rows.abs().max()), float(w_all.abs().max())) * math.sqrt(2.0)   # a rotated pair mixes
    err = (torch.cat(outs).float() - out[0].float()).abs().max()
    assert float(err) <= 2 * 2.0 ** -8 * 2 * A
    # the lse: the whole call sums rounded weights (2^-8 each, relative)
    assert float((torch.cat(lses) - lse[0]).abs().max()) <= 2.0 ** -8 + 2.0 ** -14 * 100


@pytest.mark.parametrize("shape", ["tc", "small"])
@pytest.mark.parametrize("lens", [[1, 1, 3], [2, 150, 160]])
def test_chunk_attn_last_positions(shape, lens):
    """Tokens up to position 2^31 - 2, the last one that a bound on t + 1 can name: the ends of
    their windows' tiles lie past 2^31."""
    last = 2 ** 31 - 2
    cfg = dict(TC, fmt=L.CSA_BF16) if shape == "tc" else dict(SMALL)
    cfg.update(m=2 ** 31 - 1, n_w=140)
    c = Case(lens, [last + 1 - n for n in lens], k=0, seed=131, **cfg)
    c.run().check(tokens=5)


def test_one_workspace_for_all_batches():
    """A workspace for the largest batch and context, used by calls of every smaller size: what a
    call of its own size's workspace gives."""
    big = Case([300], [30000], m=4, k=0, seed=141, fmt=L.CSA_BF16, **TC)
    ws = torch.full((L.csa_chunk_attn_workspace_bound(big.p, big.kv, 3, big.N, big.L_max),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    assert ws.numel() > L.csa_chunk_attn_workspace_size(big.p, big.kv, 1, big.N, big.L_max)
    for lens, ctx in (([300], [30000]), ([1], [30000]), ([1, 1, 1], [20000, 9, 30000]), ([148], [7000]),
                      ([150], [30000]), ([33, 2], [500, 29000])):
        c = Case(lens, ctx, m=4, k=0, seed=142, fmt=L.CSA_BF16, **TC).run()
        out, lse = c.out.clone(), c.lse.clone()
        c.out.fill_(7.0)
        c.ws = ws
        c.run()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse), lens


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
@pytest.mark.parametrize("role", [1, 2, 3])
@pytest.mark.parametrize("lens,ctx,k", [([5, 3], [2500, 900], 0), ([5, 3], [2500, 900], 64), ([310, 40], [700, 0], 0)])
def test_chunk_attn_a_wait_given_up(fmt, d_hi, role, lens, ctx, k):
    """Whichever warps' wait gives up: the error word is set and the outputs are NaN, never silently
    wrong; the next call is right again."""
    assert L.csa_device_error() == 0
    c = Case(lens, ctx, m=4, k=k, seed=151, fmt=fmt, d_hi=d_hi, d_rope_out=64, **TC)
    n = c.cu[-1]
    L.csa_selftest_chunk_give_up(role)
    with pytest.raises(AssertionError):
        c.run()                                      # (its own look at the error word)
    assert L.csa_device_error() == 0
    assert torch.all(torch.isnan(c.out[:n])) and torch.all(torch.isnan(c.lse[:n]))
    assert torch.all(c.out[n:] == 7.0) and torch.all(c.lse[n:] == 7.0)
    c.run().check(tokens=3)


@pytest.mark.parametrize("fmt,d_hi", [(L.CSA_BF16, 0), (L.CSA_FP8_E4M3, 64)])
@pytest.mark.parametrize("lens,ctx", [([300], [2500]), ([5, 3], [2500, 900])])
def test_chunk_attn_a_head_that_starts_with_infinities(fmt, d_hi, lens, ctx):
    """Head 0's logits are -inf (past float32) on the first 128 entries and all the same far
    negative number on the other rows: it weighs those alike, however low they lie."""
    c = Case(lens, ctx, m=4, k=0, seed=161, fmt=fmt, d_hi=d_hi, sink=-math.inf, **TC)
    big, low = 3.0e38, 4096.0
    pool = randn(162, (c.kv.num_pages * PE, c.d))
    pool[:, 0], pool[:, 100] = 0.0, 1.0
    for s in range(c.b):
        for e in range(128):
            pool[place(c.bt, s, e), :64] = 0.0
            pool[place(c.bt, s, e), 0] = big
    flat = L.kv_cache(fmt, c.d, d_hi, *c.kv._tensors[:3], i32([list(range(c.kv.num_pages))]))
    L.csa_cache_write(flat, L.CSA_F32, pool, i32([0, len(pool)]), i32([0]), 1, len(pool))
    for w in (c.win, c.new_win):
        w[..., 0], w[..., 100] = 0.0, 1.0
    c.q[:, :, 0] = 0.0
    c.q[:, 0] = 0.0
    c.q[:, 0, 0], c.q[:, 0, 100] = -big, -low
    c.run()
    c.rows64 = c.values()
    win, nw = f64(c.win), f64(c.new_win)
    # (the other heads' sums of 3e38 in dim 0, not yet divided by the denominator, pass float32)
    assert torch.all(torch.isfinite(c.out[:c.cu[-1], 0].float())) and torch.all(torch.isfinite(c.out[:c.cu[-1], :, 1:].float()))
    for s in range(c.b):
        for i in {0, 1, lens[s] - 1}:
            _, rows = chunk.chunk_rows(s, i, c.entry, None, ctx[s], c.cu[s], 4, c.bt.shape[1] * PE, win, nw, 128)
            rows = np.asarray(rows)
            seen = rows[rows[:, 0] == 0.0]
            assert len(rows) == len(seen) + 128
            logit = -low * c.p.scale * seen[0, 100]
            # equal weights: one sum of R rows, and the result's rounding; the lse as in check()
            tol = 2.0 ** -8 * np.abs(seen.mean(0)) + len(seen) * 2.0 ** -23 * np.abs(seen).mean(0)
            row = c.cu[s] + i
            assert np.all(np.abs(f64(c.out[row, 0]) - seen.mean(0)) <= tol + 1e-30), (s, i)
            lse = logit + math.log(len(seen))
            assert abs(float(c.lse[row, 0]) - lse) <= abs(logit) * 2.0 ** -14 + 2.0 ** -20 + 2.0 ** -22 * abs(lse)


# -------------------------------------------------------- calls large enough for several rows per warp

@pytest.mark.parametrize("dtype,d,d_rope", [
    (L.CSA_BF16, 128, 64), (L.CSA_F32, 128, 64), (L.CSA_BF16, 256, 0), (L.CSA_F32, 40, 6), (L.CSA_F32, 512, 64),
    (L.CSA_BF16, 1000, 64), (L.CSA_F32, 1024, 128), (L.CSA_BF16, 2048, 64), (L.CSA_F32, 1800, 64),
])
@pytest.mark.parametrize("norm", [0, 1])
def test_norm_rope_many_rows(dtype, d, d_rope, norm):
    """Enough rows for several per warp, with a rest: within the oracle's bound, and the same bits as
    calls of few tokens (the same operations in the same order)."""
    N, H = 6401, 2
    test_norm_rope(dtype, N, H, d, d_rope, bool(norm), True, norm)
    dt = TDT[dtype]
    q, kv = randn(171, (N, H, d), dt), randn(172, (N, d), dt)
    g = 1 + 0.2 * randn(173, (d,)) if norm else None
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 163
    p = L.NormRopeParams(H=H, d=d, d_rope=d_rope, rope_theta=THETA, eps=EPS, apply_norm=norm, dtype=dtype)
    for use_q, use_kv in ((True, True), (False, True)) if d == 128 else ((True, True),):
        n = N if use_q else 4 * N
        if not use_q:
            kv, pos = randn(174, (n, d), dt), torch.arange(n, dtype=torch.int32, device="cuda")
        outs = []
        for step in (n, 1000):
            qo = torch.full_like(q, 7.0) if use_q else None
            ko = torch.full_like(kv, 7.0)
            for a in range(0, n, step):
                z = min(a + step, n)
                L.csa_qk_norm_rope(p, q[a:z] if use_q else None, g if use_q else None, kv[a:z], g, pos[a:z], z - a,
                                   qo[a:z] if use_q else None, ko[a:z])
            outs.append((qo, ko))
        assert torch.equal(outs[0][1], outs[1][1])
        assert not use_q or torch.equal(outs[0][0], outs[1][0])


@pytest.mark.parametrize("x_dtype,c,d_hi,lens,first", [
    (L.CSA_F32, 512, 64, [39000, 77], [0, 9]),
    (L.CSA_BF16, 1104, 16, [12, 37999, 0, 1], [250, 3, 0, 0]),
    (L.CSA_F32, 64, 0, [1, 38001], [0, 255]),
])
def test_cache_write_many_rows(x_dtype, c, d_hi, lens, first):
    test_cache_write_and_read(L.CSA_FP8_E4M3, x_dtype, c, d_hi, lens, first)


@pytest.mark.parametrize("c,d_hi", [(512, 64), (1104, 16), (64, 0)])
@pytest.mark.parametrize("out_dtype", [L.CSA_BF16, L.CSA_F32])
def test_cache_read_many_rows(c, d_hi, out_dtype):
    """An odd number of slots, enough for two rows per warp, whose pairs mix rows that exist with
    ones past a count, past the table and on pages outside the pool: what reads of few slots give."""
    b, k, entries = 3, 13001, 700
    total, bt = table([entries] * b, seed=181, extra=2)
    bt[1, 1] = total + 5
    kv = cache_of(L.CSA_FP8_E4M3, c, d_hi, total, bt)
    flat = L.kv_cache(L.CSA_FP8_E4M3, c, d_hi, *kv._tensors[:3], i32([list(range(total))]))
    pool = randn(182, (total * PE, c))
    L.csa_cache_write(flat, L.CSA_F32, pool, i32([0, total * PE]), i32([0]), 1, total * PE)
    rng = np.random.default_rng(183)
    idx = torch.from_numpy(rng.integers(-40, entries + 400, (b, k)).astype(np.int32)).cuda()
    for sel, counts in ((idx, [k, 12345, 1]), (idx, None), (None, [k, 601, 0])):
        count = None if counts is None else i32(counts)
        out = torch.full((b, k, c), float("nan"), dtype=TDT[out_dtype], device="cuda")
        L.csa_cache_read(kv, sel, count, b, k, out_dtype, out)
        assert not torch.isnan(out).any()
        step = 5000 if sel is not None else k        # (entry j of slot j: a slice starts at 0 again)
        for s in range(b):
            part = L.kv_cache(L.CSA_FP8_E4M3, c, d_hi, *kv._tensors[:3], i32([bt[s].tolist()]))
            for a in range(0, k, step):
                z = min(a + step, k)
                want = torch.empty((1, z - a, c), dtype=TDT[out_dtype], device="cuda")
                n = None if counts is None else i32([min(max(counts[s] - a, 0), z - a)])
                L.csa_cache_read(part, None if sel is None else sel[s:s + 1, a:z].contiguous(), n, 1, z - a, out_dtype, want)
                assert torch.equal(out[s, a:z], want[0]), (s, a)
    # a sample of the last read's rows against the oracle
    arrs = [None if t is None else t.cpu() for t in kv._tensors[:3]]
    L.csa_cache_read(kv, idx, None, b, k, out_dtype, out)
    for s in range(b):
        for j in (0, 1, 2, k // 2, k - 2, k - 1):
            e = int(idx[s, j])
            if not (0 <= e < bt.shape[1] * PE and 0 <= bt[s, e // PE] < total):
                assert torch.all(out[s, j] == 0)
                continue
            at = place(bt, s, e)
            hi = f64(arrs[1][at]) if d_hi else np.zeros(0)
            ref = chunk.dequant_row(arrs[0][at].numpy(), hi, arrs[2][at].numpy()[: (c - d_hi) // 64])
            assert np.array_equal(f64(out[s, j]), ref), (s, j, e)


@pytest.mark.parametrize("fmt,d_hi,shape", [(L.CSA_BF16, 0, "tc"), (L.CSA_FP8_E4M3, 64, "tc"), (L.CSA_F32, 0, "small")])
@pytest.mark.parametrize("lens,ctx,k", [([5, 3], [2500, 900], 0), ([310, 4], [2500, 900], 64), ([310, 4], [2500, 90], 0)])
def test_chunk_attn_repeats_itself(fmt, d_hi, shape, lens, ctx, k):
    """The same call gives the same bits every time (no sum depends on the order of arrival)."""
    cfg = dict(TC, m=4) if shape == "tc" else dict(SMALL)
    cfg["fmt"] = fmt
    c = Case(lens, ctx, k=k, d_hi=d_hi, seed=191, **cfg).run()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(10):
        c.out.fill_(7.0)
        c.run()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("k", [0, 70])
@pytest.mark.parametrize("over", [
    dict(H=3, d=136), dict(H=2, d=256, d_rope_out=64), dict(H=2, d=1000, n_w=70),
    dict(H=16, d=512, dtype=L.CSA_BF16, fmt=L.CSA_BF16, d_rope_out=64),
    dict(H=16, d=512, dtype=L.CSA_BF16, fmt=L.CSA_FP8_E4M3, d_hi=64, d_rope_out=64),
    dict(H=64, d=512, dtype=L.CSA_BF16, fmt=L.CSA_BF16, d_rope_out=128),    # more rotary dims than the tensor cores' form
    dict(H=5, d=576, fmt=L.CSA_FP8_E4M3, d_hi=64, d_rope_out=64),
])
def test_chunk_attn_any_shape_wide_heads(k, over):
    """Head dims past 128, where a thread of the CUDA-core kernel takes one or several channels alone."""
    cfg = dict(SMALL, **over)
    Case([4, 0, 1, 17], [0, 9, 1027, 300], k=k, seed=201, **cfg).run().check()
