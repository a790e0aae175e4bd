"""Serving a chunk of new tokens over a paged latent cache, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The quantised cache row, the norm and rotation of query heads and latent rows, and the
attention of a ragged chunk, each from its definition and one token at a time.  Sources:
"DeepSeek V4 结构速览", sections "HCA（c128a 路线）" (RMSNorm and partial RoPE of the heads;
sink) and "CSA（c4a 路线）" (selected entries, then the window); "DeepSeek-V4 技术解读",
section 3.2 (paged classical cache, window state).
"""

import numpy as np

from . import codecs, csa

GROUP = 64
K_MIN, K_MAX = -110, 119


def norm_rope(x, gain, pos, d_rope, theta, eps, apply_norm=True):
    """Rows x [R][d] (one position per row) normalised, scaled by gain and rotated."""
    y = np.asarray(x, dtype=np.float64)
    if apply_norm:
        y = csa.rms_norm(y, eps)
        if gain is not None:
            y = y * np.asarray(gain, dtype=np.float64)
    return csa.rope_partial(y, pos, d_rope, theta)


def scale_exponent(amax):
    """Smallest k with amax <= 448 * 2^k, kept in [K_MIN, K_MAX]; K_MIN for amax = 0."""
    amax = float(amax)
    if amax == 0.0:
        return K_MIN
    if np.isinf(amax):
        return K_MAX
    k = int(np.floor(np.log2(amax / 448.0))) - 2
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return min(max(k, K_MIN), K_MAX)


def quant_row(x, d_hi):
    """(codes uint8 [c - d_hi], last d_hi dims rounded to bf16, exponent bytes) of one row."""
    x = np.asarray(x, dtype=np.float64)
    nc = x.shape[0] - d_hi
    codes = np.zeros(nc, dtype=np.uint8)
    exps = np.zeros(nc // GROUP, dtype=np.uint8)
    for g in range(nc // GROUP):
        v = x[GROUP * g:GROUP * (g + 1)]
        num = v[~np.isnan(v)]
        k = scale_exponent(np.max(np.abs(num)) if num.size else 0.0)
        with np.errstate(invalid="ignore"):
            y = np.clip(v * 2.0 ** -k, -448.0, 448.0)
        c = codecs.e4m3_encode(np.where(np.isnan(y), 0.0, y)).astype(np.uint8)
        codes[GROUP * g:GROUP * (g + 1)] = np.where(np.isnan(v), 0x7F, c)
        exps[g] = k + 127
    return codes, codecs.round_to_bf16(x[nc:]), exps


def dequant_row(codes, hi, exps):
    """The float64 values a quantised row stands for."""
    v = codecs.e4m3_decode(codes).reshape(-1, GROUP)
    s = 2.0 ** (np.asarray(exps, dtype=np.float64) - 127.0)
    return np.concatenate([(v * s[:, None]).reshape(-1), np.asarray(hi, dtype=np.float64)])


def chunk_rows(s, i, entries_of, idx, pos0, cu, m, cap, win, new_win, n_w):
    """Rows that token i of sequence s attends to: its entries' rows, then its window's.

    entries_of(s, e) is entry e's row or None (not in the table or the pool); idx the
    token's selection or None; cap the entries a block table spans.
    """
    t = pos0 + i
    rows = []
    if t >= 0:
        sel = range(min((t + 1) // m, cap)) if idx is None else idx
        for e in sel:
            r = entries_of(s, int(e)) if 0 <= e < cap else None
            if r is not None:
                rows.append(r)
        for u in csa.window_rows(t, n_w):
            rows.append(new_win[cu + u - pos0] if u >= pos0 else win[s][u % n_w])
    return t, rows


def attend(q, rows, sink, scale):
    """csa.attend that also takes a sink of -inf and no rows, and returns the weights' sums of
    |row| (what a relative error of the weights is measured against)."""
    H, d = q.shape
    if not rows:
        return np.zeros((H, d)), np.asarray(sink, dtype=np.float64).copy(), np.zeros((H, d))
    R = np.asarray(rows, dtype=np.float64)
    lg = scale * (np.asarray(q, dtype=np.float64) @ R.T)
    mx = np.maximum(lg.max(axis=1), sink)
    e = np.exp(lg - mx[:, None])
    den = e.sum(axis=1) + np.exp(sink - mx)
    return (e @ R) / den[:, None], mx + np.log(den), (e @ np.abs(R)) / den[:, None]
