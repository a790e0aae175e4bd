"""Measured cases of the operators that serve a chunk of new tokens over a paged cache.

  norm_rope   csa_qk_norm_rope: RMSNorm of every query head and of the token's latent row,
              and the rotation of their last dims at the token's position, in one pass.
  write       csa_cache_write: latent rows into the pages of their sequences, as bf16 / fp32
              rows or quantised (E4M3 codes with a power-of-two scale per 64 dims, the last
              dims in bf16).
  read        csa_cache_read: rows of a paged cache gathered back as plain rows.
  attn        csa_chunk_attn: attention of ragged chunks of new tokens over paged entries
              (every visible one, or a selection per token) and the sliding window.

With ``own`` false, ``run`` computes the operators from elementary torch operations in 32
bits; with ``own`` true it calls the library.
"""

import math

import numpy as np
import torch

own = False

PAGE = 256          # entries per page
GROUP = 64          # dims sharing one scale of a quantised row
THETA = 10000.0
EPS = 1e-6
K_MIN, K_MAX = -110, 119   # scale exponents of a quantised row


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 16 sequences: the smallest call of a decode step
        dict(name="norm_rope_decode", op="norm_rope", N=16, H=64, d=512, d_rope=64, dtype="bf16",
             gain=True, strided=False, L=65536),
        # a chunk of a long prompt, q and the latent row side by side in one projection output
        dict(name="norm_rope_chunk", op="norm_rope", N=4096, H=64, d=512, d_rope=64, dtype="bf16",
             gain=True, strided=True, L=1048576),
        # the entry that each of 16 decoding sequences has just completed
        dict(name="write_decode", op="write", lens="1," * 15 + "1", c=512, d_hi=64, fmt="fp8",
             x="bf16", ctx=16384),
        # every entry of three prompts, 1M tokens of them at four tokens an entry
        dict(name="write_prompts", op="write", lens="200001,50001,12142", c=512, d_hi=64, fmt="fp8",
             x="bf16", ctx=1000),
        # the selection of one decode step over 64K tokens, for a kernel that takes plain rows
        dict(name="read_selection", op="read", b=16, k=512, ragged=True, select=True, c=512,
             d_hi=64, fmt="fp8", out="bf16", ctx=16384),
        # a cached prompt of 1M tokens taken out whole
        dict(name="read_prompt", op="read", b=1, k=262144, ragged=False, select=False, c=512,
             d_hi=64, fmt="fp8", out="bf16", ctx=262144),
        # one new token for each of 8 sequences of 1M tokens, 128 tokens an entry
        dict(name="attn_single_1m", op="attn", lens="1," * 7 + "1", ctx="1048575," * 7 + "1000000",
             H=64, d=512, m=128, k=0, n_w=128, fmt="bf16", d_hi=0, d_rope_out=64),
        # a few drafted tokens to verify for each of 16 sequences of up to 64K tokens
        dict(name="attn_drafts_64k", op="attn", lens="4,1,8,3,5,2,7,4,4,6,1,8,2,3,5,4",
             ctx="65528," * 8 + "40001," * 7 + "130", H=64, d=512, m=4, k=512, n_w=128, fmt="fp8",
             d_hi=64, d_rope_out=64),
        # a prefill chunk shared by two prompts, each token with its own selection
        dict(name="attn_chunk_selected", op="attn", lens="1333,2763", ctx="62773,0", H=64, d=512,
             m=4, k=512, n_w=128, fmt="fp8", d_hi=64, d_rope_out=64),
        # the last chunk of a prompt of 1M tokens over every entry
        dict(name="attn_chunk_dense_1m", op="attn", lens="2048", ctx="1046528", H=64, d=512, m=128,
             k=0, n_w=128, fmt="bf16", d_hi=0, d_rope_out=64),
        # a mixed batch: short and long chunks, a single token, short and long contexts
        dict(name="attn_mixed_dense", op="attn", lens="1,37,500,129,261", ctx="700001,0,131,30000,255000",
             H=64, d=512, m=128, k=0, n_w=128, fmt="fp8", d_hi=64, d_rope_out=64),
        # the small 32-bit configuration
        dict(name="attn_f32_small", op="attn", lens="64,1,33", ctx="960,17,300", H=4, d=64, m=4, k=16,
             n_w=16, fmt="f32", d_hi=0, d_rope_out=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "write", "read", "attn", "attn", "attn"])
    if op == "norm_rope":
        f32 = rng.random() < 0.25
        H, d = (rng.randint(1, 8), 8 * rng.randint(1, 32)) if f32 else (64, rng.choice([128, 512]))
        return dict(op=op, N=_log(rng, 1, 4096), H=H, d=d, d_rope=min(d, rng.choice([16, 64])) // 2 * 2,
                    dtype="f32" if f32 else "bf16", gain=rng.random() < 0.7,
                    strided=rng.random() < 0.5, L=_log(rng, 16, 1 << 20))
    if op == "write":
        b = rng.randint(1, 16)
        fmt = rng.choice(["fp8", "fp8", "bf16"])
        return dict(op=op, lens=",".join(str(_log(rng, 1, 16384)) for _ in range(b)), c=512,
                    d_hi=64 if fmt == "fp8" else 0, fmt=fmt, x="bf16", ctx=_log(rng, 1, 16384))
    if op == "read":
        b = rng.randint(1, 16)
        fmt = rng.choice(["fp8", "fp8", "bf16"])
        ctx = _log(rng, 1, 16384)
        sel = rng.random() < 0.6
        return dict(op=op, b=b, k=rng.choice([512, 1024, 37]) if sel else ctx, ragged=sel,
                    select=sel, c=512, d_hi=64 if fmt == "fp8" else 0, fmt=fmt, out="bf16", ctx=ctx)
    kind = rng.random()
    if kind < 0.15:
        b = rng.randint(1, 4)
        d = 8 * rng.randint(2, 16)
        return dict(op=op, lens=",".join(str(_log(rng, 1, 96)) for _ in range(b)),
                    ctx=",".join(str(rng.randint(0, 2000)) for _ in range(b)), H=rng.randint(1, 8), d=d,
                    m=rng.choice([4, 128]), k=rng.choice([0, 16]), n_w=rng.choice([16, 128]), fmt="f32",
                    d_hi=0, d_rope_out=rng.choice([0, 16]))
    b = rng.choice([1, 1, 2, 3, 5, 8, 16])
    fmt = rng.choice(["fp8", "bf16"])
    sel = rng.random() < 0.5
    most = max(1, (4096 if sel else 2048) // b)
    top = 65536 if sel else 1 << 20
    lens = [_log(rng, 1, most) for _ in range(b)]
    return dict(op=op, lens=",".join(map(str, lens)),
                ctx=",".join(str(min(top - n, _log(rng, 1, top) - 1)) for n in lens), H=64, d=512,
                m=4 if sel else 128, k=512 if sel else 0, n_w=128, fmt=fmt,
                d_hi=64 if fmt == "fp8" else 0, d_rope_out=rng.choice([0, 64]))


def _ints(text):
    return [int(v) for v in text.split(",")]


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lens):
    return [0] + [int(v) for v in np.cumsum(lens)]


def _rows(g, n, c, dtype):
    """Latent rows as a normalised compressor writes them: unit rms, a few large channels."""
    x = _randn(g, (n, c))
    x *= torch.exp(0.5 * _randn(g, (c,)))
    x *= torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x.to(dtype)


def _tables(entries, seed):
    """Pages for sequences of the given entries, in a shuffled order, and the block table."""
    need = [max(1, -(-e // PAGE)) for e in entries]
    total = sum(need) + 1
    perm = np.random.default_rng(int(seed)).permutation(total)
    bt = np.full((len(entries), max(need)), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = perm[at:at + n]
        at += n
    return total, torch.from_numpy(bt).cuda()


def _quantise(x, d_hi):
    """(codes, last dims in bf16, scale exponents + 127) of rows x, from the format's definition."""
    c = x.shape[-1]
    y = x[:, : c - d_hi].double().reshape(x.shape[0], -1, GROUP)
    top = y.abs().nan_to_num(nan=0.0, posinf=3.4e38).amax(-1)
    mant, ex = torch.frexp(top)                       # top = mant 2^ex, mant in [0.5, 1)
    k = torch.where(mant * 2 <= 1.75, ex - 9, ex - 8)
    k = torch.where(top == 0, K_MIN, k).clamp(K_MIN, K_MAX)
    v = (y * torch.exp2(-k.double())[..., None]).clamp(-448.0, 448.0)
    codes = v.float().to(torch.float8_e4m3fn).reshape(x.shape[0], c - d_hi)
    return codes, x[:, c - d_hi:].to(torch.bfloat16), (k + 127).to(torch.uint8)


def _alloc_cache(fmt, total, c, d_hi):
    """The arrays of a paged cache: rows; or codes, last dims and scales."""
    n = total * PAGE
    if fmt != "fp8":
        return dict(rows=torch.zeros((n, c), dtype=_dt(fmt), device="cuda"), hi=None, scales=None)
    ns = (c - d_hi) // GROUP
    return dict(rows=torch.zeros((n, c - d_hi), dtype=torch.uint8, device="cuda"),
                hi=torch.zeros((n, d_hi), dtype=torch.bfloat16, device="cuda"),
                scales=torch.zeros((n, -(-ns // 8) * 8), dtype=torch.uint8, device="cuda"))


def _fill_cache(a, g, fmt, c, d_hi):
    """Every row of a cache given values, a block of rows at a time."""
    n = a["rows"].shape[0]
    for at in range(0, n, 32768):
        m = min(32768, n - at)
        x = _rows(g, m, c, torch.float32 if fmt == "f32" else torch.bfloat16)
        if fmt != "fp8":
            a["rows"][at:at + m] = x
            continue
        codes, hi, sc = _quantise(x, d_hi)
        a["rows"][at:at + m] = codes.view(torch.uint8)
        a["hi"][at:at + m] = hi
        a["scales"][at:at + m, : sc.shape[1]] = sc


def _handle(st, c, d_hi, fmt):
    if own:
        from long_context_sparse_05_b200 import _lib as L
        a = st["cache"]
        st["kv"] = L.kv_cache(L.DTYPE[fmt], c, d_hi, a["rows"], a["hi"], a["scales"], st["bt"])
    return st


def _clean(case):
    return {k: v for k, v in case.items() if k != "name"}


def prepare(case, seed):
    case = _clean(case)
    g = _gen(seed)
    return {"norm_rope": _prep_norm, "write": _prep_write, "read": _prep_read,
            "attn": _prep_attn}[case["op"]](case, g, seed)


def _prep_norm(case, g, seed):
    N, H, d, dt = case["N"], case["H"], case["d"], _dt(case["dtype"])
    if case["strided"]:
        buf = _randn(g, (N, (H + 1) * d), dt)
        q, kv = buf[:, : H * d].view(N, H, d), buf[:, H * d:]
    else:
        q, kv = _randn(g, (N, H, d), dt), _randn(g, (N, d), dt)
    st = dict(case=case, q=q, kv=kv, pos=torch.randint(0, case["L"], (N,), generator=g, device="cuda",
                                                      dtype=torch.int32),
              qg=1 + 0.1 * _randn(g, (d,)) if case["gain"] else None,
              kg=1 + 0.1 * _randn(g, (d,)) if case["gain"] else None,
              q_out=torch.empty((N, H, d), dtype=dt, device="cuda"),
              kv_out=torch.empty((N, d), dtype=dt, device="cuda"))
    if own:
        from long_context_sparse_05_b200 import _lib as L
        st["p"] = L.NormRopeParams(H=H, d=d, d_rope=case["d_rope"], rope_theta=THETA, eps=EPS,
                                   apply_norm=1, dtype=L.DTYPE[case["dtype"]])
    return st


def _prep_write(case, g, seed):
    lens, c, d_hi = _ints(case["lens"]), case["c"], case["d_hi"]
    first = np.random.default_rng(int(seed)).integers(0, case["ctx"], len(lens))
    total, bt = _tables([case["ctx"] + n for n in lens], seed)
    st = dict(case=case, x=_rows(g, sum(lens), c, _dt(case["x"])), cu=_i32(_starts(lens)),
              first=_i32([int(f) for f in first]), bt=bt, rows=sum(lens), b=len(lens),
              cache=_alloc_cache(case["fmt"], total, c, d_hi))
    return _handle(st, c, d_hi, case["fmt"])


def _prep_read(case, g, seed):
    b, k, c, d_hi, E = case["b"], case["k"], case["c"], case["d_hi"], case["ctx"]
    total, bt = _tables([E] * b, seed)
    a = _alloc_cache(case["fmt"], total, c, d_hi)
    _fill_cache(a, g, case["fmt"], c, d_hi)
    idx = None
    n = min(k, E)
    if case["select"]:
        # distinct entries in ascending order, as a top-k gives them, padded with -1
        pick = torch.rand((b, E), generator=g, device="cuda").argsort(-1)[:, :n].sort(-1).values
        idx = torch.full((b, k), -1, dtype=torch.int32, device="cuda")
        idx[:, :n] = pick.int()
    low = max(1, n // 2) if case["ragged"] else n
    count = torch.randint(low, n + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    st = dict(case=case, cache=a, bt=bt, idx=idx, count=count, b=b, k=k,
              out=torch.empty((b, k, c), dtype=_dt(case["out"]), device="cuda"))
    return _handle(st, c, d_hi, case["fmt"])


def _prep_attn(case, g, seed):
    lens, ctx = _ints(case["lens"]), _ints(case["ctx"])
    H, d, m, k, n_w, fmt, d_hi = (case[x] for x in ("H", "d", "m", "k", "n_w", "fmt", "d_hi"))
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    b, N = len(lens), sum(lens)
    total, bt = _tables([(p + n) // m for p, n in zip(ctx, lens)], seed)
    a = _alloc_cache(fmt, total, d, d_hi)
    _fill_cache(a, g, fmt, d, d_hi)
    q = _randn(g, (N, H, d))
    q *= 1.5 * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS)
    cu, pos0 = _i32(_starts(lens)), _i32(ctx)
    st = dict(case=case, cache=a, bt=bt, b=b, N=N, L_max=max(p + n for p, n in zip(ctx, lens)),
              T_max=max(lens), q=q.to(dt), cu=cu, pos0=pos0, win=_rows(g, b * n_w, d, dt),
              new_win=_rows(g, N, d, dt), sink=_randn(g, (H,)), idx=None, count=None,
              out=torch.empty((N, H, d), dtype=dt, device="cuda"),
              lse=torch.empty((N, H), dtype=torch.float32, device="cuda"))
    if k:
        seq, t = _tokens(st)
        E = (t + 1) // m
        st["count"] = torch.minimum(E, torch.tensor(k, device="cuda")).int()
        # entry j of a token's selection: one of its visible entries in the j-th of k equal
        # parts, so that the entries are distinct and ascending
        n = st["count"].long()[:, None]
        j = torch.arange(k, device="cuda")[None]
        lo, hi = j * E[:, None] // n.clamp(min=1), (j + 1) * E[:, None] // n.clamp(min=1)
        u = torch.rand((N, k), generator=g, device="cuda")
        e = lo + (u * (hi - lo)).long().clamp(min=0).minimum((hi - lo - 1).clamp(min=0))
        st["idx"] = torch.where(j < n, e, -1).int()
    if own:
        from long_context_sparse_05_b200 import _lib as L
        p = L.AttnParams(H=H, d=d, n_w=n_w, scale=1.0 / math.sqrt(d), m=m, k=k,
                         dtype=L.DTYPE["f32" if fmt == "f32" else "bf16"],
                         d_rope_out=case["d_rope_out"], rope_theta=THETA)
        _handle(st, d, d_hi, fmt)
        st["p"] = p
        n = L.csa_chunk_attn_workspace_size(p, st["kv"], b, N, st["L_max"])
        st["ws"] = torch.empty((max(n, 256),), dtype=torch.uint8, device="cuda")
    return st


def _tokens(st):
    """(sequence, position) of every new token."""
    i = torch.arange(st["N"], device="cuda")
    cu = st["cu"].long()
    seq = torch.searchsorted(cu, i, right=True) - 1
    return seq, st["pos0"].long()[seq] + i - cu[seq]


# ----------------------------------------------------------------------------- one pass

def run(st):
    return {"norm_rope": _run_norm, "write": _run_write, "read": _run_read,
            "attn": _run_attn}[st["case"]["op"]](st)


def _run_norm(st):
    if own:
        from long_context_sparse_05_b200 import _lib as L
        L.csa_qk_norm_rope(st["p"], st["q"], st["qg"], st["kv"], st["kg"], st["pos"], st["case"]["N"],
                           st["q_out"], st["kv_out"])
        return st["q_out"], st["kv_out"]
    return (_norm_rope(st["q"], st["qg"], st["pos"][:, None], st["case"]["d_rope"]),
            _norm_rope(st["kv"], st["kg"], st["pos"], st["case"]["d_rope"]))


def _rotate(y, pos, r, sign):
    """The last r dims of y rotated in interleaved pairs by sign * pos * theta^(-2j/r)."""
    d = y.shape[-1]
    f = THETA ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    ang = sign * pos.double()[..., None] * f
    cs, sn = ang.cos().float(), ang.sin().float()
    a, b = y[..., d - r::2], y[..., d - r + 1::2]
    rot = torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)
    return torch.cat([y[..., : d - r], rot], -1)


def _norm_rope(x, gain, pos, r):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    if gain is not None:
        y = y * gain
    return _rotate(y, pos, r, 1.0).to(x.dtype)


def _run_write(st):
    case, a = st["case"], st["cache"]
    if own:
        from long_context_sparse_05_b200 import _lib as L
        L.csa_cache_write(st["kv"], L.DTYPE[case["x"]], st["x"], st["cu"], st["first"], st["b"],
                          st["rows"])
    else:
        cu = st["cu"].long()
        i = torch.arange(st["rows"], device="cuda")
        seq = torch.searchsorted(cu, i, right=True) - 1
        e = st["first"].long()[seq] + i - cu[seq]
        at = st["bt"].long()[seq, e // PAGE] * PAGE + e % PAGE
        if case["fmt"] == "fp8":
            c, d_hi = case["c"], case["d_hi"]
            y = st["x"][:, : c - d_hi].float().reshape(st["rows"], -1, GROUP)
            top = y.abs().amax(-1)
            mant, ex = torch.frexp(top)
            k = torch.where(mant <= 0.875, ex - 9, ex - 8)
            k = torch.where(top == 0, K_MIN, k).clamp(K_MIN, K_MAX)
            v = torch.ldexp(y, -k[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            a["rows"][at] = v.reshape(st["rows"], c - d_hi).view(torch.uint8)
            a["hi"][at] = st["x"][:, c - d_hi:]
            a["scales"][at, : k.shape[1]] = (k + 127).to(torch.uint8)
        else:
            a["rows"][at] = st["x"]
    if case["fmt"] != "fp8":
        return a["rows"]
    return a["rows"].view(torch.float8_e4m3fn), a["hi"], a["scales"]


def _plain_rows(a, fmt, at):
    """Rows `at` of a cache in 32 bits."""
    if fmt != "fp8":
        return a["rows"][at].float()
    y = a["rows"][at].view(torch.float8_e4m3fn).float()
    ns = y.shape[-1] // GROUP
    sc = torch.exp2(a["scales"][at][..., :ns].float() - 127.0)
    return torch.cat([y * sc.repeat_interleave(GROUP, -1), a["hi"][at].float()], -1)


def _run_read(st):
    case = st["case"]
    if own:
        from long_context_sparse_05_b200 import _lib as L
        L.csa_cache_read(st["kv"], st["idx"], st["count"], st["b"], st["k"], L.DTYPE[case["out"]],
                         st["out"])
        return st["out"]
    j = torch.arange(st["k"], device="cuda")[None].expand(st["b"], -1)
    e = st["idx"].long() if st["idx"] is not None else j
    ok = (j < st["count"][:, None]) & (e >= 0)
    e = torch.where(ok, e, 0)
    at = st["bt"].long().gather(1, e // PAGE) * PAGE + e % PAGE
    rows = _plain_rows(st["cache"], case["fmt"], at)
    return torch.where(ok[..., None], rows, 0.0).to(_dt(case["out"]))


def _run_attn(st):
    case = st["case"]
    if own:
        from long_context_sparse_05_b200 import _lib as L
        L.csa_chunk_attn(st["p"], st["kv"], st["q"], st["cu"], st["pos0"], st["idx"], st["count"],
                         st["win"], st["new_win"], st["sink"], st["b"], st["N"], st["L_max"],
                         st["out"], st["lse"], st["ws"])
        return st["out"], st["lse"]
    H, d, m, k, n_w = (case[x] for x in ("H", "d", "m", "k", "n_w"))
    N, b = st["N"], st["b"]
    seq, t = _tokens(st)
    q = st["q"].float() * (1.0 / math.sqrt(d))
    # the window of each token: rows of the ring before the chunk, rows of the chunk after
    u = t[:, None] - n_w + 1 + torch.arange(n_w, device="cuda")
    new = u >= st["pos0"].long()[seq][:, None]
    at = torch.where(new, b * n_w + (st["cu"].long()[seq] - st["pos0"].long()[seq])[:, None] + u,
                     seq[:, None] * n_w + u % n_w)
    wrow = torch.cat([st["win"], st["new_win"]])[torch.where(u >= 0, at, 0)].float()
    s_w = torch.bmm(q, wrow.transpose(1, 2)).masked_fill((u < 0)[:, None], -math.inf)
    if k:
        e = st["idx"].long()
        ok = (torch.arange(k, device="cuda")[None] < st["count"][:, None]) & (e >= 0)
        e = torch.where(ok, e, 0)
        rows = _plain_rows(st["cache"], case["fmt"],
                           st["bt"].long()[seq[:, None], e // PAGE] * PAGE + e % PAGE)
        s_e = torch.bmm(q, rows.transpose(1, 2)).masked_fill(~ok[:, None], -math.inf)
    else:
        # every entry of every sequence against the sequence's tokens, padded to the longest
        E = max(1, st["L_max"] // m)
        e = torch.arange(E, device="cuda")
        page = st["bt"].long()[:, (e // PAGE)]
        rows = _plain_rows(st["cache"], case["fmt"], page.clamp(min=0) * PAGE + e % PAGE)
        slot = seq * st["T_max"] + torch.arange(N, device="cuda") - st["cu"].long()[seq]
        qp = torch.zeros((b * st["T_max"], H, d), device="cuda")
        qp[slot] = q
        s_e = torch.bmm(qp.view(b, -1, d), rows.transpose(1, 2)).view(b * st["T_max"], H, E)[slot]
        s_e = s_e.masked_fill((e >= ((t + 1) // m)[:, None])[:, None], -math.inf)
    top = torch.maximum(torch.maximum(s_w.amax(-1), s_e.amax(-1)), st["sink"])
    p_w, p_e = (s_w - top[..., None]).exp(), (s_e - top[..., None]).exp()
    den = p_w.sum(-1) + p_e.sum(-1) + (st["sink"] - top).exp()
    o = torch.bmm(p_w, wrow)
    if k:
        o = o + torch.bmm(p_e, rows)
    else:
        pp = torch.zeros((b * st["T_max"], H, E), device="cuda")
        pp[slot] = p_e
        o = o + torch.bmm(pp.view(b, -1, E), rows).view(b * st["T_max"], H, d)[slot]
    o = o / den[..., None]
    if case["d_rope_out"]:
        o = _rotate(o, t[:, None], case["d_rope_out"], -1.0)
    return o.to(st["out"].dtype), top + den.log()


# ----------------------------------------------------------------------------- work

def _row_bytes(fmt, c, d_hi):
    return {"f32": 4 * c, "bf16": 2 * c, "fp8": c + d_hi + (c - d_hi) // GROUP}[fmt]


def work(case):
    if case["op"] == "norm_rope":
        n = case["N"] * (case["H"] + 1) * case["d"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * case["N"], "flops": 6 * n}
    if case["op"] == "write":
        rows = sum(_ints(case["lens"]))
        return {"bytes": rows * (case["c"] * (2 if case["x"] == "bf16" else 4) +
                                 _row_bytes(case["fmt"], case["c"], case["d_hi"])),
                "flops": 2 * rows * case["c"]}
    if case["op"] == "read":
        n = min(case["k"], case["ctx"])
        got = case["b"] * (3 * n // 4 if case["ragged"] else n)
        return {"bytes": got * _row_bytes(case["fmt"], case["c"], case["d_hi"]) +
                case["b"] * case["k"] * case["c"] * (2 if case["out"] == "bf16" else 4),
                "flops": got * case["c"]}
    H, d, m, k, n_w = (case[x] for x in ("H", "d", "m", "k", "n_w"))
    eb = 4 if case["fmt"] == "f32" else 2
    rb = _row_bytes(case["fmt"], d, case["d_hi"])
    nbytes = flops = 0
    for n, p in zip(_ints(case["lens"]), _ints(case["ctx"])):
        t = np.arange(p, p + n, dtype=np.int64)
        E = (t + 1) // m
        sel = np.minimum(E, k) if k else E
        flops += int((sel + np.minimum(t + 1, n_w)).sum()) * H * d * 4
        # each entry read once however many tokens attend to it
        nbytes += min(int(sel.sum()), int(E[-1])) * rb + (n + min(p, n_w)) * d * eb
        nbytes += 2 * n * H * d * eb + n * H * 4 + (4 * int(sel.sum()) if k else 0)
    return {"bytes": nbytes, "flops": flops}


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The operator's definition in 64 bits, token by token or sequence by sequence."""
    st = prepare(case, seed)
    case = st["case"]
    return {"norm_rope": _exact_norm, "write": _exact_write, "read": _exact_read,
            "attn": _exact_attn}[case["op"]](case, st)


def _turn(z, pos, r, sign):
    """Complex rotation of the last r dims of z at positions pos (one per row of z)."""
    j = torch.arange(r // 2, device="cuda", dtype=torch.float64)
    ang = sign * pos.double().unsqueeze(-1) * torch.exp(-2.0 * j / r * math.log(THETA))
    tail = torch.view_as_complex(z[..., -r:].reshape(*z.shape[:-1], r // 2, 2).contiguous())
    tail = tail * torch.polar(torch.ones_like(ang), ang)
    z = z.clone()
    z[..., -r:] = torch.view_as_real(tail).flatten(-2)
    return z


def _exact_norm(case, st):
    outs = []
    for x, gain in ((st["q"], st["qg"]), (st["kv"], st["kg"])):
        z = x.double()
        z = z / torch.sqrt((z * z).sum(-1, keepdim=True) / z.shape[-1] + EPS)
        z = z if gain is None else z * gain.double()
        pos = st["pos"] if z.dim() == 2 else st["pos"][:, None].expand(-1, z.shape[1])
        outs.append(_turn(z, pos, case["d_rope"], 1.0))
    return tuple(outs)


def _exact_write(case, st):
    a, c, d_hi = st["cache"], case["c"], case["d_hi"]
    cu, first, bt = st["cu"].tolist(), st["first"].tolist(), st["bt"].cpu().numpy()
    for s in range(st["b"]):
        e = first[s] + np.arange(cu[s + 1] - cu[s])
        at = torch.from_numpy(bt[s, e // PAGE].astype(np.int64) * PAGE + e % PAGE).cuda()
        x = st["x"][cu[s]:cu[s + 1]]
        if case["fmt"] != "fp8":
            a["rows"][at] = x
            continue
        codes, hi, sc = _quantise(x, d_hi)
        a["rows"][at] = codes.view(torch.uint8)
        a["hi"][at] = hi
        a["scales"][at, : sc.shape[1]] = sc
    if case["fmt"] != "fp8":
        return a["rows"].double()
    return a["rows"].view(torch.float8_e4m3fn).double(), a["hi"].double(), a["scales"]


def _values(a, fmt, at):
    if fmt != "fp8":
        return a["rows"][at].double()
    y = a["rows"][at].view(torch.float8_e4m3fn).double()
    n = y.shape[-1] // GROUP
    two = torch.full((), 2.0, dtype=torch.float64, device="cuda")
    sc = torch.pow(two, a["scales"][at][:, :n].double() - 127)
    y = (y.reshape(-1, n, GROUP) * sc[:, :, None]).reshape(-1, n * GROUP)
    return torch.cat([y, a["hi"][at].double()], 1)


def _places(bt, s, e):
    return torch.from_numpy(bt[s, e // PAGE].astype(np.int64) * PAGE + e % PAGE).cuda()


def _exact_read(case, st):
    bt, count = st["bt"].cpu().numpy(), st["count"].tolist()
    out = torch.zeros((st["b"], st["k"], case["c"]), dtype=torch.float64, device="cuda")
    for s in range(st["b"]):
        e = np.arange(count[s]) if st["idx"] is None else st["idx"][s, : count[s]].cpu().numpy()
        out[s, : count[s]] = _values(st["cache"], case["fmt"], _places(bt, s, e))
    return out


def _exact_attn(case, st):
    H, d, m, k, n_w = (case[x] for x in ("H", "d", "m", "k", "n_w"))
    bt, sink = st["bt"].cpu().numpy(), st["sink"].double()
    out = torch.empty((st["N"], H, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((st["N"], H), dtype=torch.float64, device="cuda")
    at0 = 0
    for s, (n, p0) in enumerate(zip(_ints(case["lens"]), _ints(case["ctx"]))):
        # the tokens before the chunk that a window can reach, then the chunk's own
        old = min(p0, n_w)
        tok = np.arange(p0 - old, p0)
        ring = st["win"][torch.from_numpy(s * n_w + tok % n_w).cuda()].double()
        line = torch.cat([ring, st["new_win"][at0:at0 + n].double()])
        E_s = (p0 + n) // m
        ents = _values(st["cache"], case["fmt"], _places(bt, s, np.arange(E_s)))
        step = 64 if k else 128
        for i in range(0, n, step):
            w = min(step, n - i)
            pos = torch.arange(p0 + i, p0 + i + w, device="cuda")
            q = st["q"][at0 + i:at0 + i + w].double()
            # window columns [lo, hi) of `line` that any of these tokens sees
            lo, hi = max(0, i + old - n_w + 1), i + w + old
            src = torch.arange(lo, hi, device="cuda") + p0 - old
            sw = torch.einsum("nhd,ud->nhu", q, line[lo:hi]) / math.sqrt(d)
            see = (src[None] <= pos[:, None]) & (src[None] > pos[:, None] - n_w)
            sw = torch.where(see[:, None], sw, -math.inf)
            if k:
                e = st["idx"][at0 + i:at0 + i + w].long()
                live = torch.arange(k, device="cuda")[None] < st["count"][at0 + i:at0 + i + w, None]
                kv = ents[e.clamp(min=0)] if E_s else torch.zeros((w, k, d), dtype=torch.float64, device="cuda")
                se = torch.einsum("nhd,nkd->nhk", q, kv) / math.sqrt(d)
            else:
                live = torch.arange(E_s, device="cuda")[None] < ((pos + 1) // m)[:, None]
                se = (q.reshape(-1, d) @ ents.T).view(w, H, E_s) / math.sqrt(d)
            se = torch.where(live[:, None], se, -math.inf)
            both = torch.cat([sw, se, sink[None, :, None].expand(w, H, 1)], -1)
            z = torch.logsumexp(both, -1)
            pw, pe = torch.exp(sw - z[..., None]), torch.exp(se - z[..., None])
            o = torch.einsum("nhu,ud->nhd", pw, line[lo:hi])
            o += torch.einsum("nhk,nkd->nhd", pe, kv) if k else (pe.reshape(w * H, E_s) @ ents).view(w, H, d)
            if case["d_rope_out"]:
                o = _turn(o, pos[:, None].expand(-1, H), case["d_rope_out"], -1.0)
            out[at0 + i:at0 + i + w], lse[at0 + i:at0 + i + w] = o, z
        at0 += n
    return out, lse
