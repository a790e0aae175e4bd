"""Pins of the oracle of the chunk calls: the quantised row against its definition and torch's
E4M3 casts, the norm and rotation by identities, the chunk's rows by closed forms; each pin
rejects a planted mistake of the oracle."""

import numpy as np
import pytest
import torch

from oracle import chunk, codecs, csa


def test_scale_exponent_is_the_smallest_that_holds():
    rng = np.random.default_rng(0)
    vals = list(np.exp(rng.uniform(-60, 60, 200))) + [448.0 * 2.0 ** k for k in range(-20, 20)]
    vals += [np.nextafter(448.0 * 2.0 ** k, np.inf) for k in range(-20, 20)]
    for a in vals:
        k = chunk.scale_exponent(a)
        assert a <= 448.0 * 2.0 ** k and a > 448.0 * 2.0 ** (k - 1), (a, k)
    assert chunk.scale_exponent(0.0) == chunk.K_MIN
    assert chunk.scale_exponent(np.inf) == chunk.K_MAX
    assert chunk.scale_exponent(1e-45) == chunk.K_MIN
    assert chunk.scale_exponent(3.3e38) == chunk.K_MAX


def test_quantised_row_codes_match_torch_and_round_trip():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal(512)).to(torch.bfloat16)
    codes, hi, exps = chunk.quant_row(x.double().numpy(), 64)
    scaled = x[:448].double().numpy().reshape(7, 64) * 2.0 ** -(exps.astype(np.float64) - 127)[:, None]
    ref = torch.from_numpy(scaled).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(-1)
    assert np.array_equal(codes, ref)
    back = chunk.dequant_row(codes, hi, exps)
    assert np.array_equal(back[448:], x[448:].double().numpy())
    # one rounding of a 4-bit significand: half a step relative, or of the group's smallest step
    err = np.abs(back[:448] - x[:448].double().numpy()).reshape(7, 64)
    step = 2.0 ** (exps.astype(np.float64) - 127 - 10)[:, None]
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x[:448].double().numpy().reshape(7, 64)), step))
    # the values it stands for are bf16 values
    assert np.array_equal(codecs.round_to_bf16(back), back)


def test_quantised_row_specials():
    x = np.zeros(128)
    x[3], x[5] = np.nan, 2.0
    codes, hi, exps = chunk.quant_row(x, 0)
    assert codes[3] == 0x7F and exps[1] == chunk.K_MIN + 127
    back = chunk.dequant_row(codes, hi, exps)
    assert np.isnan(back[3]) and back[5] == 2.0 and np.all(back[64:] == 0)
    x[5] = np.inf
    codes, hi, exps = chunk.quant_row(x, 0)
    assert chunk.dequant_row(codes, hi, exps)[5] == 448.0 * 2.0 ** chunk.K_MAX


def test_norm_rope_identities():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 64))
    gain = rng.uniform(0.5, 2, 64)
    y = chunk.norm_rope(x, gain, np.zeros(5), 16, 1e4, 0.0)
    assert np.allclose(np.mean((y / gain) ** 2, axis=1), 1.0, atol=1e-12)
    # a rotation keeps each pair's length, and the inverse undoes it
    z = chunk.norm_rope(x, gain, np.arange(5) * 1000.0, 16, 1e4, 0.0)
    assert np.allclose(np.sum(z ** 2, 1), np.sum(y ** 2, 1), atol=1e-10)
    for i in range(5):
        assert np.allclose(csa.inverse_rope(z[i:i + 1], 1000.0 * i, 16, 1e4), y[i:i + 1], atol=1e-9)
    assert not np.allclose(z[1], y[1])


@pytest.mark.parametrize("n_w", [0, 3, 8])
def test_chunk_rows_window_and_entries(n_w):
    """Rows carry their own name: the list of a token is known in closed form."""
    m, pos0, n, cu = 4, 10, 6, 2
    win = [[("ring", s, j) for j in range(max(n_w, 1))] for s in range(2)]
    for u in range(pos0):                    # the ring as one token at a time leaves it
        if n_w:
            win[1][u % n_w] = ("old", u)
    new = [("new", r) for r in range(cu + n)]
    for i in range(n):
        t, rows = chunk.chunk_rows(1, i, lambda s, e: ("entry", s, e), None, pos0, cu, m, 256, win,
                                   new, n_w)
        assert t == pos0 + i
        want = [("entry", 1, e) for e in range((t + 1) // m)]
        for u in range(max(0, t - n_w + 1), t + 1):
            want.append(("new", cu + u - pos0) if u >= pos0 else ("old", u))
        assert rows == want
    # a selection is taken as given, entries outside the table are dropped
    _, rows = chunk.chunk_rows(0, 0, lambda s, e: None if e == 7 else ("entry", s, e),
                               np.array([0, 7, 300, -1, 5]), pos0, cu, m, 256, win, new, 0)
    assert rows == [("entry", 0, 0), ("entry", 0, 5)]


def test_attend_matches_the_oracle_and_the_edge_cases():
    rng = np.random.default_rng(3)
    q, rows, sink = rng.standard_normal((3, 8)), rng.standard_normal((5, 8)), rng.standard_normal(3)
    o, l, A = chunk.attend(q, list(rows), sink, 0.3)
    o2, l2 = csa.attend(q, rows, sink, 0.3)
    assert np.allclose(o, o2, atol=1e-14) and np.allclose(l, l2, atol=1e-14)
    assert np.all(A >= np.abs(o) - 1e-15)
    o, l, _ = chunk.attend(q, [], sink, 0.3)
    assert np.all(o == 0) and np.array_equal(l, sink)
    o, l, _ = chunk.attend(q, list(rows), np.full(3, -np.inf), 0.3)
    w = np.exp(0.3 * q @ rows.T)
    assert np.allclose(o, (w @ rows) / w.sum(1)[:, None], atol=1e-12)
