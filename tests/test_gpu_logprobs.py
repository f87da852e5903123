"""token_logprobs against float64: tokens exactly, numbers within a derived bound.

Tolerance, with u = 2^-24: in a row with probabilities p, distances d = max - x and a reference up to 8
above or below the maximum's own, a term e^(x - r) is off by a part of (|x - r| (1 + 1 + 0.3) + 2) u (the
difference, its product with log2 e, that constant, the exponential).  T additions one after the
other (a thread's, the rest of the sum below 32) cost T u.  So S is off by a part of
s = (2.3 (D1 + 8) + 2 + T) u with D1 = sum p d, and rescaling adds 4 u and 2.3 * 8 u more;
log p = (x - M) - ln S by s + (|x - M| + 2 |ln S|) u and its own rounding;
H = ln S - U / S by s (1 + D1) + (2.3 (D2 + 8 D1) + (T + 8) D1 + 2 |ln S|) u with D2 = sum p d^2, and its
own rounding."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from gpu_helpers import DEV, host
from oracle import decode as dec
from round_helpers import bits, i32, stored, to_bf16

pytestmark = pytest.mark.gpu


def _check(x, tokens, rows, top, got):
    """x: the exact logits (float32) of all rows."""
    lp, h, ids, likely = (host(t) if t is not None else None for t in got)
    e_lp, e_h, e_ids, e_likely = dec.token_logprobs(x, tokens, rows, top)
    assert np.array_equal(ids, e_ids), np.argwhere(ids != e_ids)[:5]
    u, V = 2.0 ** -24, x.shape[1]
    for i, r in enumerate(rows):
        if np.isnan(e_h[i]):
            assert np.isnan(lp[i]).all() and np.isnan(likely[i]).all() and (h is None or np.isnan(h[i]))
            continue
        z = x[r].astype(np.float64)
        z = z - z.max()
        p = np.exp(z)
        S = p.sum()
        p, d = p / S, np.where(p > 0, -z, 0.0)
        D1, D2, lnS = (p * d).sum(), (p * d * d).sum(), np.log(S)
        T = V // 256 + 32
        s = (2.3 * (D1 + 16) + 6 + T) * u
        for g, e in ((lp[i], e_lp[i]), (likely[i], e_likely[i])):
            assert np.array_equal(np.isfinite(g), np.isfinite(e)) and np.array_equal(g[~np.isfinite(g)], e[~np.isfinite(e)], equal_nan=True)
            f = np.isfinite(e)
            far = np.abs(e[f]) + lnS
            assert np.all(np.abs(g[f] - e[f]) <= s + (far + 2 * lnS) * u + np.abs(e[f]) * u), (i, g[f] - e[f])
        if h is not None:
            tol = s * (1 + D1) + (2.3 * (D2 + 8 * D1) + (T + 8) * D1 + 2 * lnS) * u + e_h[i] * u
            assert abs(h[i] - e_h[i]) <= tol, (i, h[i], e_h[i], tol)


def _logits(n, V, dtype, seed, scale=2.5):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, scale, (n, V)).astype(np.float32)
    x[np.arange(n), rng.integers(0, V, n)] += 8
    if dtype == "bf16":
        raw = to_bf16(x)
        return raw, bits(raw, "bf16")
    return x, x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 63, 64, 255, 1000, 2047, 8200, 32001, 151936])
@pytest.mark.parametrize("top,given", [(0, 1), (1, 0), (5, 3), (20, 1), (64, 2)])
def test_against_float64(dtype, V, top, given):
    n = 5
    raw, x = _logits(n, V, dtype, V + top)
    logits = stored(raw, dtype, (V + 7) // 8 * 8 + 8)
    rng = np.random.default_rng(1)
    tokens = rng.integers(0, V, (n, given))
    if given:
        tokens[0, 0] = V
        tokens[1, 0] = -1
    got = wf.token_logprobs(logits, i32(tokens), top=top)
    assert got[0].shape == (n, given) and got[2].shape == (n, top)
    _check(x, tokens, np.arange(n), top, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 700, 2100])
def test_row_counts_and_selected_rows(dtype, n):
    V = 5003
    raw, x = _logits(1000, V, dtype, n)
    logits = stored(raw, dtype, 5008)
    rng = np.random.default_rng(2)
    rows = rng.integers(-2, 1003, n)
    tokens = rng.integers(0, V, (n, 1))
    got = wf.token_logprobs(logits, i32(tokens[:, 0]), rows=i32(rows), top=7)
    _check(x, tokens, rows, 7, got)
    none = wf.token_logprobs(logits, rows=i32(rows), top=7, entropy=False)
    assert none[0].shape == (n, 0) and none[1] is None and torch.equal(none[2], got[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks_and_odd_rows(dtype):
    V, n = 20011, 16
    rng = np.random.default_rng(3)
    x = rng.normal(0, 3, (n, V)).astype(np.float32)
    lowest = np.float32(-3.3895314e38) if dtype == "bf16" else np.finfo(np.float32).min
    x[0] = -np.inf                              # nothing is left
    x[1, rng.random(V) < 0.999] = -np.inf       # fewer than `top` are left
    x[1, 20:] = -np.inf
    x[2, :] = -np.inf
    x[2, 17] = 4.0                              # one token
    x[3, rng.random(V) < 0.9] = lowest          # masked by the lowest number
    x[4] = lowest                               # ... everywhere: all alike
    x[5] = 1.0                                  # all alike
    x[6, 9] = np.nan
    x[7, V - 1] = np.inf
    x[8, :9000] = -np.inf                       # whole chunks masked
    x[9] = np.sort(x[9])                        # every element is a candidate
    x[10] = -np.sort(-x[10])
    x[11] = np.round(x[11])                     # many equal ones
    x[12, :] = -0.0
    x[12, 3::7] = 0.0                           # zeros of both signs are equal
    x[13] = x[13] * 1e-3 + 900.0                # far from 0
    x[14] = x[14] * 100                         # sharp
    x[15, 5] = 3e38
    raw = to_bf16(x) if dtype == "bf16" else x
    x = bits(raw, "bf16") if dtype == "bf16" else x
    logits = stored(raw, dtype, 20016)
    tokens = np.stack([rng.integers(0, V, n), np.full(n, V - 1), np.full(n, 17)], 1)
    for top in (0, 1, 10, 64):
        _check(x, tokens, np.arange(n), top, wf.token_logprobs(logits, i32(tokens), top=top))
    # one row each, cut into more chunks
    for i in range(n):
        _check(x, tokens[i:i + 1], [i], 30, wf.token_logprobs(logits, i32(tokens[i:i + 1]), rows=i32([i]), top=30))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_odd_rows_in_one_piece(dtype):
    # So many rows that each is one workgroup's: long runs of equal logits, few logits, masks.
    V, n = 20011, 12
    rng = np.random.default_rng(4)
    x = rng.normal(0, 3, (n, V)).astype(np.float32)
    x[0] = 2.5
    x[1] = np.round(x[1] / 4)
    x[2, 40:] = -np.inf
    x[3, :-5] = -np.inf
    x[4] = np.sort(x[4])
    x[5] = -np.inf
    x[6, ::3] = -np.inf
    x[7] = 3e6 + np.round(x[7])                 # too far from 0 for the short way to 2^t
    x[8, 5000:9000] += 40                       # the likely ones side by side
    x[9, 0] = np.nan
    x[10, :10000] = -1e30
    x[11] = -4e6 - np.arange(V) / 4
    raw = to_bf16(x) if dtype == "bf16" else x
    x = bits(raw, "bf16") if dtype == "bf16" else x
    logits = stored(raw, dtype, 20016)
    rows = np.tile(np.arange(n), 180)
    tokens = rng.integers(0, V, (len(rows), 1))
    for top in (0, 3, 64):
        got = wf.token_logprobs(logits, i32(tokens), rows=i32(rows), top=top)
        _check(x, tokens[:n], np.arange(n), top, [t[:n] for t in got])
        for t in got[1:]:
            first = torch.nan_to_num(t[:n], nan=5.0)
            for a in range(n, len(rows), n):
                assert torch.equal(torch.nan_to_num(t[a:a + n], nan=5.0), first)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_rows_in_one_piece(dtype):
    # Rows of 4 million, one workgroup each: groups of many vectors.
    V = (1 << 22) + 5
    raw, x = _logits(2, V, dtype, 11)
    logits = stored(raw, dtype, (1 << 22) + 8)
    rows = np.arange(2100) % 2
    for top in (1, 20, 64):
        got = wf.token_logprobs(logits, i32(np.arange(2100) + V - 2100), rows=i32(rows), top=top)
        tokens = (np.arange(2100) + V - 2100)[:, None]
        _check(x, tokens[:2], [0, 1], top, [t[:2] for t in got])
        for t in got[1:]:
            assert torch.equal(t[2:], t[:2].repeat(1049, *[1] * (t.dim() - 1)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [20011, 151936])
@pytest.mark.parametrize("copies", [1, 260])
def test_the_entropy_of_a_dominant_token_keeps_its_digits(dtype, V, copies):
    # T = 1 + S: H = ln(1 + S) - ln 2 U / T is a sum of two positive numbers, each as exact as S and U:
    # every term e^(x - r) is off by a part of (2.3 (d + 8) + 3) u, d at most that of the likeliest of
    # the others' range that counts (40: what lies further holds less than 2^-24 of the rest), a sum of
    # V / 256 + 32 of them by as many u, the scaling by 2.3 (d + 8) u, the logarithms and H by 8 u.
    raw, x = _logits(9, V, "f32", 7, scale=1.0)
    x = np.array(x)
    where = [0, 3, V - 1, V - 2, V // 2, 511, 4096, V - 1, 77]
    gap = [8, 12, 16, 16, 20, 24, 28, 30, 22]
    for i, (at, d) in enumerate(zip(where, gap)):
        x[i] = np.random.default_rng(i).normal(0, 1, V)
        x[i, at] = x[i].max() + d
    raw = to_bf16(x) if dtype == "bf16" else x
    x = bits(raw, "bf16") if dtype == "bf16" else x
    logits = stored(raw, dtype, (V + 7) // 8 * 8)
    rows = np.tile(np.arange(9), copies)
    got = host(wf.token_logprobs(logits, rows=i32(rows), top=2)[1]).reshape(copies, 9).astype(np.float64)
    want = dec.token_logprobs(x, np.zeros((9, 0), int), np.arange(9), 0)[1]
    tol = (2 * 2.3 * (40 + 8) + 3 + V / 256 + 32 + 8) * 2.0 ** -24 * want
    assert np.all(np.abs(got - want) <= tol), np.abs(got / want - 1).max()


def test_three_dimensions_repeat_and_do_not_depend_on_the_other_rows():
    raw, x = _logits(6, 999, "f32", 5)
    logits = stored(raw, "f32", 1000).unflatten(0, (2, 3))
    tokens = np.arange(6)[:, None]
    first = wf.token_logprobs(logits, i32(tokens), top=3)
    _check(x, tokens, np.arange(6), 3, first)
    again = wf.token_logprobs(logits, i32(tokens), top=3)
    other = stored(raw, "f32", 1000).unflatten(0, (2, 3))  # (a clone would pack the rows: 999 is no whole vector)
    other[0] = 7.0
    changed = wf.token_logprobs(other, i32(tokens), top=3)
    for a, b, c in zip(first, again, changed):
        assert torch.equal(a, b) and torch.equal(a[3:], c[3:])


def test_past_32_bits():
    # The last rows lie past 2^31 elements.
    V, n = 151936, 14200
    logits = torch.zeros(n, V, dtype=torch.bfloat16, device=DEV)
    logits[-2:].normal_()
    logits[-1, 5] = 9.0
    rows = i32([n - 1, n - 2])
    got = wf.token_logprobs(logits, i32([[5], [V - 1]]), rows=rows, top=2)
    _check(host(logits[-2:].float()), np.array([[5], [V - 1]]), [1, 0], 2, got)


def test_nothing_to_do():
    logits = torch.zeros(0, 16, device=DEV)
    got = wf.token_logprobs(logits, torch.zeros(0, 2, dtype=torch.int32, device=DEV), top=3)
    assert got[0].shape == (0, 2) and got[2].shape == (0, 3) and got[1].numel() == 0
