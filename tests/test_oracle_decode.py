"""Pins of the oracle of a decoding step: closed forms, torch's own 8-bit type on the CPU, invariants."""

import numpy as np
import pytest
import torch

from oracle import decode as dec
from oracle import rounds as orc


def test_e4m3_is_torchs_on_every_number_and_on_ties():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(dec.round_e4m3(codes), codes, equal_nan=True)
    fine = np.sort(codes[np.isfinite(codes)]).astype(np.float64)
    mid = (fine[1:] + fine[:-1]) / 2
    rng = np.random.default_rng(0)
    x = np.concatenate([mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng.normal(0, 100, 5000).clip(-448, 448)])
    x = x.astype(np.float32)
    assert np.array_equal(dec.round_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy())
    assert np.isnan(dec.round_e4m3([np.inf, -np.inf, np.nan])).all()


def test_block_exponents():
    for e in (-100, -20, 0, 7, 119):
        assert dec.block_exponent([448 * 2.0 ** e, -1e-30]) == e
        if e < 119:
            assert dec.block_exponent([-np.nextafter(448 * 2.0 ** e, np.inf)]) == e + 1
    assert dec.block_exponent([0.0]) == -100 and dec.block_exponent([np.nan, np.inf, 1.0]) == -8
    assert dec.block_exponent([3.4e38]) == 119


def _cache(block, page=16, heads=2, dim=4, pages=6):
    shape = (1, pages, heads, page, dim)
    return dec.Cache8(np.zeros(shape, np.float32), np.zeros(shape, np.float32), np.array([[0, 2, 4], [1, 3, 5]]),
                      np.array([3, 3]), np.array([0, 0]), np.ones(pages, int),
                      np.full((1, pages, heads, page // block), 27, np.uint8),
                      np.full((1, pages, heads, page // block), 27, np.uint8))


@pytest.mark.parametrize("block", [1, 4, 16])
def test_append_then_read(block):
    o = _cache(block)
    rng = np.random.default_rng(1)
    o.context[:] = (0, 3)
    seqs = [orc.chain_seq(0, [0] * 9, 5), orc.chain_seq(10, [0] * 9, 5)]
    k, v = rng.normal(0, 1, (2, 20, 2, 4))
    dec.cache_append(o, seqs, k, v)
    rk, rv = dec.cache_read(o, 10, first=o.context, pending=10)
    # half a step of three bits behind the leading one, relative to the value or to 2^-6 of the
    # block's scale, which is at most twice the largest value / 224
    assert np.all(np.abs(rk.reshape(20, 2, 4) - k) <= 2.0 ** -4 * np.maximum(np.abs(k), 2.0 ** -6 * 5 / 224))
    assert np.all(dec.cache_read(o, 10, first=o.context)[0] == 0)
    # appended again at the end, the first rows keep their values within another shift's rounding
    o.context += 10
    dec.cache_append(o, seqs, k * 1000, v * 1000)
    again = dec.cache_read(o, 10, first=o.context - 10)[1]
    if block == 1:
        assert np.array_equal(again, rv)
    assert np.all(np.abs(again - rv) <= 2.0 ** -4 * np.maximum(np.abs(rv), 2.0 ** -6 * 5000 / 224))


def test_compaction_with_a_scale_for_every_position_moves_values():
    o, plain = _cache(1), _cache(1)
    rng = np.random.default_rng(2)
    o.context[:] = (5, 0)
    parent = [-1, 0, 0, 2, 2, 4, 1]
    q = [orc.tree_seq(0, parent, [0] * 7, [0], 5), orc.Seq(7, [], [])]
    k, v = rng.normal(0, 1, (2, 7, 2, 4))
    dec.cache_append(o, q, k, v)
    plain = o.values()
    after = np.zeros(2, int)
    dec.cache_compact(o, q, [4, 0], [5, 0], after)
    orc.cache_compact(plain, q, [4, 0], [5, 0], np.zeros(2, int))
    assert np.array_equal(o.values().k, plain.k) and np.array_equal(o.values().v, plain.v)
    assert after.tolist() == [9, 0]


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(3)
    seqs = [orc.chain_seq(0, [0] * 5, 5)]
    f = 100.0 ** (-np.arange(3) / 3)
    x = rng.normal(0, 1, (6, 1, 8))
    x[:] = x[0]
    for layout in ("half", "interleaved"):
        y = dec.rotate(x, seqs, f, layout, 1.0, [1000])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 6:], x[..., 6:])
        # products of rows the same distance apart are the same
        assert np.allclose((y[0] * y[2]).sum(), (y[3] * y[5]).sum())
    tree = [orc.tree_seq(0, [-1, 0, 0, 1, 2, 9], [0] * 6, [0], 5)]
    y = dec.rotate(x, tree, f, "half", 2.0, [7])
    assert np.allclose(y[1], y[2]) and np.allclose(y[3], y[4]) and np.allclose(y[5], y[0])


def test_log_probabilities_in_closed_form():
    x = np.array([[0.0, np.log(3.0), -np.inf, 0.0], [2.0, 2.0, 2.0, 2.0], [-np.inf] * 4, [np.nan, 0, 0, 0], [0, np.inf, 0, 0]])
    lp, h, ids, top = dec.token_logprobs(x, np.array([[1, 2], [0, 9]] + [[0, 0]] * 4), [0, 1, 2, 3, 4, 5], 3)
    assert np.allclose(lp[0], [np.log(0.6), -np.inf]) and np.isclose(lp[1, 0], -np.log(4)) and np.isnan(lp[1, 1])
    assert np.isclose(h[0], -(0.6 * np.log(0.6) + 0.4 * np.log(0.2))) and np.isclose(h[1], np.log(4))
    assert ids[0].tolist() == [1, 0, 3] and ids[1].tolist() == [0, 1, 2]
    assert np.isnan(h[2:]).all() and np.isnan(lp[2:]).all() and (ids[2:] == -1).all() and np.isnan(top[2:]).all()
    _, _, ids, top = dec.token_logprobs(x[:1], np.zeros((1, 0), int), [0], 4)
    assert ids[0].tolist() == [1, 0, 3, -1] and top[0, 3] == -np.inf
