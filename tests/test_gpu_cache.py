"""The paged cache's calls against the oracle, exactly: moved bits and whole numbers."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from gpu_helpers import DEV, dev, host
from oracle import rounds as orc
from round_helpers import Round, bits, device_cache, i32, make_cache, same_cache, to_bf16

pytestmark = pytest.mark.gpu


def _rows_of(total, heads, dim, dtype, seed):
    """New keys and values as slices of one wider projection, and their float32 values."""
    x = np.random.default_rng(seed).normal(0, 1, (total, 3, heads, dim)).astype(np.float32)
    if dtype == "bf16":
        t = dev(to_bf16(x))
        x = bits(to_bf16(x), "bf16")
    else:
        t = dev(x)
    return t[:, 1], t[:, 2], x[:, 1], x[:, 2]


@pytest.mark.parametrize("kind,K,N", [("chain", 0, 0), ("chain", 16, 0), ("tree", 0, 21), ("routed", 5, 9)])
@pytest.mark.parametrize("dtype,heads,dim,page", [("bf16", 2, 128, 16), ("f32", 3, 64, 32), ("bf16", 1, 64, 1024)])
def test_append(kind, K, N, dtype, heads, dim, page):
    B = 4
    r = Round(kind, B, K, N, 100, seed=7)
    context = [0, 1, page - 1, 2 * page + 5]
    o, cache = make_cache(2, heads, page, dim, context, 40, 8, dtype=dtype, empty=2)
    o.table[2, 0] = -1                          # a hole
    o.context[3] = -4
    cache = device_cache(o, dtype)
    k, v, ok, ov = _rows_of(r.total, heads, dim, dtype, 9)
    seq = np.array([2, 0, 3, 1])
    seq[3] = 99 if kind == "tree" else 1
    wf.cache_append(cache, r.rows, k, v, layer=1, seqs=i32(seq))
    orc.cache_append(o, r.seqs, ok, ov, layer=1, seq=seq)
    same_cache(o, cache)


@pytest.mark.parametrize("kind,K,N", [("chain", 8, 0), ("tree", 0, 1), ("tree", 0, 61), ("routed", 16, 33),
                                      ("tree", 0, 300)])
@pytest.mark.parametrize("dtype,heads,dim,page", [("bf16", 8, 128, 16), ("f32", 2, 64, 16), ("f32", 3, 128, 64)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(kind, K, N, dtype, heads, dim, page, in_place):
    B = 6
    r = Round(kind, B, K, N, 50, seed=N, bad=N == 33)
    context = [0, 3, 15, 16, 40, 7]
    o, _ = make_cache(3, heads, page, dim, context, 301, 3, dtype=dtype, empty=1)
    rng = np.random.default_rng(1)
    al, best = np.zeros(B, int), np.zeros(B, int)
    for b, q in enumerate(r.seqs):
        u = q.n - 1 - int(rng.integers(0, 2)) if q.n > 2 else 0
        best[b], al[b] = u, len(q.path(u)) if q.n else 0
    al[1] += 1                                  # no path of that length
    best[2] = N + 4
    o.context[4] = -1
    seq = np.array([1, 0, 2, 5, 4, 3])
    if kind == "tree":
        seq[5] = -1
    cache = device_cache(o, dtype)
    after = o.context if in_place else np.full(7, -3, np.int32)
    out = None if in_place else i32(after)
    wf.cache_compact(cache, r.rows, i32(al), None if kind == "chain" else i32(best), seqs=i32(seq),
                     next_context=out)
    orc.cache_compact(o, r.seqs, al, best, after, seq)
    same_cache(o, cache)
    if out is not None:
        assert np.array_equal(host(out), after)


def test_compact_moves_whole_long_paths():
    # A path of every node (nothing moves), and one of every other node, 511 rows far.
    N = 1023
    parent = np.stack([np.arange(-1, N - 1), np.arange(-2, N - 2)])
    parent[1, 1] = 0
    r = Round("tree", 2, 0, N, 50, seed=1, parent=parent)
    o, cache = make_cache(1, 1, 16, 64, [5, 9], N, 2, dtype="f32")
    best = np.array([N - 1, N - 1])
    al = np.array([N, 512])
    wf.cache_compact(cache, r.rows, i32(al), i32(best))
    orc.cache_compact(o, r.seqs, al, best, o.context)
    same_cache(o, cache)


@pytest.mark.parametrize("dtype,heads,dim,page", [("bf16", 2, 64, 16), ("f32", 1, 128, 64)])
def test_fork_reserve_free(dtype, heads, dim, page):
    context = [0, 1, page, page + 1, 3 * page - 1]
    o, cache = make_cache(2, heads, page, dim, context, 0, 4, dtype=dtype, spare=4, empty=9)
    o.held[13] = 1                               # holds a page already: no dst
    o.table[13, 0] = np.flatnonzero(o.refs == 0)[0]
    o.refs[o.table[13, 0]] = 1
    cache = device_cache(o, dtype)
    # one source twice, a dst twice, dst that is a source, indices outside, too few pages
    src = np.array([1, 2, 3, 3, 4, 0, 1, 77, 2, 4])
    dst = np.array([5, 6, 7, 7, 8, 9, 2, 10, -1, 13])
    e = orc.cache_fork(o, src, dst)
    assert e.tolist() == [1, 1, 1, 0, 1, 1, 0, 0, 0, 0]
    status = wf.cache_fork(cache, i32(src), i32(dst))
    assert np.array_equal(host(status), e)
    same_cache(o, cache)
    # no page is free now: a fork that needs one is refused, one that needs none is not
    src, dst = np.array([3, 2, 4]), np.array([10, 11, 12])
    e = orc.cache_fork(o, src, dst)
    assert e.tolist() == [0, 1, 0]
    assert np.array_equal(host(wf.cache_fork(cache, i32(src), i32(dst))), e)
    same_cache(o, cache)
    # free: twice the same, one that holds nothing, indices outside; shared pages stay
    gone = np.array([7, 7, 3, 10, -3, 99, 13])
    orc.cache_free(o, gone)
    wf.cache_free(cache, i32(gone))
    same_cache(o, cache)
    # reserve: nothing to do, some pages, one named twice, past max_pages, too many, then none left
    seq = np.array([0, 5, 5, 2, 6, 9, 50])
    most = o.table.shape[1] * page
    count = np.array([0, page + 3, 1, most, 2 * page, 1, 1])
    e = orc.cache_reserve(o, seq, count)
    status = wf.cache_reserve(cache, i32(count), seqs=i32(seq))
    assert np.array_equal(host(status), e)
    same_cache(o, cache)
    seq = np.array([0, 6, 1])
    count = np.array([most, most - page, 0])
    e = orc.cache_reserve(o, seq, count)
    assert np.array_equal(host(wf.cache_reserve(cache, i32(count), seqs=i32(seq))), e)
    same_cache(o, cache)


def test_reserve_hands_out_the_lowest_pages_of_a_large_pool():
    P, S = 5000, 1500
    o = orc.Cache(np.zeros((1, P, 1, 16, 64), np.float32), np.zeros((1, P, 1, 16, 64), np.float32),
                  np.full((S, 40), -1, np.int32), np.zeros(S, np.int32), np.zeros(S, np.int32),
                  (np.random.default_rng(0).random(P) < 0.3).astype(np.int32))
    cache = device_cache(o, "f32")
    rng = np.random.default_rng(1)
    seq = rng.permutation(S)[:1300]
    count = rng.integers(0, 90, 1300)
    e = orc.cache_reserve(o, seq, count)
    assert 0 < e.sum() < 1300
    assert np.array_equal(host(wf.cache_reserve(cache, i32(count), seqs=i32(seq))), e)
    same_cache(o, cache)


@pytest.mark.parametrize("free", [0, 1, 3])
@pytest.mark.parametrize("entries", [6, 40, 1100])
def test_demands_far_past_the_pool(free, entries):
    # More pages are wanted than the pool has in all: every entry behind its end that needs
    # one is refused, one that needs none (an empty context) is not.
    P, S = free + 1, entries + 3
    o = orc.Cache(np.zeros((1, P, 1, 16, 64), np.float32), np.zeros((1, P, 1, 16, 64), np.float32),
                  np.full((S, 8), -1, np.int32), np.zeros(S, np.int32), np.zeros(S, np.int32),
                  np.zeros(P, np.int32))
    o.table[0, 0], o.held[0], o.context[0], o.refs[P // 2] = P // 2, 1, 5, 1
    o.k[:] = np.random.default_rng(3).normal(0, 1, o.k.shape)
    cache = device_cache(o, "f32")
    src, dst = np.zeros(entries, int), np.arange(2, entries + 2)
    src[1::2] = 1                                # holds nothing
    e = orc.cache_fork(o, src, dst)
    assert e[::2].sum() == min(free, (entries + 1) // 2) and e[1::2].all()
    assert np.array_equal(host(wf.cache_fork(cache, i32(src), i32(dst))), e)
    same_cache(o, cache)
    gone = np.arange(2, entries + 2)
    orc.cache_free(o, gone)
    wf.cache_free(cache, i32(gone))
    count = np.where(np.arange(entries) % 3 == 2, 0, 8 * 16)
    e = orc.cache_reserve(o, dst, count)
    assert e.sum() == (count == 0).sum()
    assert np.array_equal(host(wf.cache_reserve(cache, i32(count), seqs=i32(dst))), e)
    same_cache(o, cache)


def test_random_lives_of_sequences():
    # Forks, rows, acceptances and frees in turn; the pool balances at the end.
    rng = np.random.default_rng(17)
    heads, dim, page = 2, 64, 16
    o, cache = make_cache(1, heads, page, dim, [20, 0], 0, 5, dtype="f32", spare=30, empty=6)
    live = {0, 1}
    for turn in range(12):
        print("turn", turn, flush=True)
        seq = np.array(sorted(live))
        N = int(rng.integers(1, 12))
        r = Round("tree", len(seq), 0, N, 40, seed=turn)
        e = orc.cache_reserve(o, seq, np.full(len(seq), N))
        assert np.array_equal(host(wf.cache_reserve(cache, i32(np.full(len(seq), N)), seqs=i32(seq))), e)
        k, v, ok, ov = _rows_of(r.total, heads, dim, "f32", turn)
        wf.cache_append(cache, r.rows, k, v, seqs=i32(seq))
        orc.cache_append(o, r.seqs, ok, ov, seq=seq)
        best = rng.integers(0, N, len(seq))
        al = np.array([len(q.path(int(u))) for q, u in zip(r.seqs, best)])
        wf.cache_compact(cache, r.rows, i32(al), i32(best), seqs=i32(seq))
        orc.cache_compact(o, r.seqs, al, best, o.context, seq)
        spare = [s for s in range(8) if s not in live][:2]
        if turn % 2 == 0 and spare:
            src, dst = rng.choice(seq, len(spare)), np.array(spare)
            e = orc.cache_fork(o, src, dst)
            assert np.array_equal(host(wf.cache_fork(cache, i32(src), i32(dst))), e)
            live |= {int(d) for d, s in zip(dst, e) if s}
        elif len(live) > 2:
            gone = rng.choice(sorted(live), 2, replace=False)
            wf.cache_free(cache, i32(gone))
            orc.cache_free(o, gone)
            live -= {int(s) for s in gone}
        same_cache(o, cache)
        held = np.bincount(o.table[o.table >= 0], minlength=len(o.refs))
        assert np.array_equal(held, o.refs), "references and table entries agree"
    wf.cache_free(cache, i32(np.arange(8)))
    assert int(cache.refs.abs().sum()) == 0 and int(cache.held.sum()) == 0


def test_a_cache_past_32_bits():
    # The last page of the last layer lies past 2^31 elements.
    P, layers, dim, page = 20000, 2, 128, 64
    cache = wf.PageCache.empty(layers, P, 8, page, dim, 3, 4, device=DEV)
    cache.table[0, 0] = P - 1
    cache.refs[P - 1] = 1
    cache.held[0] = 1
    cache.context[0] = 50
    rows = wf.tree_rows(i32(np.array([[-1, 0, 0, 2]])))
    assert cache.k[1, P - 1].data_ptr() - cache.k.data_ptr() > 2**32
    x = torch.randn(4, 8, dim, device=DEV).to(torch.bfloat16)
    seq = torch.zeros(1, dtype=torch.int32, device=DEV)
    wf.cache_append(cache, rows, x, -x, layer=1, seqs=seq)
    assert torch.equal(cache.k[1, P - 1, :, 50:54].transpose(0, 1), x)
    wf.cache_compact(cache, rows, i32([3]), i32([3]), seqs=seq)
    assert torch.equal(cache.v[1, P - 1, :, 52], -x[3]) and int(cache.context[0]) == 53
    wf.cache_fork(cache, seq, seq + 1)
    assert cache.table[1, 0].item() == 0
    assert torch.equal(cache.k[1, 0, :, :53], cache.k[1, P - 1, :, :53])
    assert int(cache.k[1, 0, :, 53:].abs().sum()) == 0
