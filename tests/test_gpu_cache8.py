"""The 8-bit cache's calls against the oracle, exactly: every number and every scale."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from decode_helpers import TORCH, device_cache8, full, make_cache8, same_cache8, to_e4m3, vectors
from gpu_helpers import DEV, dev, host
from oracle import decode as dec
from oracle import rounds as orc
from round_helpers import Round, i32, to_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,K,N", [("chain", 0, 0), ("chain", 16, 0), ("tree", 0, 21), ("routed", 5, 40)])
@pytest.mark.parametrize("dtype,heads,dim,page,block", [
    ("bf16", 2, 128, 16, 1), ("f32", 3, 64, 32, 1), ("bf16", 2, 128, 16, 16), ("f32", 1, 64, 32, 8),
    ("bf16", 5, 64, 64, 2), ("f32", 9, 128, 64, 32), ("bf16", 1, 64, 1024, 1024)])
def test_append(kind, K, N, dtype, heads, dim, page, block):
    B = 5
    r = Round(kind, B, K, N, 100, seed=7, bad=kind == "routed")
    context = [0, 1, page - 1, 2 * page + 5, 2 * page - 3]
    o, _ = make_cache8(2, heads, page, dim, block, context, 40, 8, empty=2)
    o.table[2, 0] = -1                          # a hole
    o.table[4, 1] = o.k.shape[1] + 4            # a page that is none
    o.context[3] = -4
    cache = device_cache8(o)
    # sizes far apart, so that committed values are shifted in both directions
    (k, v), (kx, vx) = vectors(r.total, heads, dim, dtype, 9, parts=2, scale=np.exp(
        3 * np.random.default_rng(3).normal(0, 1, (r.total, 1, 1))))
    seq = np.array([2, 0, 3, 1, 4])
    if kind == "tree":
        seq[4] = 99
    wf.cache_append(cache, r.rows, k, v, layer=1, seqs=i32(seq))
    dec.cache_append(o, r.seqs, kx, vx, layer=1, seq=seq)
    same_cache8(o, cache)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f32", 64), ("f32", 128), ("bf16", 64)])
@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64, 128])
def test_append_blocks_of_every_length(dtype, dim, block):
    # Starts and ends at every place of a block, spans of several blocks, one row and many.
    heads, page = 3, 128
    context = [0, 1, 2, 3, 5, 7, 8, 9, 12, 15, 16, 23, 31, 33, 63, 64, 100, 127, 128, 250]
    for K in (0, 5, 40, 130):
        r = Round("chain", len(context), K, 0, 100, seed=K)
        o, cache = make_cache8(1, heads, page, dim, block, context, K + 1, block + K)
        (k, v), (kx, vx) = vectors(r.total, heads, dim, dtype, 9, parts=2, scale=np.exp(
            2 * np.random.default_rng(3).normal(0, 1, (r.total, 1, 1))))
        wf.cache_append(cache, r.rows, k, v)
        dec.cache_append(o, r.seqs, kx, vx)
        same_cache8(o, cache)


@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_number_and_odd_values(dtype, block):
    # Ties between e4m3 numbers, the borders of the scales, zeros, subnormal numbers, the largest
    # ones, infinities and NaN.
    dim = 64
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    fine = np.sort(codes[np.isfinite(codes)])
    ties = (fine[1:] + fine[:-1]) / 2
    top = 3.4e38 if dtype == "f32" else 3.38e38
    rows = [np.resize(np.concatenate([ties, fine])[i:], dim) for i in range(0, 448, 32)]
    rows = [np.where(np.arange(dim) == 0, 448, x) * 2.0 ** e for x, e in zip(rows, [0, 0, 1, -3, 9, -60, 60] * 2)]
    rows += [np.zeros(dim), np.full(dim, 1e-40), np.resize([top, -top, 1.0, 0.0], dim),
             np.resize([np.inf, 1.0, np.nan, -np.inf, -2.5], dim), np.full(dim, np.nan),
             np.resize([448.0, 448.5, 3.0], dim), np.resize([2.0 ** -101, 2.0 ** -112, 2.0 ** -111, -2.0 ** -100], dim)]
    n = len(rows)
    x = np.stack(rows).astype(np.float32)[:, None]
    if dtype == "bf16":
        t = dev(to_bf16(x))
        x = t.float().cpu().numpy()
    else:
        t = dev(x)
    r = Round("chain", 1, n - 1, 0, 50, seed=1)
    o, cache = make_cache8(1, 1, 32, dim, block, [3], n, 2)
    wf.cache_append(cache, r.rows, t, -t)
    dec.cache_append(o, r.seqs, x, -x)
    same_cache8(o, cache)
    for out in ("f32", "bf16"):
        k, v = wf.cache_read(cache, n + 3, pending=n, dtype=TORCH[out])
        want = dec.cache_read(o, n + 3, pending=n)
        assert np.array_equal(host(k.float()), want[0], equal_nan=True)
        assert np.array_equal(host(v.float()), want[1], equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,dim,page,block", [(2, 128, 16, 16), (3, 64, 32, 1), (1, 64, 16, 4), (8, 128, 64, 32)])
def test_read(dtype, heads, dim, page, block):
    context = [0, 1, page, 3 * page + 5, 40, 17]
    o, _ = make_cache8(2, heads, page, dim, block, context, 9, 8, empty=2)
    o.table[3, 1] = -1
    o.context[4] = -4
    cache = device_cache8(o)
    for layer, seq, first, count, pending in ((0, None, None, 3 * page + 20, 0), (1, [3, 3, 99, -1, 4, 1], [7, -9, 0, 0, 0, 1], 33, 5),
                                              (1, [2], [1 << 30], 5, 3), (0, [5, 2], None, 1, 0), (0, None, None, 0, 0)):
        n = len(seq) if seq is not None else 8
        shape = (n, count, heads, dim)
        ko, vo = full(shape, 9.0, dtype), full(shape, 9.0, dtype)
        got = wf.cache_read(cache, count, seqs=None if seq is None else i32(seq), first=None if first is None else i32(first),
                            pending=pending, layer=layer, k_out=ko, v_out=vo)
        want = dec.cache_read(o, count, seq, first, pending, layer)
        assert got[0] is ko and got[1] is vo
        for g, w in zip(got, want):
            assert np.array_equal(host(g.float()), w)


@pytest.mark.parametrize("kind,K,N", [("chain", 8, 0), ("tree", 0, 1), ("tree", 0, 61), ("routed", 16, 33), ("tree", 0, 300)])
@pytest.mark.parametrize("heads,dim,page,block", [(8, 128, 16, 1), (2, 64, 16, 16), (3, 128, 64, 8), (1, 64, 128, 128)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(kind, K, N, heads, dim, page, block, in_place):
    B = 6
    r = Round(kind, B, K, N, 50, seed=N, bad=N == 33)
    context = [0, 3, 15, 16, 40, 7]
    o, _ = make_cache8(2, heads, page, dim, block, context, 301, 3, empty=1)
    rng = np.random.default_rng(1)
    al, best = np.zeros(B, int), np.zeros(B, int)
    for b, q in enumerate(r.seqs):
        u = q.n - 1 - int(rng.integers(0, 2)) if q.n > 2 else 0
        best[b], al[b] = u, len(q.path(u)) if q.n else 0
    al[1] += 1                                  # no path of that length
    best[2] = N + 4
    o.context[4] = -1
    o.table[0, 1] = -1 if N == 300 else o.table[0, 1]
    seq = np.array([1, 0, 2, 5, 4, 3])
    if kind == "tree":
        seq[5] = -1
    cache = device_cache8(o)
    after = o.context if in_place else np.full(7, -3, np.int32)
    out = None if in_place else i32(after)
    wf.cache_compact(cache, r.rows, i32(al), None if kind == "chain" else i32(best), seqs=i32(seq), next_context=out)
    dec.cache_compact(o, r.seqs, al, best, after, seq)
    same_cache8(o, cache)
    if out is not None:
        assert np.array_equal(host(out), after)


@pytest.mark.parametrize("block", [1, 16])
def test_compact_moves_whole_long_paths(block):
    N = 1023
    parent = np.stack([np.arange(-1, N - 1), np.arange(-2, N - 2)])
    parent[1, 1] = 0
    r = Round("tree", 2, 0, N, 50, seed=1, parent=parent)
    o, cache = make_cache8(1, 1, 16, 64, block, [5, 9], N, 2)
    best, al = np.array([N - 1, N - 1]), np.array([N, 512])
    wf.cache_compact(cache, r.rows, i32(al), i32(best))
    dec.cache_compact(o, r.seqs, al, best, o.context)
    same_cache8(o, cache)


@pytest.mark.parametrize("heads,dim,page,block", [(2, 64, 16, 1), (1, 128, 64, 16), (3, 64, 32, 32)])
def test_fork_reserve_free(heads, dim, page, block):
    context = [0, 1, page, page + 1, 3 * page - 1]
    o, cache = make_cache8(2, heads, page, dim, block, context, 0, 4, spare=4, empty=9)
    src, dst = np.array([1, 2, 3, 3, 4, 0, 1, 77, 2]), np.array([5, 6, 7, 7, 8, 9, 2, 10, -1])
    e = dec.cache_fork(o, src, dst)
    assert e.tolist() == [1, 1, 1, 0, 1, 1, 0, 0, 0]
    assert np.array_equal(host(wf.cache_fork(cache, i32(src), i32(dst))), e)
    same_cache8(o, cache)
    gone = np.array([7, 7, 3, 10, -3, 99])
    orc.cache_free(o, gone)
    wf.cache_free(cache, i32(gone))
    same_cache8(o, cache)
    seq, count = np.array([0, 5, 5, 2, 6, 9, 50]), np.array([0, page + 3, 1, 9999, 2 * page, 1, 1])
    e = orc.cache_reserve(o, seq, count)
    assert np.array_equal(host(wf.cache_reserve(cache, i32(count), seqs=i32(seq))), e)
    same_cache8(o, cache)


@pytest.mark.parametrize("block", [1, 8])
def test_random_lives_of_sequences(block):
    rng = np.random.default_rng(17)
    heads, dim, page = 2, 64, 16
    o, cache = make_cache8(1, heads, page, dim, block, [20, 0], 0, 5, spare=30, empty=6)
    live = {0, 1}
    for turn in range(10):
        print("turn", turn, flush=True)
        seq = np.array(sorted(live))
        N = int(rng.integers(1, 12))
        r = Round("tree", len(seq), 0, N, 40, seed=turn)
        e = orc.cache_reserve(o, seq, np.full(len(seq), N))
        assert np.array_equal(host(wf.cache_reserve(cache, i32(np.full(len(seq), N)), seqs=i32(seq))), e)
        (k, v), (kx, vx) = vectors(r.total, heads, dim, "bf16", turn, parts=2, scale=np.exp(rng.normal(0, 2)))
        wf.cache_append(cache, r.rows, k, v, seqs=i32(seq))
        dec.cache_append(o, r.seqs, kx, vx, seq=seq)
        best = rng.integers(0, N, len(seq))
        al = np.array([len(q.path(int(u))) for q, u in zip(r.seqs, best)])
        wf.cache_compact(cache, r.rows, i32(al), i32(best), seqs=i32(seq))
        dec.cache_compact(o, r.seqs, al, best, o.context, seq)
        spare = [s for s in range(8) if s not in live][:2]
        if turn % 2 == 0 and spare:
            src, dst = rng.choice(seq, len(spare)), np.array(spare)
            e = dec.cache_fork(o, src, dst)
            assert np.array_equal(host(wf.cache_fork(cache, i32(src), i32(dst))), e)
            live |= {int(d) for d, s in zip(dst, e) if s}
        elif len(live) > 2:
            gone = rng.choice(sorted(live), 2, replace=False)
            wf.cache_free(cache, i32(gone))
            orc.cache_free(o, gone)
            live -= {int(s) for s in gone}
        same_cache8(o, cache)


def test_a_cache_past_32_bits():
    # The last page of the last layer lies past 2^32 bytes.
    P, layers, dim, page = 40000, 2, 128, 64
    cache = wf.PageCache8.empty(layers, P, 8, page, dim, 3, 4, block=16, device=DEV)
    cache.table[0, 0] = P - 1
    cache.refs[P - 1] = 1
    cache.held[0] = 1
    cache.context[0] = 50
    rows = wf.tree_rows(i32(np.array([[-1, 0, 0, 2]])))
    assert cache.k[1, P - 1].data_ptr() - cache.k.data_ptr() > 2**32
    x = to_e4m3(np.random.default_rng(1).normal(0, 30, (4, 8, dim)).clip(-400, 400)).to(torch.bfloat16)
    x[..., 0] = 448
    seq = torch.zeros(1, dtype=torch.int32, device=DEV)
    wf.cache_append(cache, rows, x, -x, layer=1, seqs=seq)
    k, v = wf.cache_read(cache, 4, seqs=seq, first=cache.context[:1], pending=4, layer=1)
    assert torch.equal(k[0], x) and torch.equal(v[0], -x)
    wf.cache_compact(cache, rows, i32([3]), i32([3]), seqs=seq)
    assert int(cache.context[0]) == 53
    wf.cache_fork(cache, seq, seq + 1)
    assert cache.table[1, 0].item() == 0
    k, v = wf.cache_read(cache, 3, seqs=seq + 1, first=i32([50]), layer=1)
    assert torch.equal(k[0], x[[0, 2, 3]]) and torch.equal(v[0], -x[[0, 2, 3]])
