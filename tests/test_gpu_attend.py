"""attend against float64 attention over the oracle's cache.

Tolerance, per output: with u = 2^-24, A the largest sum |q . k| scale of a row's seen keys and L its
number of keys, a float32 score is off by at most d = (D + 4) u A, its weight relative to the others
by 2 d + 8 u (two rounded exponentials and rescalings), and a sum of L such terms by another L u; so
the output by (2 d + (L + 16) u) sum p |v|.  In bfloat16 each weight p is rounded to p (1 + e),
|e| <= 2^-8, in the product and in the sum: sum p (1 + e) v / sum p (1 + e) is off by
sum p e (v - out) / sum p (1 + e), so by 2^-8 (sum p |v| + |out|) (and a part in 2^8 of that); the
output's own rounding adds 2^-8 |out|."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from gpu_helpers import DEV, dev, host
from oracle import rounds as orc
from round_helpers import Round, bits, device_cache, i32, make_cache, to_bf16

pytestmark = pytest.mark.gpu


def _queries(total, heads, dim, dtype, seed, scale=1.0):
    """q as a slice of a wider projection, and its exact float32 values."""
    x = (np.random.default_rng(seed).normal(0, 1, (total, heads + 2, dim)) * scale).astype(np.float32)
    t = dev(to_bf16(x)) if dtype == "bf16" else dev(x)
    x = bits(to_bf16(x), "bf16") if dtype == "bf16" else x
    return t[:, :heads], x[:, :heads]


def _check(r, o, cache, q, qx, dtype, *, scale=None, max_context=None, seq=None, layer=0):
    dim = o.k.shape[4]
    s = dim ** -0.5 if scale is None else scale
    top = o.table.shape[1] * o.page if max_context is None else max_context
    start = torch.full((r.total, qx.shape[1], dim), 55.0, device=DEV, dtype=q.dtype)
    got = wf.attend(q, r.rows, cache, layer=layer, seqs=None if seq is None else i32(seq), scale=scale,
                    max_context=max_context, out=start)
    got = host(got.float()).astype(np.float64)
    clean = lambda x: np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
    oc = orc.Cache(clean(o.k), clean(o.v), o.table, o.held, o.context, o.refs)
    want = orc.attend(qx, r.seqs, oc, s, top, layer, seq, out=np.full(got.shape, 55.0))
    oc.v = np.abs(oc.v)
    mag = orc.attend(qx, r.seqs, oc, s, top, layer, seq)
    u = 2.0 ** -24
    keys = np.abs(oc.k[layer]).max(initial=0)
    A = np.abs(qx).sum(-1).max() * keys * abs(s)
    L = int(o.context.max()) + max(q_.n for q_ in r.seqs) if r.seqs else 0
    tol = (2 * (dim + 4) * u * A + (L + 16) * u) * mag
    if dtype == "bf16":
        tol = tol + (2.0 ** -8 + 2.0 ** -16) * (mag + np.abs(want)) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.isfinite(got))
    off = np.abs(got - want) - tol
    assert np.all(off <= 0), f"worst {off.max():.3e} over, error {np.abs(got - want).max():.3e}"
    return got


# Contexts around the vector, tile and page sizes, ragged.
CONTEXTS = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 130, 200, 255, 257, 300]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page,heads,group", [(128, 16, 2, 4), (64, 32, 1, 1), (64, 16, 2, 7), (128, 256, 1, 8)])
@pytest.mark.parametrize("kind,K,N", [("chain", 0, 0), ("chain", 1, 0), ("chain", 16, 0), ("tree", 0, 1),
                                      ("tree", 0, 61), ("routed", 5, 20)])
def test_against_float64(dtype, dim, page, heads, group, kind, K, N):
    print(f"attend {dtype} {dim} {page} {heads}x{group} {kind} {K} {N}", flush=True)
    r = Round(kind, len(CONTEXTS), K, N, 50, seed=K + N)
    o, _ = make_cache(2, heads, page, dim, CONTEXTS, max(K + 1, N), 6, dtype=dtype)
    # positions that no row of the round sees hold NaN
    for s, q in enumerate(r.seqs):
        for j in range(int(o.context[s]) + q.n, o.table.shape[1] * page):
            w = o.where(s, j)
            if w:
                o.k[:, w[0], :, w[1]] = o.v[:, w[0], :, w[1]] = np.nan
    free = o.refs == 0
    o.k[:, free] = o.v[:, free] = np.inf
    cache = device_cache(o, dtype)
    q, qx = _queries(r.total, heads * group, dim, dtype, 5)
    _check(r, o, cache, q, qx, dtype, layer=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,K,N,group", [("chain", 0, 0, 4), ("chain", 16, 0, 4), ("tree", 0, 61, 2)])
def test_long_contexts(dtype, kind, K, N, group):
    context = [5000, 1, 2048, 4095, 0]
    r = Round(kind, 5, K, N, 50, seed=2)
    o, cache = make_cache(1, 1, 16, 128, context, max(K + 1, N), 7, dtype=dtype)
    q, qx = _queries(r.total, group, 128, dtype, 8)
    _check(r, o, cache, q, qx, dtype, max_context=5000)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_trees_and_chains(dtype):
    r = Round("routed", 3, 700, 1024, 50, seed=4)
    o, cache = make_cache(1, 1, 64, 64, [40, 3, 90], 1024, 9, dtype=dtype)
    q, qx = _queries(r.total, 2, 64, dtype, 10)
    _check(r, o, cache, q, qx, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sharp_and_shifted_scores(dtype):
    # Scores of some hundreds: weights of 0 and 1, and maxima that rise along the keys.
    r = Round("chain", 2, 3, 0, 50, seed=5)
    o, _ = make_cache(1, 1, 16, 64, [700, 129], 4, 11, dtype=dtype)
    ramp = np.linspace(0, 1, 16, dtype=np.float32)
    for s in range(2):
        for j in range(int(o.context[s])):
            w = o.where(s, j)
            o.k[:, w[0], :, w[1], 0] = np.float32(j // 16) + (ramp[j % 16] if dtype == "f32" else 0)
    cache = device_cache(o, dtype)
    if dtype == "bf16":
        o.k, o.v = (bits(to_bf16(x), "bf16") for x in (o.k, o.v))
    q, qx = _queries(r.total, 3, 64, dtype, 12)
    for scale in (4.0, -4.0, 0.0):
        _check(r, o, cache, q, qx, dtype, scale=scale)


def test_bad_data_has_its_defined_result():
    r = Round("routed", 8, 4, 11, 50, seed=13, bad=True)
    o, _ = make_cache(1, 2, 16, 64, [40, 20, 33, 0, 64, 5, 90, 17], 11, 14, dtype="bf16")
    o.table[0, 1] = -1                     # a hole
    o.table[2, 0] = o.k.shape[1] + 7       # a page that is none
    o.context[4] = -2
    o.table[3] = -1                        # no page at all
    cache = device_cache(o, "bf16")
    q, qx = _queries(r.total, 4, 64, "bf16", 15)
    seq = np.array([0, 1, 2, 3, 4, 99, -1, 7])
    _check(r, o, cache, q, qx, "bf16", seq=seq)
    _check(r, o, cache, q, qx, "bf16", seq=seq, max_context=20)   # longer contexts give zeros


@pytest.mark.parametrize("dtype,dim", [("f32", 64), ("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("group", [1, 8])
def test_odd_values_reach_only_the_rows_that_see_them(dtype, dim, group):
    # Node 2 (a leaf) and node 5 hold infinities and NaN in some dimensions of their values, node 7
    # in its key: rows on whose path they lie get NaN there, the others are as without them.
    parent = np.array([[-1, 0, 0, 1, 1, 3, 5, 4, 7, 8, 3]])
    r = Round("tree", 1, 0, 11, 50, seed=2, parent=parent)
    o, cache = make_cache(1, 1, 16, dim, [37], 11, 7, dtype=dtype)
    q, _ = _queries(r.total, group, dim, dtype, 8)
    clean = host(wf.attend(q, r.rows, cache).float())
    at = {u: o.where(0, 37 + u) for u in (2, 5, 7)}
    cache.v[0, at[2][0], 0, at[2][1], 3] = float("nan")
    cache.v[0, at[2][0], 0, at[2][1], 8] = float("inf")
    cache.v[0, at[5][0], 0, at[5][1], dim - 1] = float("-inf")
    cache.k[0, at[7][0], 0, at[7][1], 1] = float("nan")
    got = host(wf.attend(q, r.rows, cache).float())
    for u in range(11):
        path = r.seqs[0].path(u)
        odd = np.zeros(dim, bool)
        if 2 in path:
            odd[[3, 8]] = True
        if 5 in path:
            odd[dim - 1] = True
        if 7 in path:
            odd[:] = True
        assert np.all(~np.isfinite(got[u][:, odd])), u
        assert np.array_equal(got[u][:, ~odd], clean[u][:, ~odd]), u


def test_results_repeat_and_do_not_depend_on_the_batch():
    r1 = Round("chain", 1, 4, 0, 50, seed=16)
    o, cache = make_cache(1, 2, 16, 128, [3000], 5, 17)
    q, _ = _queries(r1.total, 8, 128, "bf16", 18)
    first = wf.attend(q, r1.rows, cache, max_context=3000)
    for _ in range(3):
        assert torch.equal(wf.attend(q, r1.rows, cache, max_context=3000), first)


def test_append_then_attend_past_32_bits():
    # 2^31 elements before the pages that are read.
    P, page, dim, heads = 20000, 128, 128, 8
    cache = wf.PageCache.empty(1, P, heads, page, dim, 1, 2, device=DEV)
    cache.table[0] = i32([P - 1, P - 3])
    cache.context[0] = 150
    cache.k[0, P - 1].normal_()
    cache.k[0, P - 3].normal_()
    cache.v[0, P - 1].normal_()
    cache.v[0, P - 3].normal_()
    rows = wf.chain_rows(i32(np.zeros((1, 2))))
    x = torch.randn(3, heads, dim, device=DEV).to(torch.bfloat16)
    wf.cache_append(cache, rows, x, x)
    q = torch.randn(3, heads, dim, device=DEV).to(torch.bfloat16)
    out = wf.attend(q, rows, cache)
    k, v = (torch.cat([t[0, P - 1], t[0, P - 3]], 1)[:, :153].float() for t in (cache.k, cache.v))
    w = torch.matmul(q.float().transpose(0, 1), k.transpose(1, 2).contiguous()) * dim ** -0.5
    see = torch.arange(153, device=DEV) <= torch.arange(150, 153, device=DEV)[:, None]
    ref = torch.matmul(torch.softmax(w.masked_fill(~see, -np.inf), -1), v).transpose(0, 1)
    # normal data: scores of a few units; two bfloat16 roundings of values of order one
    assert float((out.float() - ref).abs().max()) < 2 * 2.0 ** -8 * float(v.abs().max())


@pytest.mark.parametrize("dtype,dim", [("f32", 64), ("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("kind,K,N,group", [("chain", 0, 0, 4), ("chain", 4, 0, 5), ("chain", 11, 0, 4),
                                            ("chain", 16, 0, 8), ("tree", 0, 13, 3), ("tree", 0, 40, 4)])
def test_infinite_values_do_as_the_sum_has_it(dtype, dim, kind, K, N, group):
    # One rule wherever a seen position lies, among tiles that all rows see or those that some do:
    # an infinity with a weight stays one, NaN, two signs and infinities whose weight is 0 give NaN.
    for context in (6, 40, 64, 2500):
        r = Round(kind, 1, K, N, 50, seed=2)
        o, cache = make_cache(1, 1, 16, dim, [context], max(K + 1, N), 7, dtype=dtype)
        q, _ = _queries(r.total, group, dim, dtype, 8)
        q[:, :, 0] = 4.0
        cache.k[..., 0] = 0.0
        for first, last in ((1, context - 1), (context - 1, 1), (1, 2), (context - 2, context - 1)):
            if first == last:
                continue
            clean = host(wf.attend(q, r.rows, cache).float())
            (p0, o0), (p1, o1) = o.where(0, first), o.where(0, last)
            kept = cache.k.clone(), cache.v.clone()
            at, to = cache.v[0, p0, 0, o0], cache.v[0, p1, 0, o1]
            at[3], at[8], at[9] = float("inf"), float("-inf"), float("nan")
            at[11], to[11] = float("inf"), float("-inf")      # two signs
            at[12], to[12] = float("inf"), float("inf")
            # a score some thousands below the others: its weight is 0
            cache.k[0, p1, 0, o1, 0] = -8192.0
            to[dim - 1] = float("inf")
            got = host(wf.attend(q, r.rows, cache).float())
            want = {3: np.inf, 8: -np.inf, 9: np.nan, 11: np.nan, 12: np.nan, dim - 1: np.nan}
            for d in range(dim):
                if d in want:
                    assert np.array_equal(got[..., d], np.full(got.shape[:2], want[d]), equal_nan=True), \
                        (context, first, last, d, got[..., d])
                else:
                    assert np.all(np.isfinite(got[..., d])), (context, first, last, d)
            cache.k.copy_(kept[0])
            cache.k[0, p1, 0, o1, 0] = 0.0
            got = host(wf.attend(q, r.rows, cache).float())
            want[12], want[dim - 1] = np.inf, np.inf
            for d in range(dim):
                if d in want:
                    assert np.array_equal(got[..., d], np.full(got.shape[:2], want[d]), equal_nan=True), \
                        (context, first, last, d, got[..., d])
                else:
                    assert np.array_equal(got[..., d], clean[..., d]), (context, first, last, d)
            cache.v.copy_(kept[1])
