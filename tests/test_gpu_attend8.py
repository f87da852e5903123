"""attend over a PageCache8 against float64 attention over what the cache stands for.

Tolerance, per output: with u = 2^-24, A the largest sum |q . k| scale of a row's seen keys and L its
number of keys, a float32 score is off by at most d = (D + 4) u A, its weight relative to the others
by 2 d + 8 u (two rounded exponentials and rescalings), and a sum of L such terms by another L u; so
the output by (2 d + (L + 16) u) sum p |v|.  With bfloat16 queries each weight p is rounded to
p (1 + e), |e| <= 2^-8, in the product and in the sum: sum p (1 + e) v / sum p (1 + e) is off by
sum p e (v - out) / sum p (1 + e), so by 2^-8 (sum p |v| + |out|) (and a part in 2^8 of that); the
output's own rounding adds 2^-8 |out|."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from decode_helpers import TORCH, device_cache8, make_cache8, to_e4m3, vectors
from gpu_helpers import DEV, host
from oracle import decode as dec
from oracle import rounds as orc
from round_helpers import Round, i32

pytestmark = pytest.mark.gpu


def _check(r, o, cache, q, qx, dtype, *, scale=None, max_context=None, seq=None, layer=0):
    dim = o.k.shape[4]
    s = dim ** -0.5 if scale is None else scale
    top = o.table.shape[1] * o.page if max_context is None else max_context
    start = torch.full((r.total, qx.shape[1], dim), 55.0, device=DEV, dtype=TORCH[dtype])
    got = wf.attend(q, r.rows, cache, layer=layer, seqs=None if seq is None else i32(seq), scale=scale,
                    max_context=max_context, out=start)
    got = host(got.float()).astype(np.float64)
    oc = o.values()
    oc.k, oc.v = (np.nan_to_num(x, nan=0.0) for x in (oc.k, oc.v))
    want = orc.attend(qx, r.seqs, oc, s, top, layer, seq, out=np.full(got.shape, 55.0))
    oc.v = np.abs(oc.v)
    mag = orc.attend(qx, r.seqs, oc, s, top, layer, seq)
    u = 2.0 ** -24
    A = np.abs(qx).sum(-1).max() * np.abs(oc.k[layer]).max(initial=0) * abs(s)
    L = int(o.context.max()) + max(q_.n for q_ in r.seqs) if r.seqs else 0
    tol = (2 * (dim + 4) * u * A + (L + 16) * u) * mag
    if dtype == "bf16":
        tol = tol + (2.0 ** -8 + 2.0 ** -16) * (mag + np.abs(want)) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.isfinite(got))
    off = np.abs(got - want) - tol
    assert np.all(off <= 0), f"worst {off.max():.3e} over, error {np.abs(got - want).max():.3e}"
    return got


# Contexts around the block, tile and page sizes, ragged.
CONTEXTS = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 130, 200, 255, 257, 300]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page,block,heads,group", [(128, 16, 16, 2, 4), (64, 32, 1, 1, 1), (64, 16, 4, 2, 7),
                                                        (128, 256, 64, 1, 8), (128, 32, 2, 1, 16)])
@pytest.mark.parametrize("kind,K,N", [("chain", 0, 0), ("chain", 1, 0), ("chain", 16, 0), ("tree", 0, 1),
                                      ("tree", 0, 61), ("routed", 5, 20)])
def test_against_float64(dtype, dim, page, block, heads, group, kind, K, N):
    print(f"attend8 {dtype} {dim} {page} {block} {heads}x{group} {kind} {K} {N}", flush=True)
    r = Round(kind, len(CONTEXTS), K, N, 50, seed=K + N)
    o, _ = make_cache8(2, heads, page, dim, block, CONTEXTS, max(K + 1, N), 6, spread=0.5)
    # positions that no row of the round sees hold NaN
    for s, q in enumerate(r.seqs):
        for j in range(int(o.context[s]) + q.n, o.table.shape[1] * page):
            w = o.where(s, j)
            if w:
                o.k[:, w[0], :, w[1]] = o.v[:, w[0], :, w[1]] = np.nan
    free = o.refs == 0
    o.k[:, free] = o.v[:, free] = np.nan
    o.k_scale[:, free] = o.v_scale[:, free] = 255
    cache = device_cache8(o)
    o.k_scale[:, free] = o.v_scale[:, free] = 127
    (q,), (qx,) = vectors(r.total, heads * group, dim, dtype, 5)
    _check(r, o, cache, q, qx, dtype, layer=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,K,N,group", [("chain", 0, 0, 4), ("chain", 16, 0, 4), ("tree", 0, 61, 2),
                                            ("chain", 7, 0, 4)])
@pytest.mark.parametrize("block", [1, 16])
def test_long_contexts(dtype, kind, K, N, group, block):
    context = [5000, 1, 2048, 4095, 0]
    r = Round(kind, 5, K, N, 50, seed=2)
    o, cache = make_cache8(1, 1, 16, 128, block, context, max(K + 1, N), 7, spread=0.5)
    (q,), (qx,) = vectors(r.total, group, 128, dtype, 8)
    _check(r, o, cache, q, qx, dtype, max_context=5000)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_uneven_lengths_under_a_large_bound(dtype):
    # One long sequence among short ones, and a bound far above all of them.
    context = [9000] + [int(x) for x in np.random.default_rng(1).integers(0, 300, 23)]
    r = Round("chain", 24, 2, 0, 50, seed=2)
    o, cache = make_cache8(1, 2, 64, 64, 32, context, 3, 7, spread=0.5)
    o.table = np.concatenate([o.table, np.full((24, 2000), -1, np.int32)], 1)
    cache = device_cache8(o)
    (q,), (qx,) = vectors(r.total, 4, 64, dtype, 8)
    _check(r, o, cache, q, qx, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_trees_and_chains(dtype):
    r = Round("routed", 3, 700, 1024, 50, seed=4)
    o, cache = make_cache8(1, 1, 64, 64, 16, [40, 3, 90], 1024, 9, spread=0.5)
    (q,), (qx,) = vectors(r.total, 2, 64, dtype, 10)
    _check(r, o, cache, q, qx, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sharp_and_shifted_scores(dtype):
    # Scores of some hundreds: weights of 0 and 1, and maxima that rise along the keys.
    r = Round("chain", 2, 3, 0, 50, seed=5)
    o, _ = make_cache8(1, 1, 16, 64, 1, [700, 129], 4, 11, spread=0.3)
    for s in range(2):
        for j in range(int(o.context[s])):
            w = o.where(s, j)
            top = float(j // 16) + 1
            e = int(np.floor(np.log2(top))) - 7
            o.k[0, w[0], :, w[1]] = dec.round_e4m3(np.random.default_rng(j).normal(0, 1, 64) * 2.0 ** -e)
            o.k[0, w[0], :, w[1], 0] = dec.round_e4m3(top * 2.0 ** -e)
            o.k_scale[0, w[0], :, w[1]] = e + 127
    cache = device_cache8(o)
    (q,), (qx,) = vectors(r.total, 3, 64, dtype, 12)
    for scale in (4.0, -4.0, 0.0):
        _check(r, o, cache, q, qx, dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales_far_apart(dtype):
    # Blocks from 2^-60 to 2^40 in the values, and keys whose scales differ from one position to the next.
    r = Round("tree", 2, 0, 9, 50, seed=5)
    o, _ = make_cache8(1, 2, 16, 128, 1, [300, 77], 9, 11, spread=0.7)
    rng = np.random.default_rng(3)
    o.v_scale[:] = (o.v_scale.astype(int) + rng.choice([-60, -20, 0, 5, 40], o.v_scale.shape)).astype(np.uint8)
    cache = device_cache8(o)
    (q,), (qx,) = vectors(r.total, 6, 128, dtype, 12)
    _check(r, o, cache, q, qx, dtype)


def test_bad_data_has_its_defined_result():
    r = Round("routed", 8, 4, 11, 50, seed=13, bad=True)
    o, _ = make_cache8(1, 2, 16, 64, 8, [40, 20, 33, 0, 64, 5, 90, 17], 11, 14, spread=0.5)
    o.table[0, 1] = -1                     # a hole
    o.table[2, 0] = o.k.shape[1] + 7       # a page that is none
    o.context[4] = -2
    o.table[3] = -1                        # no page at all
    cache = device_cache8(o)
    for dtype in ("bf16", "f32"):
        (q,), (qx,) = vectors(r.total, 4, 64, dtype, 15)
        seq = np.array([0, 1, 2, 3, 4, 99, -1, 7])
        _check(r, o, cache, q, qx, dtype, seq=seq)
        _check(r, o, cache, q, qx, dtype, seq=seq, max_context=20)   # longer contexts give zeros


@pytest.mark.parametrize("dtype,dim", [("f32", 64), ("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("group", [1, 8])
def test_odd_values_reach_only_the_rows_that_see_them(dtype, dim, group):
    # Node 2 (a leaf) and node 5 hold NaN in some dimensions of their values, node 7 in its key: rows on
    # whose path they lie get NaN there, the others are as without them.
    parent = np.array([[-1, 0, 0, 1, 1, 3, 5, 4, 7, 8, 3]])
    r = Round("tree", 1, 0, 11, 50, seed=2, parent=parent)
    o, cache = make_cache8(1, 1, 16, dim, 16, [37], 11, 7, spread=0.5)
    (q,), _ = vectors(r.total, group, dim, dtype, 8)
    clean = host(wf.attend(q, r.rows, cache).float())
    at = {u: o.where(0, 37 + u) for u in (2, 5, 7)}
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    v[0, at[2][0], 0, at[2][1], 3] = v[0, at[2][0], 0, at[2][1], 8] = 0x7F
    v[0, at[5][0], 0, at[5][1], dim - 1] = 0xFF
    k[0, at[7][0], 0, at[7][1], 1] = 0x7F
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
        assert np.all(np.isnan(got[u][:, odd])), u
        assert np.array_equal(got[u][:, ~odd], clean[u][:, ~odd]), u


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,K,N,group", [("chain", 0, 0, 4), ("chain", 11, 0, 4), ("tree", 0, 40, 4)])
def test_nan_among_values_that_every_row_sees(dtype, kind, K, N, group):
    for context in (6, 64, 2500):
        r = Round(kind, 1, K, N, 50, seed=2)
        o, cache = make_cache8(1, 1, 16, 64, 1, [context], max(K + 1, N), 7, spread=0.5)
        (q,), _ = vectors(r.total, group, 64, dtype, 8)
        clean = host(wf.attend(q, r.rows, cache).float())
        for j in (1, context - 1):
            p, off = o.where(0, j)
            old = cache.v.view(torch.uint8)[0, p, 0, off, 9].clone()
            cache.v.view(torch.uint8)[0, p, 0, off, 9] = 0x7F
            got = host(wf.attend(q, r.rows, cache).float())
            cache.v.view(torch.uint8)[0, p, 0, off, 9] = old
            assert np.all(np.isnan(got[..., 9]))
            rest = np.arange(64) != 9
            assert np.array_equal(got[..., rest], clean[..., rest])


@pytest.mark.parametrize("K", [0, 4])
def test_results_repeat(K):
    r = Round("chain", 3, K, 0, 50, seed=16)
    o, cache = make_cache8(1, 2, 16, 128, 16, [3000, 10, 700], 5, 17, spread=0.5)
    (q,), _ = vectors(r.total, 8, 128, "bf16", 18)
    first = wf.attend(q, r.rows, cache, max_context=3000)
    for _ in range(3):
        assert torch.equal(wf.attend(q, r.rows, cache, max_context=3000), first)


def test_a_sequence_keeps_its_bits_whatever_its_batch_holds():
    r = Round("chain", 3, 2, 0, 50, seed=16)
    o, _ = make_cache8(1, 2, 16, 128, 16, [3000, 10, 700], 5, 17, spread=0.5)
    (q,), _ = vectors(r.total, 8, 128, "bf16", 18)
    seen = []
    for others in ((10, 700), (0, 0), (2990, 1)):
        o.context[1:] = others
        o.table[1:, :] = o.table[0]            # pages enough; the values do not matter here
        seen.append(wf.attend(q, r.rows, device_cache8(o), max_context=3000)[:3])
    assert torch.equal(seen[0], seen[1]) and torch.equal(seen[0], seen[2])


def test_past_32_bits():
    # 2^32 bytes before the pages that are read.
    P, page, dim, heads = 70000, 64, 128, 8
    cache = wf.PageCache8.empty(1, P, heads, page, dim, 1, 3, block=1, device=DEV)
    at = [P - 1, P - 3, P - 2]
    cache.table[0] = i32(at)
    cache.context[0] = 150
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        for p in at:
            x[0, p] = to_e4m3(np.random.default_rng(p).normal(0, 80, (heads, page, dim)).clip(-448, 448))
            s[0, p] = 120
    rows = wf.chain_rows(i32(np.zeros((1, 2))))
    x = torch.randn(3, heads, dim, device=DEV).to(torch.bfloat16)
    wf.cache_append(cache, rows, x, x)
    q = torch.randn(3, heads, dim, device=DEV).to(torch.bfloat16)
    out = wf.attend(q, rows, cache)
    k, v = (t.float()[0].transpose(0, 1) for t in wf.cache_read(cache, 153, pending=3))
    w = torch.matmul(q.float().transpose(0, 1), k.transpose(1, 2).contiguous()) * dim ** -0.5
    see = torch.arange(153, device=DEV) <= torch.arange(150, 153, device=DEV)[:, None]
    ref = torch.matmul(torch.softmax(w.masked_fill(~see, -np.inf), -1), v.contiguous()).transpose(0, 1)
    # two bfloat16 roundings, of the weights and of the output
    assert float((out.float() - ref).abs().max()) < 2 * 2.0 ** -8 * float(v.abs().max())
