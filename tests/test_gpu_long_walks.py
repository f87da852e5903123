"""Rounds whose workgroups walk far: many rows of a sequence one after the other in the rules' kernel,
and positions past the first 1,024 of a wave, unsplit pieces and joins of more than 64 pieces in the
attention, pools that the page bookkeeping looks through in several passes.  The plans are worked out here from their definition, so that each case says which walk it
takes."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from gpu_helpers import DEV, dev, host
from oracle import rounds as orc
from round_helpers import Round, bits, device_cache, i32, make_cache, make_logits, make_rules, same_cache, to_bf16
from test_gpu_rules import _check as check_rules

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- rules


def rows_of_a_workgroup(B, rmax, V, dtype):
    chunks = -(-V // (1024 * (8 if dtype == "bf16" else 4)))
    groups = max(min(-(-12288 // (B * chunks)), rmax), -(-rmax // 64))
    return -(-rmax // groups)


# (kind, B, K, N, V), rows of a workgroup: a list of special elements and none, one chunk and several,
# chains shorter than the trees beside them, trees past 64 nodes, a sequence in one workgroup.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,group", [
    (("chain", 1100, 16, 0, 33), 2), (("routed", 1500, 9, 40, 300), 5), (("tree", 200, 0, 130, 70), 3),
    (("tree", 400, 0, 20, 8300), 2), (("routed", 1300, 20, 7, 61), 3), (("chain", 12400, 3, 0, 17), 4),
], ids=str)
def test_rules_over_groups_of_rows(shape, group, dtype):
    kind, B, K, N, V = shape
    assert rows_of_a_workgroup(B, max(K + 1, N), V, dtype) == group
    print(f"groups {shape} {dtype}", flush=True)
    r = Round(*shape, seed=B, bad=kind == "routed")
    o, rules = make_rules(r, seed=V)
    check_rules(r, make_logits(r, dtype, 7), dtype, o, rules)


def test_rules_written_past_32_bits():
    # 40,000 rows of 56,000 float32 logits end past 8 GiB and 2^31 elements, and so does the output.
    B, V, words = 40000, 56000, 1750
    g = torch.Generator(device=DEV).manual_seed(3)
    logits = torch.randn(B, V, device=DEV, generator=g)
    rows = wf.chain_rows(torch.zeros(B, 0, dtype=torch.int32, device=DEV))
    ids = torch.randint(0, V, (B,), device=DEV, generator=g, dtype=torch.int32)
    values = torch.randn(B, device=DEV, generator=g)
    banned = torch.randint(0, V, (B,), device=DEV, generator=g)
    allow = torch.full((B, words), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(B, device=DEV)
    allow[at, banned // 32] = (-1 ^ (1 << (banned % 32))).to(torch.int32)
    rules = wf.LogitRules(bias=(torch.arange(B + 1, dtype=torch.int32, device=DEV), ids, values), allow=allow)
    out = torch.full((B, V), -77.0, device=DEV)
    wf.process_logits(logits, rows, rules, out=out)
    _, _, _, t = wf.verify_constrained(logits, rows, rules)
    logits[at, ids.long()] += values
    logits[at, banned] = -float("inf")
    place = torch.arange(V, dtype=torch.int32, device=DEV)
    for lo in range(0, B, 4000):
        x = logits[lo:lo + 4000]
        assert torch.equal(out[lo:lo + 4000], x), lo
        first = torch.where(x == x.amax(1, keepdim=True), place, V).amin(1)
        assert torch.equal(t[lo:lo + 4000], first.to(torch.int32)), lo


# ----------------------------------------------------------------------------- attention


def pieces(cache, rows, q_heads, max_context):
    """Pieces of the plan, from the workspace that holds their parts (0 bytes: one piece)."""
    part = rows.total * q_heads * (cache.head_dim + 2) * 4
    size = wf.attend_workspace_bytes(cache, rows, q_heads, max_context)
    return max(1, size // part)


def _tolerance(qx, o, r, mag, want, scale, dtype):
    """test_gpu_attend's bound."""
    u, dim = 2.0 ** -24, qx.shape[2]
    A = np.abs(qx).sum(-1).max() * np.abs(o.k).max() * scale
    L = int(o.context.max()) + max(q.n for q in r.seqs)
    tol = (2 * (dim + 4) * u * A + (L + 16) * u) * mag
    if dtype == "bf16":
        tol = tol + (2.0 ** -8 + 2.0 ** -16) * (mag + np.abs(want)) + 2.0 ** -8 * np.abs(want)
    return tol


def _compare(got, qx, r, o, dtype):
    """Rows of attend against the oracle's float64."""
    scale, top = o.k.shape[4] ** -0.5, o.table.shape[1] * o.page
    want = orc.attend(qx, r.seqs, o, scale, top)
    mag = orc.attend(qx, r.seqs, orc.Cache(o.k, np.abs(o.v), o.table, o.held, o.context, o.refs), scale, top)
    off = np.abs(got - want) - _tolerance(qx, o, r, mag, want, scale, dtype)
    assert np.all(off <= 0), f"worst {off.max():.3e} over, error {np.abs(got - want).max():.3e}"


def _values(total, heads, dim, dtype, seed):
    x = np.random.default_rng(seed).normal(0, 1, (total, heads, dim)).astype(np.float32)
    x[..., 0] = 20.0
    return x if dtype == "f32" else bits(to_bf16(x), "bf16")


def _long_cache(context, most, dim, dtype, page):
    """Keys whose scores rise by some 40 along the first sequence's positions and fall along the
    second's, pages missing past the first 1,024 positions of the last."""
    o, _ = make_cache(1, 1, page, dim, context, most, 7, dtype=dtype)
    for s, sign in ((0, 1.0), (1, -1.0)):
        for j in range(context[s]):
            p, off = o.where(s, j)
            o.k[0, p, :, off, 0] = sign * 20.0 * j / context[s] * (dim / 128) ** 0.5
    if dtype == "bf16":
        o.k = bits(to_bf16(o.k), "bf16")
    holes = np.arange(1100 // page, context[2] // page, 7)
    o.table[2, holes] = -1
    o.table[2, holes[1::2]] = o.k.shape[1] + 1
    return o, device_cache(o, dtype)


# Queries of a key-value head up to 16, 32, 64 and more: every form of the kernel, in one piece whose
# waves (or workgroups) pass more than 2,048 positions.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64)])
@pytest.mark.parametrize("kind,K,N", [("chain", 0, 0), ("chain", 4, 0), ("tree", 0, 12), ("chain", 16, 0),
                                      ("tree", 0, 20)])
def test_one_piece_over_a_long_context(dtype, dim, page, kind, K, N):
    print(f"one piece {dtype} {dim} {page} {kind} {K} {N}", flush=True)
    B, group, context = 512, 4, [9001, 8300, 9000]
    n = max(K + 1, N)
    r = Round(kind, 3, K, N, 50, seed=2)
    o, cache = _long_cache(context, n, dim, dtype, page)
    qx = _values(3 * n, group, dim, dtype, 8)
    # Every sequence of the batch is one of the three, with that one's queries.
    who = np.arange(B) % 3
    rows = wf.chain_rows(i32(np.zeros((B, K)))) if kind == "chain" else wf.tree_rows(i32(r.parent[who]))
    assert pieces(cache, rows, group, 9001) == 1
    x = qx.reshape(3, n, group, dim)[who].reshape(B * n, group, dim)
    q = dev(to_bf16(x)) if dtype == "bf16" else dev(x)
    got = host(wf.attend(q, rows, cache, seqs=i32(who), max_context=9001).float()).astype(np.float64)
    got = got.reshape(B, n, group, dim)
    for b in range(3, B):
        assert np.array_equal(got[b], got[b % 3]), "the same rows elsewhere in the batch"
    _compare(got[:3].reshape(3 * n, group, dim), qx, r, o, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("kind,K,N", [("chain", 0, 0), ("tree", 0, 20)])
def test_more_than_64_pieces(dtype, dim, kind, K, N):
    print(f"many pieces {dtype} {dim} {kind}", flush=True)
    n = max(K + 1, N)
    r = Round(kind, 3, K, N, 50, seed=3)
    o, cache = _long_cache([20000, 9000, 16385], n, dim, dtype, 32)
    assert pieces(cache, r.rows, 2, 20000) > 64
    qx = _values(3 * n, 2, dim, dtype, 9)
    q = dev(to_bf16(qx)) if dtype == "bf16" else dev(qx)
    got = host(wf.attend(q, r.rows, cache, max_context=20000).float()).astype(np.float64)
    _compare(got, qx, r, o, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,K,N", [("chain", 3, 0), ("routed", 5, 21)])
def test_a_sequence_does_not_see_the_rest_of_its_batch(dtype, kind, K, N):
    # One plan (shapes, cache geometry, max_context): a sequence's rows keep every bit whatever the
    # other sequences' lengths, pages, keys and queries are, and on every repetition.
    B = 6
    r = Round(kind, B, K, N, 50, seed=4)
    o, cache = make_cache(1, 2, 16, 64, [3000, 700, 1, 2990, 40, 1025], 21, 5, dtype=dtype)
    x = np.random.default_rng(6).normal(0, 1, (r.total, 8, 64)).astype(np.float32)
    q = dev(to_bf16(x)) if dtype == "bf16" else dev(x)
    first = wf.attend(q, r.rows, cache, max_context=3000)
    assert torch.equal(wf.attend(q, r.rows, cache, max_context=3000)[:r.seqs[-1].row0], first[:r.seqs[-1].row0])
    keep = (0, 3)
    mine = np.concatenate([np.arange(r.seqs[b].row0, r.seqs[b].row0 + r.seqs[b].n) for b in keep])
    other = torch.ones(r.total, dtype=torch.bool, device=DEV)
    other[dev(mine)] = False
    q[other] = 3.0
    for b in set(range(B)) - set(keep):
        held = host(cache.table)[b, :host(cache.held)[b]]
        cache.k[:, i32(held).long()] = float("nan")
        cache.context[b] = (7 * b) % 12
        cache.table[b, 0] = -1
    got = wf.attend(q, r.rows, cache, max_context=3000)
    assert torch.equal(got[dev(mine)], first[dev(mine)])


# ----------------------------------------------------------------------------- pages


@pytest.mark.parametrize("taken", [0.0, 0.98, 0.9995])
def test_pages_of_a_pool_of_several_passes(taken):
    # A pass looks at 16,384 pages: the first suffices where all are free, the demands reach into the
    # second, or through all three, where some twenty are free and the last demands find too few.
    P, S = 40000, 700
    rng = np.random.default_rng(int(taken * 1e4))
    refs = (rng.random(P) < taken).astype(np.int32)
    kv = np.zeros((1, P, 1, 16, 64), np.float32)
    o = orc.Cache(kv, kv.copy(), np.full((S, 12), -1, np.int32), np.zeros(S, np.int32),
                  np.zeros(S, np.int32), refs)
    cache = device_cache(o, "f32")
    seq = rng.permutation(S)[:300]
    count = rng.integers(0, 40, 300)
    e = orc.cache_reserve(o, seq, count)
    assert o.table.max() // 16384 == {0.0: 0, 0.98: 1, 0.9995: 2}[taken]
    assert np.array_equal(host(wf.cache_reserve(cache, i32(count), seqs=i32(seq))), e)
    same_cache(o, cache)
    o.context[:] = np.minimum(5, 16 * o.held)
    cache.context.copy_(i32(o.context))
    src = np.flatnonzero(o.held > 0)[:150]
    dst = np.flatnonzero(o.held == 0)[:len(src)]
    e = orc.cache_fork(o, src, dst)
    assert np.array_equal(host(wf.cache_fork(cache, i32(src), i32(dst))), e)
    same_cache(o, cache)
