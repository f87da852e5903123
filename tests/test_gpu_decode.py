"""A decoding step's calls used together: several steps of a small serving loop against the oracle,
the same calls captured in a graph and replayed, two streams at once, a captured call beside an
eager one, and the refusals that need GPU tensors."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from decode_helpers import full, make_cache8, same_cache8, vectors
from gpu_helpers import DEV, host
from oracle import decode as dec
from oracle import rounds as orc
from round_helpers import Round, bits, i32, make_logits, stored
from test_gpu_attend8 import _check as check_attend
from test_gpu_logprobs import _check as check_logprobs
from test_gpu_rotary import _check as check_rotary

pytestmark = pytest.mark.gpu

HEADS, GROUP, DIM, PAGE = 2, 4, 64, 16
PAIRS = 24


def _rotary():
    return wf.Rotary.of(PAIRS, 5000.0, scaling=("wavelength", 4.0, 1.0, 4.0, 64), layout="interleaved", device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,K,N,block", [("chain", 4, 0, 1), ("tree", 0, 13, 16), ("routed", 3, 9, 4)])
def test_a_serving_loop(dtype, kind, K, N, block):
    # reserve, then a layer at a time rotate, append, attend; verify, compact, log probabilities of
    # what was accepted; a fork, a free and a read back
    B, V, S, layers = 4, 700, 7, 2
    o, cache = make_cache8(layers, HEADS, PAGE, DIM, block, [5, 16, 33, 0], 0, 3, spare=40, empty=S - B)
    rotary = _rotary()
    frequency = host(rotary.frequency)
    seq = np.array([2, 0, 3, 1])
    for turn in range(5):
        print("turn", turn, flush=True)
        r = Round(kind, B, K, N, V, seed=turn)
        most = max(K + 1, N)
        e = orc.cache_reserve(o, seq, np.full(B, most))
        assert np.array_equal(host(wf.cache_reserve(cache, i32(np.full(B, most)), seqs=i32(seq))), e) and e.all()
        mine = r.owned()
        for layer in range(layers):
            (q,), (qx,) = vectors(r.total, GROUP * HEADS, DIM, dtype, 100 * turn + layer)
            (k, v), (kx, vx) = vectors(r.total, HEADS, DIM, dtype, 100 * turn + layer + 50, parts=2)
            q2, k2 = full((r.total, GROUP * HEADS, DIM), 3.0, dtype), full((r.total, HEADS, DIM), 3.0, dtype)
            wf.rotate(q, k, r.rows, rotary, cache.context, seqs=i32(seq), q_out=q2, k_out=k2)
            check_rotary(r, qx, q2, frequency, "interleaved", 1.0, o.context, dtype, seq, fill=3.0)
            check_rotary(r, kx, k2, frequency, "interleaved", 1.0, o.context, dtype, seq, fill=3.0)
            wf.cache_append(cache, r.rows, k2, v, layer=layer, seqs=i32(seq))
            dec.cache_append(o, r.seqs, host(k2.float()), vx, layer=layer, seq=seq)
            same_cache8(o, cache)
            check_attend(r, o, cache, q2, host(q2.float()), dtype, seq=seq, layer=layer)
        raw = make_logits(r, "bf16", 90 + turn)
        logits = stored(raw, "bf16", 704)
        al, bonus, best, _ = wf.verify_constrained(logits, r.rows, wf.LogitRules())
        x = bits(raw, "bf16")
        # the last accepted row of each sequence, and the token that follows it
        last = np.array([s.row0 + (int(host(best)[b]) if s.tree else int(host(al)[b]) - 1) for b, s in enumerate(r.seqs)])
        tokens = host(bonus).reshape(B, 1)
        check_logprobs(x, tokens, last, 4, wf.token_logprobs(logits, bonus, rows=i32(last), top=4))
        wf.cache_compact(cache, r.rows, al, best, seqs=i32(seq))
        dec.cache_compact(o, r.seqs, host(al), host(best), o.context, seq)
        same_cache8(o, cache)
        if turn in (1, 3):   # one sequence is replaced by a fork of another
            gone, to, new = seq[1], seq[0], next(s for s in range(S) if s not in seq)
            assert np.array_equal(host(wf.cache_fork(cache, i32([to]), i32([new]))),
                                  dec.cache_fork(o, np.array([to]), np.array([new])))
            wf.cache_free(cache, i32([gone]))
            orc.cache_free(o, np.array([gone]))
            seq = np.array([seq[0], new, seq[2], seq[3]])
        for got, want in zip(wf.cache_read(cache, 50, seqs=i32(seq), layer=1, dtype=torch.float32),
                             dec.cache_read(o, 50, seq, None, 0, 1)):
            assert np.array_equal(host(got), want)


def _steps():
    """Two chains of calls, each on state, buffers and workspaces of its own."""
    made = []
    for n, (kind, dtype, block) in enumerate((("chain", "bf16", 16), ("routed", "f32", 1))):
        r = Round(kind, 5, 6, 17, 5003, seed=n)
        logits = stored(make_logits(r, dtype, 30 + n), dtype, 5008)
        _, cache = make_cache8(2, HEADS, PAGE, DIM, block, [40, 3, 16, 700, 0], 17, 40 + n, spare=9, empty=2)
        rotary = _rotary()
        (q,), _ = vectors(r.total, GROUP * HEADS, DIM, dtype, 60 + n)
        (k, v), _ = vectors(r.total, HEADS, DIM, dtype, 70 + n, parts=2)
        state = [cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, cache.table,
                 cache.held, cache.context, cache.refs]
        src, dst = i32([0, 3]), i32([5, 6])
        tokens = i32(np.arange(r.total))
        ws = [torch.empty(max(256, x), dtype=torch.uint8, device=DEV) for x in (
            wf.attend_workspace_bytes(cache, r.rows, GROUP * HEADS, 800, dtype=q.dtype),
            wf.token_logprobs_workspace_bytes(r.total, 5003, 9),
            wf.cache_pages_workspace_bytes(cache, 2))]
        made.append((r, cache, rotary, q, k, v, logits, tokens, src, dst, ws, state))

    def fn(step):
        r, cache, rotary, q, k, v, logits, tokens, src, dst, ws, _ = step
        qo, ko = torch.zeros_like(q), torch.zeros_like(k)
        wf.rotate(q, k, r.rows, rotary, cache.context, q_out=qo, k_out=ko)
        wf.cache_append(cache, r.rows, ko, v, layer=1)
        out = torch.zeros_like(qo)
        wf.attend(qo, r.rows, cache, layer=1, max_context=800, out=out, workspace=ws[0])
        done = wf.verify_constrained(logits, r.rows, wf.LogitRules(), row_argmax=False)[:3]
        found = wf.token_logprobs(logits, tokens, top=9, workspace=ws[1])
        wf.cache_compact(cache, r.rows, done[0], done[2])
        forked = wf.cache_fork(cache, src, dst, workspace=ws[2])
        kv = wf.cache_read(cache, 60, layer=1, dtype=q.dtype)
        wf.cache_free(cache, src)
        return [qo, ko, out, *done, *found, forked, *kv]

    return made, fn


def _same(got, want, what):
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(torch.nan_to_num(a.float(), nan=9.0), torch.nan_to_num(b.float(), nan=9.0)), (what, i)


def test_graphs_replay_like_eager_calls():
    made, fn = _steps()
    start = [[t.clone() for t in step[-1]] for step in made]

    def reset():
        for step, old in zip(made, start):
            for t, x in zip(step[-1], old):
                t.copy_(x)

    want, after = [], []
    for step in made:
        want.append([t.clone() for t in fn(step)])
        after.append([t.clone() for t in step[-1]])
    torch.cuda.synchronize()
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [fn(step) for step in made]
    for rep in range(3):
        reset()
        for got in outs:
            for t in got:
                t.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, step in enumerate(made):
            _same(outs[n], want[n], f"replay {rep}")
            _same(step[-1], after[n], f"state after replay {rep}")
        reset()
        for n, step in enumerate(made):  # eager work between the replays
            _same(fn(step), want[n], f"eager {rep}")


def test_two_streams_at_once():
    made, fn = _steps()
    start = [[t.clone() for t in step[-1]] for step in made]
    want = [[t.clone() for t in fn(step)] for step in made]
    for step, old in zip(made, start):
        for t, x in zip(step[-1], old):
            t.copy_(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for step, s in zip(made, streams):
        with torch.cuda.stream(s):
            got.append(fn(step))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        _same(a, b, "two streams")


def test_a_given_stream_is_used():
    # The call is ordered behind what the stream still has to do, not behind the current stream's work.
    logits = torch.zeros(64, 4096, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):
            big = (big @ big).clamp(-1, 1)
        logits[:, 7] = 30.0 + 0 * big[0, 0]
    got = wf.token_logprobs(logits, top=1, stream=s)
    torch.cuda.synchronize()
    assert (got[2] == 7).all()


def test_a_page_cache_of_another_class_is_still_one():
    class Mine(wf.PageCache):
        pass

    r = Round("tree", 2, 0, 5, 50, seed=1)
    (q,), _ = vectors(r.total, GROUP * HEADS, DIM, "bf16", 1)
    (k, v), _ = vectors(r.total, HEADS, DIM, "bf16", 2, parts=2)
    outs = []
    for kind in (wf.PageCache, Mine):
        cache = kind.empty(1, 8, HEADS, PAGE, DIM, 3, 4, dtype=torch.bfloat16, device=DEV)
        wf.cache_reserve(cache, i32([5, 5]), seqs=i32([0, 1]))
        wf.cache_append(cache, r.rows, k, v)
        out = wf.attend(q, r.rows, cache)
        wf.cache_compact(cache, r.rows, i32([2, 1]), i32([1, 0]))
        outs.append([out, wf.cache_fork(cache, i32([0]), i32([2])), cache.context, cache.k])
    _same(*outs, "subclass")


def test_refusals():
    r = Round("chain", 2, 3, 0, 50, seed=1)
    _, cache = make_cache8(2, HEADS, PAGE, DIM, 16, [5, 6], 4, 1)
    _, other = make_cache8(2, HEADS, PAGE, 128, 16, [5, 6], 4, 1)
    (q,), _ = vectors(r.total, GROUP * HEADS, DIM, "bf16", 1)
    (k, v), _ = vectors(r.total, HEADS, DIM, "bf16", 2, parts=2)
    rotary = _rotary()
    before = [t.clone() for t in (cache.k.view(torch.uint8), cache.k_scale, cache.context)]

    def refused(kind, call):
        with pytest.raises(kind):
            call()

    value = (ValueError, wf.WhiflashError)
    refused(value, lambda: wf.cache_append(cache, r.rows, k, v, layer=2))
    refused(value, lambda: wf.cache_append(cache, r.rows, k, v, layer=-1))
    refused(value, lambda: wf.cache_append(other, r.rows, k, v))
    refused(value, lambda: wf.cache_append(cache, r.rows, k[1:], v))
    refused(value, lambda: wf.cache_append(cache, r.rows, k, v.float()))
    refused((TypeError, *value), lambda: wf.cache_append(cache, r.rows, k.half(), v.half()))
    refused(value, lambda: wf.attend(q[:, :3], r.rows, cache))        # three query heads over two
    refused(value, lambda: wf.attend(q, r.rows, cache, layer=2))
    refused(value, lambda: wf.attend(q, r.rows, cache, scale=float("nan")))
    refused((TypeError, *value), lambda: wf.attend(q, r.rows, cache, out=q.float()))
    refused((TypeError, *value), lambda: wf.attend(q.transpose(0, 1), r.rows, cache))
    refused(TypeError, lambda: wf.cache_read(object(), 4))
    refused(value, lambda: wf.cache_read(cache, -1))
    refused(value, lambda: wf.cache_read(cache, 4, layer=7))
    refused(value, lambda: wf.cache_read(cache, 4, pending=-1))
    refused((TypeError, *value), lambda: wf.cache_read(cache, 4, dtype=torch.float16))
    refused((TypeError, *value), lambda: wf.rotate(q, k.float(), r.rows, rotary, cache.context))
    refused(value, lambda: wf.rotate(q[:, :, :40], None, r.rows, rotary, cache.context))   # 48 elements turn
    refused(value, lambda: wf.rotate(q, k, r.rows, rotary, cache.context, q_out=q[:, :, :48]))
    refused((TypeError, *value), lambda: wf.rotate(q, k, r.rows, rotary, cache.context.long()))
    refused(TypeError, lambda: wf.Rotary(torch.zeros(4, device=DEV)))
    logits = torch.zeros(4, 512, device=DEV)
    refused(value, lambda: wf.token_logprobs(torch.zeros(1, 64000, device=DEV), top=1,
                                             workspace=torch.empty(1, dtype=torch.uint8, device=DEV)))
    refused(value, lambda: wf.token_logprobs(logits, top=65))
    refused(value, lambda: wf.token_logprobs(logits, top=-1))
    refused(value, lambda: wf.token_logprobs(logits, i32([[1], [2]])))
    refused((TypeError, *value), lambda: wf.token_logprobs(logits.half(), top=1))
    refused((TypeError, *value), lambda: wf.token_logprobs(logits, i32([1, 2, 3, 4]).long()))
    refused(value, lambda: wf.token_logprobs(logits[:, 1:], top=1))    # 16-byte rows
    refused(value, lambda: wf.PageCache8(cache.k, cache.v, cache.k_scale, cache.v_scale[..., :0], cache.table, cache.held,
                                         cache.context, cache.refs))
    torch.cuda.synchronize()
    for a, b in zip(before, (cache.k.view(torch.uint8), cache.k_scale, cache.context)):
        assert torch.equal(a, b)
