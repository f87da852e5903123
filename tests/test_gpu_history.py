"""history_prompt and history_update against the oracle, exactly."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from gpu_helpers import DEV, host
from oracle import rounds as orc
from round_helpers import Round, i32

pytestmark = pytest.mark.gpu


def _history(S, V, seed):
    h = np.random.default_rng(seed).integers(0, 3, (S, V)).astype(np.uint16)
    h[:, ::7] = 0x7FFE          # one below a full count
    buf = np.zeros((S, (V + 7) // 8 * 8), np.int16)
    buf[:, :V] = h.view(np.int16)
    return h, torch.from_numpy(buf).to(DEV)[:, :V]


@pytest.mark.parametrize("V,B,n", [(1, 1, 0), (33, 3, 5), (4099, 5, 700), (151936, 2, 9000)])
def test_prompt(V, B, n):
    rng = np.random.default_rng(V)
    h, g = _history(B + 1, V, 1)
    lens = rng.integers(0, n + 1, B)
    tokens = rng.integers(-2, V + 2, int(lens.sum()))
    offsets = np.cumsum([0, *lens])
    slot = rng.integers(-1, B + 2, B)          # shared slots and slots outside the table
    wf.history_prompt(g, i32(tokens), i32(offsets), slot=i32(slot))
    orc.history_prompt(h, tokens, offsets, slot)
    assert np.array_equal(host(g).view(np.uint16), h)


@pytest.mark.parametrize("kind,B,K,N", [("chain", 1, 0, 0), ("chain", 7, 16, 0), ("tree", 5, 0, 61),
                                        ("routed", 9, 8, 20), ("chain", 1, 1023, 0), ("tree", 1, 0, 1024)])
@pytest.mark.parametrize("bad", [False, True])
def test_update(kind, B, K, N, bad):
    V = 301
    r = Round(kind, B, K, N, V, seed=B + N, bad=bad)
    rng = np.random.default_rng(5)
    h, g = _history(B, V, 2)
    al, best, bonus = np.zeros(B, int), np.zeros(B, int), rng.integers(-1, V + 1, B)
    for b, q in enumerate(r.seqs):
        u = int(rng.integers(0, max(q.n, 1)))
        best[b], al[b] = u, len(q.path(u)) if q.n else 0
    if bad:
        al[rng.random(B) < 0.2] = 5000
        best[rng.random(B) < 0.2] = -1
    slot = rng.integers(0, B, B)               # sequences that share a row add up
    for _ in range(3):                         # the third passes the full count
        wf.history_update(g, r.rows, i32(al), None if kind == "chain" else i32(best), i32(bonus), slot=i32(slot))
        orc.history_update(h, r.seqs, al, best, bonus, slot)
    assert np.array_equal(host(g).view(np.uint16), h)
    assert np.all(h[:, ::7] <= 0x7FFF), "no count runs over into the prompt's bit"


@pytest.mark.parametrize("V", [1, 5, 33])
@pytest.mark.parametrize("slots", [1, 3])
@pytest.mark.parametrize("kind", ["chain", "tree", "routed"])
def test_last_token_of_an_odd_vocabulary(V, slots, kind):
    # The storage ends with the last row's V words, another tensor's follow: more sequences than a
    # wave has lanes share the slots, and the last token comes up several times on a path.
    B = 150
    print(f"odd vocabulary {V} {slots} {kind}", flush=True)
    seed = next(s for s in range(99) if any(V - 1 in q.token for q in Round(kind, B, 6, 9, V, seed=s, bad=True).seqs))
    r = Round(kind, B, 6, 9, V, seed=seed, bad=True)
    rng = np.random.default_rng(6)
    stride = (V + 7) // 8 * 8
    end = (slots - 1) * stride + V
    buf = np.full(end + 3, 0x1234, np.int16)
    dense = np.lib.stride_tricks.as_strided(buf, (slots, V), (2 * stride, 2))
    dense[:] = rng.integers(0, 3, (slots, V))
    dense[:, -1] = 0x7FFF - 40
    h, before = dense.astype(np.uint16).copy(), buf.copy()
    store = torch.from_numpy(buf).to(DEV)
    g = torch.as_strided(store, (slots, V), (stride, 1))
    al, best = np.zeros(B, int), np.zeros(B, int)
    for b, q in enumerate(r.seqs):
        u = int(rng.integers(0, max(q.n, 1)))
        best[b], al[b] = u, len(q.path(u)) if q.n else 0
    bonus = np.where(rng.random(B) < 0.5, V - 1, rng.integers(-1, V + 1, B))
    slot = rng.integers(0, slots, B)
    slot[rng.random(B) < 0.1] = slots
    args = (r.rows, i32(al), i32(best), i32(bonus))
    for turn in range(4):
        wf.history_update(g, *args, slot=i32(slot))
        orc.history_update(h, r.seqs, al, best, bonus, slot)
        assert np.array_equal(host(g).view(np.uint16), h), turn
    assert np.all(h[:, -1] == 0x7FFF), "four updates pass the full count"
    tokens, offsets = rng.integers(max(0, V - 2), V, 5000), np.array([0, 2000, 5000])
    two = np.array([slots - 1, slots - 1])
    wf.history_prompt(g, i32(tokens), i32(offsets), slot=i32(two))
    orc.history_prompt(h, tokens, offsets, two)
    assert np.array_equal(host(g).view(np.uint16), h)
    wf.history_update(g, *args)                # without a map: sequences past the slots enter nothing
    orc.history_update(h, r.seqs, al, best, bonus)
    assert np.array_equal(host(g).view(np.uint16), h)
    inside = np.zeros(end + 3, bool)
    np.lib.stride_tricks.as_strided(inside, (slots, V), (stride, 1))[:] = True
    assert np.array_equal(host(store)[~inside], before[~inside]), "words of no token changed"
