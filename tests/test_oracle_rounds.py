"""The oracle of the calls around a round, pinned by hand-worked cases and invariants (no GPU)."""

import math

import numpy as np

from oracle import rounds as orc


def test_paths_of_chains_and_trees():
    c = orc.chain_seq(3, [7, -1, 99], 50)
    assert c.n == 4 and c.path(3) == [3, 2, 1, 0] and c.token == [-1, 7, -1, -1]
    t = orc.tree_seq(0, [5, 0, 0, 1, 9, 3], [0, 1, 2, 0, 1, 7], np.array([4, 60, 5]), 50)
    assert t.path(5) == [5, 3, 1, 0] and t.path(4) == [4]     # node 4's parent is no earlier node
    assert t.token == [-1, -1, 5, 4, -1, -1]                  # 60 is past V, id 7 past the table
    r = orc.routed_seqs([0, 2, 5, 4], 9, [0, 1, 0], np.zeros((3, 1), int), np.zeros((3, 3), int),
                        np.zeros((3, 3), int), np.arange(4), 50)
    assert [q.n for q in r] == [2, 3, 0]


def test_rules_worked_by_hand():
    q = orc.chain_seq(0, [2], 4)
    h = np.array([[0x8000, 0, 3, 0]], np.uint16)
    rules = orc.Rules(history=h, penalties=np.array([[2, 0.5, 0.25]], np.float32),
                      bias=([0, 1], [3], np.array([1.5], np.float32)),
                      allow=np.array([[0b1111], [0b0111]], np.uint32))
    x = orc.process_rows(np.array([[4, 1, -1, 0], [-4, 1, 8, 0]], np.float32), 0, q, rules)
    # token 0: prompt only; token 2: put out 3 times, and once more on row 1's path
    assert x.tolist() == [[2, 1, -2 - 1.5 - 0.25, 1.5], [-8, 1, 4 - 2 - 0.25, -math.inf]]
    assert orc.constrained_tokens(x).tolist() == [0, 2]
    assert orc.constrained_tokens(np.full((1, 3), -np.inf)).tolist() == [-1]


def test_verification_of_rows_without_a_token():
    q = orc.chain_seq(0, [-1, 5], 50)
    assert orc.verify_seq(q, [-1, 5, 7]) == (1, -1, 0)
    q = orc.chain_seq(0, [5, 6], 50)
    assert orc.verify_seq(q, [5, 6, 7]) == (3, 7, 2) and orc.verify_seq(q, [5, -1, 7]) == (2, -1, 1)


def test_history_counts_stop_at_their_full_value():
    h = np.array([[0x7FFE, 0xFFFF, 0]], np.uint16)
    q = [orc.chain_seq(0, [0, 0, 1], 3)]
    orc.history_update(h, q, [4], None, [2])
    assert h.tolist() == [[0x7FFF, 0xFFFF, 1]]
    orc.history_update(h, q, [9], None, [2])
    assert h.tolist() == [[0x7FFF, 0xFFFF, 1]]
    orc.history_prompt(h, [2, 5, -1], [0, 3])
    assert h.tolist() == [[0x7FFF, 0xFFFF, 0x8001]]


def _cache(P=6, S=3, most=3):
    k = np.arange(P * 16, dtype=np.float32).reshape(1, P, 1, 16, 1)
    return orc.Cache(k, -k, np.full((S, most), -1), np.zeros(S, int), np.zeros(S, int), np.zeros(P, int))


def test_pages_lowest_first_and_balanced():
    c = _cache()
    assert orc.cache_reserve(c, [1, 0, 1], [17, 1, 5]).tolist() == [1, 1, 0]
    assert c.table[1].tolist() == [0, 1, -1] and c.table[0].tolist() == [2, -1, -1]
    c.context[1] = 20
    assert orc.cache_fork(c, [1], [2]).tolist() == [1]
    assert c.table[2].tolist() == [0, 3, -1] and c.refs.tolist() == [2, 1, 1, 1, 0, 0]
    assert c.k[0, 3, 0, :4, 0].tolist() == c.k[0, 1, 0, :4, 0].tolist() and c.k[0, 3, 0, 4, 0] == 3 * 16 + 4
    orc.cache_free(c, [1, 1])
    assert c.refs.tolist() == [1, 0, 1, 1, 0, 0] and c.held.tolist() == [1, 0, 2]
    # after the first entry that finds too few, only those that need none
    assert orc.cache_reserve(c, [1, 0], [48, 17]).tolist() == [1, 0]
    assert orc.cache_reserve(c, [0, 2], [33, 12]).tolist() == [0, 1]


def test_compaction_keeps_the_path():
    c = _cache()
    orc.cache_reserve(c, [0], [30])
    c.context[0] = 10
    before = [c.k[0, c.table[0, (10 + u) // 16], 0, (10 + u) % 16, 0] for u in range(8)]
    q = [orc.tree_seq(0, [0, 0, 0, 2, 2, 4, 4, 6], [0] * 8, np.array([1]), 9)]
    orc.cache_compact(c, q, [5], [7], c.context)
    after = [c.k[0, c.table[0, (10 + u) // 16], 0, (10 + u) % 16, 0] for u in range(5)]
    assert after == [before[u] for u in (0, 2, 4, 6, 7)] and c.context[0] == 15
    orc.cache_compact(c, q, [4], [7], c.context)               # no path of 4 rows to node 7
    assert c.context[0] == 15


def test_attention_of_one_and_of_equal_keys():
    c = _cache()
    orc.cache_reserve(c, [0], [8])
    q = [orc.chain_seq(0, [1, 1], 9)]
    c.context[0] = 4
    c.k[:] = 0                                                 # equal scores: the mean of the seen values
    out = orc.attend(np.ones((3, 2, 1), np.float32), q, c, 1.0, 100)
    seen = [-float(j) for j in range(7)]
    assert np.allclose(out[:, 0, 0], [np.mean(seen[:5]), np.mean(seen[:6]), np.mean(seen)])
    assert np.all(orc.attend(np.ones((3, 2, 1), np.float32), q, c, 1.0, 3) == 0)   # longer than max_context
