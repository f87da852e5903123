"""Plain CPU definitions of the calls around a round: the rules of decoding, the token history,
the attention over a paged cache, and the cache's rows and pages.

TEST INFRASTRUCTURE ONLY (see the package docstring).  A round is a list of Seq, one per
sequence; whoever builds one says where its packed rows start.  The rules are computed in
float32 with every operation rounded once, because that is how they are defined; the attention
in float64 from the exact input values.
"""

from __future__ import annotations

import dataclasses

import numpy as np

from .whiflash import MALFORMED_AL, MALFORMED_BONUS


@dataclasses.dataclass
class Seq:
    """One sequence's rows: packed rows row0 .. row0 + n - 1 (n = 0: malformed).  parent[u] is the
    parent row of row u >= 1 or -1 where its path ends, token[u] the target id its node drafted or
    -1 for none (entry 0 of both is not used)."""
    row0: int
    parent: list
    token: list
    tree: bool = False

    @property
    def n(self) -> int:
        return len(self.parent)

    def path(self, u: int) -> list:
        """Row u and its ancestors, from the last to the first that is reached."""
        nodes = []
        while u >= 0:
            nodes.append(u)
            u = self.parent[u] if u > 0 else -1
        return nodes


def chain_seq(row0, draft, V) -> Seq:
    token = [-1] + [int(t) if 0 <= t < V else -1 for t in draft]
    return Seq(row0, [-1] + list(range(len(draft))), token)


def tree_seq(row0, parent, draft_ids, d2t, V) -> Seq:
    N = len(parent)
    par = [-1] + [int(parent[u]) if 0 <= parent[u] < u else -1 for u in range(1, N)]
    token = [-1] * N
    for u in range(1, N):
        if 0 <= draft_ids[u] < len(d2t) and 0 <= d2t[draft_ids[u]] < V:
            token[u] = int(d2t[draft_ids[u]])
    return Seq(row0, par, token, True)


def routed_seqs(row_offsets, total_rows, choice, chain_draft, parent, draft_ids, d2t, V) -> list:
    K, N = chain_draft.shape[1], parent.shape[1]
    seqs = []
    for b, c in enumerate(choice):
        lo, hi = int(row_offsets[b]), int(row_offsets[b + 1])
        n = hi - lo if 0 <= lo <= hi <= total_rows else -1
        if c == 0 and n == K + 1:
            seqs.append(chain_seq(lo, chain_draft[b], V))
        elif c == 1 and n == N:
            seqs.append(tree_seq(lo, parent[b], draft_ids[b], d2t, V))
        else:
            seqs.append(Seq(lo, [], []))
    return seqs


# ----------------------------------------------------------------------------- rules


@dataclasses.dataclass
class Rules:
    """history uint16 [slots, V], slot [B], penalties float32 [B, 3], bias (offsets, ids, values),
    allow uint32 [rows, words]; None: the rule is off."""
    history: np.ndarray | None = None
    slot: np.ndarray | None = None
    penalties: np.ndarray | None = None
    bias: tuple | None = None
    allow: np.ndarray | None = None


def process_rows(x, b, seq: Seq, rules: Rules) -> np.ndarray:
    """Processed logits [n, V] float32 of one sequence, from its exact float32 logits x [n, V]."""
    x = np.array(x, np.float32)
    n, V = x.shape
    if rules.penalties is not None:
        rep, freq, pres = (np.float32(p) for p in rules.penalties[b])
        word = np.zeros(V, np.int64)
        if rules.history is not None:
            s = b if rules.slot is None else int(rules.slot[b])
            if 0 <= s < len(rules.history):
                word = rules.history[s].astype(np.int64)
        for u in range(n):
            count = word & 0x7FFF
            for a in seq.path(u):
                if a > 0 and seq.token[a] >= 0:
                    count[seq.token[a]] += 1
            seen = (count > 0) | (word >= 0x8000)
            with np.errstate(all="ignore"):
                y = np.where(x[u] > 0, x[u] / rep, x[u] * rep)
                y = y - freq * count.astype(np.float32)
                y = y - np.where(count > 0, pres, np.float32(0))
                x[u] = np.where(seen, y, x[u])
    if rules.bias is not None:
        offsets, ids, values = rules.bias
        lo = min(max(int(offsets[b]), 0), len(ids))
        hi = min(max(int(offsets[b + 1]), lo), len(ids))
        for i in range(lo, hi):
            if 0 <= ids[i] < V:
                x[:, ids[i]] = x[:, ids[i]] + np.float32(values[i])
    if rules.allow is not None:
        v = np.arange(V)
        words = rules.allow[seq.row0:seq.row0 + n].astype(np.int64) & 0xFFFFFFFF
        x[((words[:, v // 32] >> (v % 32)) & 1) == 0] = -np.inf
    return x


def constrained_tokens(x) -> np.ndarray:
    """t of processed rows: the lowest index of the maximum, -1 where all entries are -inf."""
    return np.where(np.max(x, axis=1) == -np.inf, -1, np.argmax(x, axis=1))


def verify_seq(seq: Seq, t):
    """(accept_len, bonus, best_node) of one sequence from its rows' tokens t."""
    if seq.n == 0:
        return MALFORMED_AL, MALFORMED_BONUS, -1
    best = 0
    for u in range(seq.n):
        p = seq.path(u)
        if p[-1] == 0 and all(seq.token[c] >= 0 and seq.token[c] == t[a] for c, a in zip(p, p[1:])):
            if len(p) > len(seq.path(best)):
                best = u
    return len(seq.path(best)), int(t[best]), best


# ----------------------------------------------------------------------------- history


def history_prompt(history, tokens, offsets, slot=None) -> None:
    for b in range(len(offsets) - 1):
        s = b if slot is None else int(slot[b])
        if 0 <= s < len(history):
            for v in tokens[max(int(offsets[b]), 0):max(int(offsets[b + 1]), 0)]:
                if 0 <= v < history.shape[1]:
                    history[s, v] |= np.uint16(0x8000)


def history_update(history, seqs, accept_len, best_node, bonus, slot=None) -> None:
    for b, q in enumerate(seqs):
        s = b if slot is None else int(slot[b])
        if not 0 <= s < len(history) or q.n == 0:
            continue
        u = int(best_node[b]) if q.tree else int(accept_len[b]) - 1
        if not 0 <= u < q.n or q.path(u)[-1] != 0:
            continue
        for v in [q.token[a] for a in q.path(u) if a > 0] + [int(bonus[b])]:
            if 0 <= v < history.shape[1] and history[s, v] & 0x7FFF != 0x7FFF:
                history[s, v] += np.uint16(1)


# ----------------------------------------------------------------------------- cache


@dataclasses.dataclass
class Cache:
    """k, v [layers, pages, heads, page_size, dim]; table [seqs, max_pages], held, context, refs."""
    k: np.ndarray
    v: np.ndarray
    table: np.ndarray
    held: np.ndarray
    context: np.ndarray
    refs: np.ndarray

    @property
    def page(self) -> int:
        return self.k.shape[3]

    def where(self, s: int, pos: int):
        """(page, offset) of a position, or None where it has no page."""
        j = pos // self.page
        if pos < 0 or j >= self.table.shape[1] or not 0 <= self.table[s, j] < self.k.shape[1]:
            return None
        return int(self.table[s, j]), pos % self.page


def _slots(cache, seqs, seq):
    for b, q in enumerate(seqs):
        s = b if seq is None else int(seq[b])
        yield b, q, s if 0 <= s < len(cache.table) else -1


def cache_append(cache: Cache, seqs, k_rows, v_rows, layer=0, seq=None) -> None:
    for b, q, s in _slots(cache, seqs, seq):
        if s < 0 or cache.context[s] < 0:
            continue
        for i in range(q.n):
            w = cache.where(s, int(cache.context[s]) + i)
            if w:
                cache.k[layer, w[0], :, w[1]] = k_rows[q.row0 + i]
                cache.v[layer, w[0], :, w[1]] = v_rows[q.row0 + i]


def attend(queries, seqs, cache: Cache, scale, max_context, layer=0, seq=None, out=None) -> np.ndarray:
    """float64 [rows, q_heads, dim]; rows of no well-formed sequence keep out's values."""
    rows, q_heads, dim = queries.shape
    out = np.zeros((rows, q_heads, dim)) if out is None else np.array(out, np.float64)
    heads = cache.k.shape[2]
    for b, q, s in _slots(cache, seqs, seq):
        out[q.row0:q.row0 + q.n] = 0
        c = int(cache.context[s]) if s >= 0 else -1
        if c < 0 or c > max_context or c + q.n > cache.table.shape[1] * cache.page:
            continue
        places = [cache.where(s, j) for j in range(c + q.n)]
        for u in range(q.n):
            path = set(q.path(u))
            see = [w for j, w in enumerate(places) if w and (j < c or j - c in path)]
            if not see:
                continue
            p, o = np.array(see).T
            for h in range(q_heads):
                kv = h // (q_heads // heads)
                x = cache.k[layer, p, kv, o].astype(np.float64) @ queries[q.row0 + u, h].astype(np.float64) * scale
                e = np.exp(x - x.max())
                out[q.row0 + u, h] = e @ cache.v[layer, p, kv, o].astype(np.float64) / e.sum()
    return out


def cache_compact(cache: Cache, seqs, accept_len, best_node, next_context, seq=None) -> None:
    for b, q, s in _slots(cache, seqs, seq):
        if s < 0:
            continue
        c, al = int(cache.context[s]), int(accept_len[b])
        ok = q.n > 0 and c >= 0 and 0 <= al <= q.n
        if ok and q.tree:
            u = int(best_node[b])
            path = q.path(u)[::-1] if 0 <= u < q.n else [-1]
            ok = al > 0 and path[0] == 0 and len(path) == al
            for j, node in enumerate(path if ok else []):
                a, d = cache.where(s, c + node), cache.where(s, c + j)
                if a and d:
                    cache.k[:, d[0], :, d[1]] = cache.k[:, a[0], :, a[1]]
                    cache.v[:, d[0], :, d[1]] = cache.v[:, a[0], :, a[1]]
        next_context[s] = c + al if ok else c


def _grant(cache: Cache, needs):
    """Pages for each entry (None: refused) out of the free ones, lowest first: entries are
    granted in order until one finds too few; after it only entries that need none."""
    free = [p for p in range(len(cache.refs)) if cache.refs[p] == 0]
    before, got = 0, []
    for need in needs:
        if need is None or (need > 0 and before + need > len(free)):
            got.append(None)
        else:
            got.append(free[before:before + need])
        before += need or 0
    return got


def cache_fork(cache: Cache, src, dst) -> np.ndarray:
    S, ps = len(cache.table), cache.page
    needs = []
    for i, (o, s) in enumerate(zip(src, dst)):
        ok = 0 <= o < S and 0 <= s < S and o != s and s not in list(src) and s not in list(dst[:i])
        ok = ok and cache.held[s] == 0 and 0 <= cache.context[o] <= cache.held[o] * ps
        needs.append((1 if cache.context[o] % ps else 0) if ok else None)
    status = np.zeros(len(needs), np.int32)
    for i, pages in enumerate(_grant(cache, needs)):
        if pages is None:
            continue
        o, s, c = src[i], dst[i], int(cache.context[src[i]])
        full = c // ps
        cache.table[s, :full] = cache.table[o, :full]
        for p in cache.table[o, :full]:
            if 0 <= p < len(cache.refs):
                cache.refs[p] += 1
        for p in pages:
            a = cache.table[o, full]
            cache.table[s, full], cache.refs[p] = p, 1
            if 0 <= a < len(cache.refs):
                cache.k[:, p, :, :c % ps] = cache.k[:, a, :, :c % ps]
                cache.v[:, p, :, :c % ps] = cache.v[:, a, :, :c % ps]
        cache.held[s], cache.context[s], status[i] = full + len(pages), c, 1
    return status


def cache_reserve(cache: Cache, seq, count) -> np.ndarray:
    S, most = cache.table.shape
    needs = []
    for i, (s, m) in enumerate(zip(seq, count)):
        ok = 0 <= s < S and s not in list(seq[:i]) and m >= 0 and cache.context[s] >= 0
        pages = -(-(int(cache.context[s]) + int(m)) // cache.page) if ok else 0
        needs.append(max(0, pages - int(cache.held[s])) if ok and pages <= most else None)
    status = np.zeros(len(needs), np.int32)
    for i, pages in enumerate(_grant(cache, needs)):
        if pages is not None:
            s = seq[i]
            for p in pages:
                cache.table[s, cache.held[s]], cache.refs[p] = p, 1
                cache.held[s] += 1
            status[i] = 1
    return status


def cache_free(cache: Cache, seq) -> None:
    for s in seq:
        if 0 <= s < len(cache.table) and cache.held[s] > 0:
            for j in range(cache.held[s]):
                if 0 <= cache.table[s, j] < len(cache.refs):
                    cache.refs[cache.table[s, j]] -= 1
                cache.table[s, j] = -1
            cache.held[s] = cache.context[s] = 0
