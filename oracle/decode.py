"""Plain CPU definitions of a decoding step's calls: rotary positions, the paged cache of 8 bits and
the attention over it, log probabilities.

TEST INFRASTRUCTURE ONLY (see the package docstring).  In float64 from the exact input values; what
the 8-bit cache holds is defined value by value and compared exactly.
"""

from __future__ import annotations

import dataclasses

import numpy as np

from . import rounds

LEAST, MOST = -100, 119  # exponents of a block's scale


# ----------------------------------------------------------------------------- rotary


def rotate(x, seqs, frequency, layout, magnitude, context, seq=None, out=None):
    """Rows x [rows, heads, dim] turned, in float64; rows that are left as they were keep out's."""
    x = np.asarray(x, np.float64)
    out = np.array(x if out is None else out, np.float64)
    pairs = len(frequency)
    one = np.arange(pairs) * (2 if layout == "interleaved" else 1)
    two = one + (1 if layout == "interleaved" else pairs)
    for b, q in enumerate(seqs):
        s = b if seq is None else int(seq[b])
        if not 0 <= s < len(context) or context[s] < 0:
            continue
        for u in range(q.n):
            angle = (int(context[s]) + len(q.path(u)) - 1) * np.asarray(frequency, np.float64)
            c, d = np.cos(angle) * magnitude, np.sin(angle) * magnitude
            row = x[q.row0 + u]
            out[q.row0 + u] = row
            out[q.row0 + u][:, one] = row[:, one] * c - row[:, two] * d
            out[q.row0 + u][:, two] = row[:, two] * c + row[:, one] * d
    return out


# ----------------------------------------------------------------------------- 8-bit cache


def round_e4m3(x):
    """The nearest e4m3 number (ties to even), at most 448; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x)
    y = np.where(ok, x, 0.0)
    lead = np.frexp(y)[1] - 1
    step = np.ldexp(1.0, np.maximum(lead, -6) - 3)
    return np.where(ok, np.clip(np.rint(y / step) * step, -448, 448), np.nan).astype(np.float32)


def block_exponent(x) -> int:
    """The exponent of a block that holds the values x."""
    x = np.abs(np.asarray(x, np.float64))
    top = x[np.isfinite(x)].max(initial=0.0)
    e = LEAST
    while e < MOST and top > 448 * 2.0 ** e:
        e += 1
    return e


@dataclasses.dataclass
class Cache8(rounds.Cache):
    """A Cache whose k and v hold the e4m3 numbers; k_scale, v_scale [layers, pages, heads, blocks] the
    bytes of their scales."""
    k_scale: np.ndarray = None
    v_scale: np.ndarray = None

    @property
    def block(self) -> int:
        return self.page // self.k_scale.shape[3]

    def values(self) -> rounds.Cache:
        """The cache of what the numbers stand for."""
        up = lambda x, s: (x.astype(np.float64) * np.ldexp(1.0, np.repeat(s.astype(int) - 127, self.block, 3))[..., None])  # noqa: E731
        return rounds.Cache(up(self.k, self.k_scale), up(self.v, self.v_scale), self.table, self.held, self.context,
                            self.refs)

    def parts(self):
        return (self.k, self.k_scale), (self.v, self.v_scale)


def _write_block(x, scale, layer, page, h, off, values) -> None:
    """A block's first positions from offset `off` of a page hold `values` [n, dim]."""
    block = x.shape[3] // scale.shape[3]
    e = block_exponent(values)
    x[layer, page, h, off:off + len(values)] = round_e4m3(np.asarray(values, np.float64) * 2.0 ** -e)
    scale[layer, page, h, off // block] = e + 127


def _block_values(x, scale, layer, page, h, off, n):
    block = x.shape[3] // scale.shape[3]
    e = int(scale[layer, page, h, off // block]) - 127
    return x[layer, page, h, off:off + n].astype(np.float64) * 2.0 ** e


def cache_append(cache: Cache8, seqs, k_rows, v_rows, layer=0, seq=None) -> None:
    block = cache.block
    for b, q, s in rounds._slots(cache, seqs, seq):
        c = int(cache.context[s]) if s >= 0 else -1
        if c < 0 or q.n == 0:
            continue
        for lo in range(c // block * block, c + q.n, block):
            w = cache.where(s, lo)
            if not w:
                continue
            first, last = max(lo, c), min(lo + block, c + q.n)
            for (x, scale), rows in zip(cache.parts(), (k_rows, v_rows)):
                for h in range(x.shape[2]):
                    new = rows[q.row0 + first - c:q.row0 + last - c, h]
                    held = _block_values(x, scale, layer, w[0], h, w[1], first - lo)
                    _write_block(x, scale, layer, w[0], h, w[1], np.concatenate([held, new]))


def cache_read(cache: Cache8, count, seq=None, first=None, pending=0, layer=0):
    """(k, v) [B, count, heads, dim] in float64."""
    v = cache.values()
    n = len(cache.table) if seq is None else len(seq)
    out = np.zeros((2, n, count, cache.k.shape[2], cache.k.shape[4]))
    for b in range(n):
        s = b if seq is None else int(seq[b])
        if not 0 <= s < len(cache.table) or cache.context[s] < 0:
            continue
        for i in range(count):
            pos = i + (0 if first is None else int(first[b]))
            w = cache.where(s, pos) if 0 <= pos < cache.context[s] + pending else None
            if w:
                out[0, b, i], out[1, b, i] = v.k[layer, w[0], :, w[1]], v.v[layer, w[0], :, w[1]]
    return out[0], out[1]


def cache_compact(cache: Cache8, seqs, accept_len, best_node, next_context, seq=None) -> None:
    block = cache.block
    for b, q, s in rounds._slots(cache, seqs, seq):
        if s < 0:
            continue
        c, al = int(cache.context[s]), int(accept_len[b])
        ok = q.n > 0 and c >= 0 and 0 <= al <= q.n
        if ok and q.tree:
            u = int(best_node[b])
            path = q.path(u)[::-1] if 0 <= u < q.n else [-1]
            ok = al > 0 and path[0] == 0 and len(path) == al
            moved = next((j for j, node in enumerate(path) if node != j), al) if ok else al
            if ok and moved < al:
                was = cache.values()
                for lo in range((c + moved) // block * block, c + al, block):
                    d = cache.where(s, lo)
                    if not d:
                        continue
                    last = min(lo + block, c + al)
                    places = [cache.where(s, p if p < c else c + path[p - c]) for p in range(lo, last)]
                    for (x, scale), old in zip(cache.parts(), (was.k, was.v)):
                        for layer in range(x.shape[0]):
                            for h in range(x.shape[2]):
                                vals = [old[layer, w[0], h, w[1]] if w else None for w in places]
                                e = block_exponent(np.concatenate([y for y in vals if y is not None] or [np.zeros(1)]))
                                for j, y in enumerate(vals):
                                    if y is not None:
                                        x[layer, d[0], h, d[1] + j] = round_e4m3(y * 2.0 ** -e)
                                scale[layer, d[0], h, d[1] // block] = e + 127
        next_context[s] = c + al if ok else c


def cache_fork(cache: Cache8, src, dst):
    status = rounds.cache_fork(cache, src, dst)
    for o, s, done in zip(src, dst, status):
        c = int(cache.context[s]) if done else 0
        if c % cache.page:
            a, p = cache.table[o, c // cache.page], cache.table[s, c // cache.page]
            used = -(-(c % cache.page) // cache.block)
            if 0 <= a < cache.k.shape[1]:
                for _, scale in cache.parts():
                    scale[:, p, :, :used] = scale[:, a, :, :used]
    return status


def attend(queries, seqs, cache: Cache8, scale, max_context, layer=0, seq=None, out=None):
    return rounds.attend(queries, seqs, cache.values(), scale, max_context, layer, seq, out)


# ----------------------------------------------------------------------------- log probabilities


def token_logprobs(logits, tokens, rows, top):
    """(logprob [n, given], entropy [n], top_tokens, top_logprobs [n, top]) in float64."""
    logits = np.asarray(logits, np.float64)
    n, V = len(rows), logits.shape[1]
    logprob = np.full(tokens.shape, np.nan)
    entropy, ids, likely = np.full(n, np.nan), np.full((n, top), -1), np.full((n, top), np.nan)
    for i, r in enumerate(rows):
        if not 0 <= r < len(logits):
            continue
        x = logits[r]
        if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
            continue
        z = x - x.max()
        p = np.exp(z)
        logp = z - np.log(p.sum())
        some = p > 0
        entropy[i] = -(p[some] * logp[some]).sum() / p.sum()
        inside = (tokens[i] >= 0) & (tokens[i] < V)
        logprob[i, inside] = logp[tokens[i][inside]]
        order = np.argsort(-x, kind="stable")[:top]
        order = order[x[order] > -np.inf]
        likely[i] = -np.inf
        ids[i, :len(order)], likely[i, :len(order)] = order, logp[order]
    return logprob, entropy, ids, likely
