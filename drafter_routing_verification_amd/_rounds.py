"""ctypes binding of the calls around a round: decoding rules on the logits, the token
history, the paged key-value cache and the attention over it (argument marshalling only).

Three handles describe what the calls work on, each a host struct of device pointers built
once and usable for as long as its tensors are: RoundRows (the rows of a round, laid out as
the verify calls lay them out), LogitRules and PageCache.
"""

from __future__ import annotations

import ctypes

import torch

from ._binding import (_check, _device_tensor, _dtype_code, _i32, _opt_out, _out, _rows_view,
                       _workspace, lib)

ROWS_CHAIN, ROWS_TREE, ROWS_ROUTED = 0, 1, 2

_p, _i, _l, _sz, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class _RowsStruct(ctypes.Structure):
    _fields_ = [(n, _i) for n in ("kind", "B", "K", "N", "Vd", "total_rows")] + [
        (n, _p) for n in ("chain_draft", "parent", "draft_ids", "d2t", "row_offsets", "choice")]


class _RulesStruct(ctypes.Structure):
    _fields_ = [("history", _p), ("history_stride", _l), ("slots", _i), ("bias_count", _i),
                ("slot", _p), ("penalties", _p), ("bias_offsets", _p), ("bias_ids", _p),
                ("bias_values", _p), ("allow", _p), ("allow_stride", _l)]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("layer_stride", _l), ("page_stride", _l)] + [
        (n, _i) for n in ("dtype", "layers", "pages", "heads", "page_size", "head_dim", "seqs",
                          "max_pages")] + [(n, _p) for n in ("table", "held", "context", "refs")]


_R, _U, _C = (ctypes.POINTER(s) for s in (_RowsStruct, _RulesStruct, _CacheStruct))

_SIGNATURES = {
    "whiflash_process_logits": (_i, [_p, _i, _i, _l, _R, _U, _p, _i, _l, _p]),
    "whiflash_verify_constrained_workspace_bytes": (_sz, [_R, _i]),
    "whiflash_verify_constrained": (_i, [_p, _i, _i, _l, _R, _U, _p, _p, _p, _p, _p, _sz, _p]),
    "whiflash_history_prompt": (_i, [_p, _i, _i, _l, _i, _p, _p, _p, _i, _p]),
    "whiflash_history_update": (_i, [_p, _i, _i, _l, _R, _p, _p, _p, _p, _p]),
    "whiflash_cache_append": (_i, [_C, _i, _R, _p, _p, _l, _p, _l, _p]),
    "whiflash_attend_workspace_bytes": (_sz, [_C, _R, _i, _i]),
    "whiflash_attend": (_i, [_p, _l, _i, _C, _i, _R, _p, _i, _f, _p, _p, _sz, _p]),
    "whiflash_cache_compact": (_i, [_C, _R, _p, _p, _p, _p, _p]),
    "whiflash_cache_pages_workspace_bytes": (_sz, [_C, _i]),
    "whiflash_cache_fork": (_i, [_C, _i, _p, _p, _p, _p, _sz, _p]),
    "whiflash_cache_reserve": (_i, [_C, _i, _p, _p, _p, _p, _sz, _p]),
    "whiflash_cache_free": (_i, [_C, _i, _p, _p]),
}

_FN = None


def functions():
    """The library's functions of this module, with their signatures set."""
    global _FN
    if _FN is None:
        handle = lib()
        fns = {}
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
            fns[name[len("whiflash_"):]] = fn
        _FN = type("Functions", (), {k: staticmethod(v) for k, v in fns.items()})
    return _FN


_I32, _F32 = torch.int32, torch.float32


def _enter(index: int, stream):
    """Where a call runs: (its raw stream, a context to leave or None).  The tensors' device is
    made current, and a stream given is too, so that what the call allocates belongs to the
    stream that uses it."""
    if stream is None:
        if torch._C._cuda_getDevice() == index:
            return torch._C._cuda_getCurrentRawStream(index), None
        ctx = torch.cuda.device(index)
        ctx.__enter__()
        return torch._C._cuda_getCurrentRawStream(index), ctx
    if stream.device_index != index:
        raise ValueError(f"stream is of GPU {stream.device_index}, the call runs on GPU {index}")
    ctx = torch.cuda.stream(stream)
    ctx.__enter__()
    return stream.cuda_stream, ctx


def _leave(ctx) -> None:
    if ctx is not None:
        ctx.__exit__(None, None, None)


def _word(x: int, name: str) -> int:
    """x, which the C interface takes as an int32 (ctypes would drop the bits past it)."""
    if not -0x80000000 <= x <= 0x7FFFFFFF:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def _ints(t, name: str, n: int, index: int) -> int:
    """The address of a contiguous int32 tensor of n elements on GPU `index`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _I32 and t.numel() == n
            and t.get_device() == index and t.is_contiguous()):
        _i32(t, name, n)
        raise ValueError(f"{name} is on {t.device}, the call runs on GPU {index}")
    return t.data_ptr()


def _scratch(ws, nbytes: int, device):
    """(a tensor to hold, its address, its bytes) of a call's workspace."""
    ws = _workspace(ws, nbytes, device)
    return (None, None, 0) if ws is None else (ws, ws.data_ptr(), ws.numel() * ws.element_size())


class RoundRows:
    """The rows of one round (wf_round_rows).  Built by chain_rows, tree_rows and routed_rows;
    holds its tensors."""

    __slots__ = ("struct", "ref", "total", "B", "kind", "device", "index", "tensors", "tokens")

    def __init__(self, kind, B, K, N, total, device, tokens, **tensors):
        index = device.index
        self.kind, self.B, self.total, self.device, self.index = kind, B, total, device, index
        self.tokens, self.tensors = tokens, tensors
        s = self.struct = _RowsStruct(kind, B, K, N, 0, total)
        for name, t in tensors.items():
            if t is not None:
                if t.get_device() != index:
                    raise ValueError(f"{name} is on {t.device}, the round on {device}")
                setattr(s, name, t.data_ptr())
                if name == "d2t":
                    s.Vd = t.numel()
        self.ref = ctypes.byref(s)


def chain_rows(draft) -> RoundRows:
    """B chains of K drafts: draft [B, K] int32.  K = 0 is one new token per sequence."""
    _i32(draft, "draft")
    if draft.dim() != 2:
        raise ValueError("draft must be [B, K]")
    B, K = draft.shape
    return RoundRows(ROWS_CHAIN, B, K, 0, B * (K + 1), draft.device, True, chain_draft=draft)


def _tree_tensors(parent, draft_ids, d2t):
    _i32(parent, "parent")
    if parent.dim() != 2:
        raise ValueError("parent must be [B, N]")
    if (draft_ids is None) != (d2t is None):
        raise ValueError("draft_ids and d2t come together")
    if draft_ids is not None:
        _i32(draft_ids, "draft_ids", parent.numel())
        _i32(d2t, "d2t")
    return parent.shape


def tree_rows(parent, draft_ids=None, d2t=None) -> RoundRows:
    """B trees of N nodes: parent, draft_ids [B, N], d2t [Vd] int32.  The cache and the
    attention need parent alone."""
    B, N = _tree_tensors(parent, draft_ids, d2t)
    return RoundRows(ROWS_TREE, B, 0, N, B * N, parent.device, draft_ids is not None, parent=parent,
                     draft_ids=draft_ids, d2t=d2t)


def routed_rows(row_offsets, total_rows: int, choice, chain_draft, parent, draft_ids=None,
                d2t=None) -> RoundRows:
    """A routed mix, as verify_routed takes it: chains where choice is 0, trees where it is 1."""
    _i32(choice, "choice")
    B = choice.numel()
    _i32(row_offsets, "row_offsets", B + 1)
    _i32(chain_draft, "chain_draft")
    _, N = _tree_tensors(parent, draft_ids, d2t)
    if chain_draft.dim() != 2 or chain_draft.shape[0] != B or parent.shape[0] != B:
        raise ValueError("chain_draft must be [B, K] and parent [B, N] with the batch of choice")
    return RoundRows(ROWS_ROUTED, B, chain_draft.shape[1], N, _word(total_rows, "total_rows"), choice.device,
                     draft_ids is not None, chain_draft=chain_draft, parent=parent,
                     draft_ids=draft_ids, d2t=d2t, row_offsets=row_offsets, choice=choice)


def _history(history, V=None):
    """(slots, V, row stride) of a token history: an int16 [slots, V] tensor whose rows are a
    multiple of 16 bytes apart (its words are the uint16 words of the C interface)."""
    _device_tensor(history, "history")
    if history.dtype != torch.int16 or history.dim() != 2 or history.stride(1) != 1:
        raise TypeError("history must be a 2-D int16 tensor with unit stride along the vocabulary")
    slots, have = history.shape
    if V is not None and have != V:
        raise ValueError(f"history has {have} tokens, the logits {V}")
    return slots, have, history.stride(0) if slots > 1 else (have + 7) // 8 * 8


class LogitRules:
    """The rules of decoding (wf_logit_rules); every rule is optional.

    history [slots, V] int16 (history_prompt, history_update) with slot [B] int32 or None;
    penalties [B, 3] float32 (repetition, frequency, presence); bias (offsets [B + 1] int32,
    ids int32, values float32), each sequence's ids ascending; allow [rows, >= ceil(V / 32)]
    int32 bit masks.  Holds its tensors."""

    __slots__ = ("struct", "ref", "tensors", "V", "B", "rows", "index", "words")

    def __init__(self, history=None, *, slot=None, penalties=None, bias=None, allow=None):
        s = self.struct = _RulesStruct()
        self.V = self.B = self.rows = self.words = self.index = None
        self.tensors = (history, slot, penalties, bias, allow)
        if history is not None:
            s.slots, self.V, s.history_stride = _history(history)
            s.history = history.data_ptr()
            self._place(history, "history")
        if slot is not None:
            if history is None:
                raise ValueError("slot without a history")
            _i32(slot, "slot")
            s.slot = slot.data_ptr()
            self._batch(slot.numel(), "slot")
            self._place(slot, "slot")
        if penalties is not None:
            _device_tensor(penalties, "penalties")
            if penalties.dtype != torch.float32 or not penalties.is_contiguous() or \
                    penalties.dim() != 2 or penalties.shape[1] != 3:
                raise TypeError("penalties must be a contiguous float32 tensor [B, 3]")
            s.penalties = penalties.data_ptr()
            self._batch(penalties.shape[0], "penalties")
            self._place(penalties, "penalties")
        if bias is not None:
            offsets, ids, values = bias
            _i32(offsets, "bias offsets")
            _i32(ids, "bias ids")
            _device_tensor(values, "bias values")
            if values.dtype != torch.float32 or not values.is_contiguous():
                raise TypeError("bias values must be a contiguous float32 tensor")
            if values.numel() != ids.numel():
                raise ValueError(f"{ids.numel()} bias ids, {values.numel()} values")
            s.bias_offsets, s.bias_ids, s.bias_values = (t.data_ptr() for t in bias)
            s.bias_count = ids.numel()
            self._batch(offsets.numel() - 1, "bias offsets")
            for t in bias:
                self._place(t, "bias")
        if allow is not None:
            _device_tensor(allow, "allow")
            if allow.dtype != torch.int32 or allow.dim() != 2 or allow.stride(1) != 1:
                raise TypeError("allow must be a 2-D int32 tensor with unit stride along the words")
            self.rows, self.words = allow.shape
            s.allow = allow.data_ptr()
            s.allow_stride = allow.stride(0) if self.rows > 1 else max(self.words, 1)
            self._place(allow, "allow")
        self.ref = ctypes.byref(s)

    def _place(self, t, name):
        if self.index is None:
            self.index = t.get_device()
        elif t.get_device() != self.index:
            raise ValueError(f"{name} is on {t.device}, the other rules on GPU {self.index}")

    def _batch(self, B, name):
        if self.B is None:
            self.B = B
        elif self.B != B:
            raise ValueError(f"{name} is for {B} sequences, the other rules for {self.B}")

    def check(self, rows: RoundRows, V: int) -> None:
        if self.index is not None and self.index != rows.index:
            raise ValueError(f"the rules are on GPU {self.index}, the round on {rows.device}")
        if self.V is not None and self.V != V:
            raise ValueError(f"the history has {self.V} tokens, the logits {V}")
        if self.B is not None and self.B != rows.B:
            raise ValueError(f"the rules are for {self.B} sequences, the round for {rows.B}")
        if self.rows is not None and (self.rows != rows.total or self.words * 32 < V):
            raise ValueError(f"allow must hold {rows.total} rows of {(V + 31) // 32} words")


class PageCache:
    """A paged key-value cache (wf_page_cache).  k, v [layers, pages, heads, page_size, head_dim]
    (or without layers) float32 or bfloat16, each page contiguous; table [seqs, max_pages], held,
    context [seqs], refs [pages] int32.  Holds its tensors, which the calls update in place."""

    __slots__ = ("struct", "ref", "k", "v", "table", "held", "context", "refs", "device", "index",
                 "dtype", "heads", "head_dim", "seqs")

    def __init__(self, k, v, table, held, context, refs):
        _device_tensor(k, "k")
        _device_tensor(v, "v")
        if k.dim() not in (4, 5) or v.shape != k.shape or v.stride() != k.stride() or v.dtype != k.dtype:
            raise ValueError("k and v must be [layers,] pages, heads, page_size, head_dim tensors of "
                             "one shape, type and strides")
        pages, heads, page, dim = k.shape[-4:]
        st = k.stride()
        if st[-1] != 1 or st[-2] != dim or st[-3] != page * dim:
            raise ValueError("each page of k and v must be contiguous")
        layers = k.shape[0] if k.dim() == 5 else 1
        _device_tensor(table, "table")
        if table.dim() != 2:
            raise ValueError("table must be [seqs, max_pages]")
        seqs, most = table.shape
        index = self.index = k.get_device()
        if v.get_device() != index:
            raise ValueError(f"v is on {v.device}, k on {k.device}")
        self.k, self.v, self.table, self.held, self.context, self.refs = k, v, table, held, context, refs
        self.device, self.dtype, self.heads, self.head_dim, self.seqs = k.device, k.dtype, heads, dim, seqs
        self.struct = _CacheStruct(
            k.data_ptr(), v.data_ptr(), st[0] if k.dim() == 5 else 0,
            st[-4] if pages > 1 else heads * page * dim, _dtype_code(k), layers, pages, heads, page, dim,
            seqs, most, _ints(table, "table", seqs * most, index), _ints(held, "held", seqs, index),
            _ints(context, "context", seqs, index), _ints(refs, "refs", pages, index))
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, layers: int, pages: int, heads: int, page_size: int, head_dim: int, seqs: int,
              max_pages: int, *, dtype=torch.bfloat16, device="cuda"):
        """A cache of free pages and empty sequences."""
        shape = (layers, pages, heads, page_size, head_dim)
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros(shape, dtype=dtype, device=device),
                   torch.zeros(shape, dtype=dtype, device=device),
                   torch.full((seqs, max_pages), -1, **i32), torch.zeros(seqs, **i32),
                   torch.zeros(seqs, **i32), torch.zeros(pages, **i32))


# ----------------------------------------------------------------------------- logits


def _ruled(logits, rows: RoundRows, rules: LogitRules):
    _device_tensor(logits, "logits")
    if logits.get_device() != rows.index:
        raise ValueError(f"logits is on {logits.device}, the round on {rows.device}")
    if not rows.tokens:
        raise ValueError("the rules need the round's draft tokens (draft_ids and d2t)")
    V, stride = _rows_view(logits, rows.total)
    rules.check(rows, V)
    return V, stride


def process_logits(logits, rows: RoundRows, rules: LogitRules, *, out=None, dtype=torch.float32,
                   stream=None):
    """The processed logits of a round's rows (see whiflash_process_logits).  logits [rows, V] or
    [B, R, V]; out: a tensor of the rows' shape (logits itself for in place), or None for a new
    one of `dtype` whose rows are a multiple of 16 bytes apart.  Returns out."""
    V, stride = _ruled(logits, rows, rules)
    raw, ctx = _enter(rows.index, stream)
    try:
        if out is None:
            ostride = (V + 7) // 8 * 8
            out = torch.empty((rows.total, ostride), dtype=dtype, device=rows.device)
            if ostride != V:
                out = out[:, :V]
        else:
            _device_tensor(out, "out")
            if out.get_device() != rows.index:
                raise ValueError(f"out is on {out.device}, the round on {rows.device}")
            oV, ostride = _rows_view(out, rows.total)
            if oV != V:
                raise ValueError(f"out has {oV} entries a row, the logits {V}")
        _check(functions().process_logits(logits.data_ptr(), _dtype_code(logits), V, stride, rows.ref,
                                          rules.ref, out.data_ptr(), _dtype_code(out), ostride, raw))
    finally:
        _leave(ctx)
    return out


def verify_constrained_workspace_bytes(rows: RoundRows, V: int) -> int:
    return functions().verify_constrained_workspace_bytes(rows.ref, _word(V, "V"))


def verify_constrained(logits, rows: RoundRows, rules: LogitRules, *, row_argmax=True,
                       accept_len=None, bonus=None, best_node=None, workspace=None, stream=None):
    """Greedy verification of a round under the rules.  Returns (accept_len, bonus, best_node,
    row_argmax); tokens are -1 where the rules leave nothing.  row_argmax: True to allocate, a
    tensor to fill, or False/None to skip."""
    V, stride = _ruled(logits, rows, rules)
    dev, B = rows.device, rows.B
    raw, ctx = _enter(rows.index, stream)
    try:
        if accept_len is None and bonus is None and best_node is None and row_argmax is True:
            accept_len, bonus, best_node, row_argmax = torch.empty(
                3 * B + rows.total, dtype=_I32, device=dev).split_with_sizes((B, B, B, rows.total))
        else:
            accept_len = _out(accept_len, _I32, B, dev, "accept_len")
            bonus = _out(bonus, _I32, B, dev, "bonus")
            best_node = _out(best_node, _I32, B, dev, "best_node")
            row_argmax = _opt_out(row_argmax, rows.total, dev, "row_argmax")
        ws, at, size = _scratch(workspace, verify_constrained_workspace_bytes(rows, V), dev)
        _check(functions().verify_constrained(
            logits.data_ptr(), _dtype_code(logits), V, stride, rows.ref, rules.ref,
            accept_len.data_ptr(), bonus.data_ptr(), best_node.data_ptr(),
            None if row_argmax is None else row_argmax.data_ptr(), at, size, raw))
    finally:
        _leave(ctx)
    return accept_len, bonus, best_node, row_argmax


# ----------------------------------------------------------------------------- history


def history_prompt(history, tokens, offsets, *, slot=None, stream=None) -> None:
    """Marks prompt tokens: tokens[offsets[b]:offsets[b+1]] in row slot[b] (None: b)."""
    slots, V, stride = _history(history)
    index = history.get_device()
    _i32(tokens, "tokens")
    _i32(offsets, "offsets")
    if offsets.numel() < 1:
        raise ValueError("offsets must hold B + 1 elements")
    B = offsets.numel() - 1
    tokens_at = _ints(tokens, "tokens", tokens.numel(), index)
    offsets_at = _ints(offsets, "offsets", B + 1, index)
    slot_at = None if slot is None else _ints(slot, "slot", B, index)
    raw, ctx = _enter(index, stream)
    try:
        _check(functions().history_prompt(history.data_ptr(), slots, V, stride, B, slot_at, tokens_at,
                                          offsets_at, tokens.numel(), raw))
    finally:
        _leave(ctx)


def _verified(rows: RoundRows, accept_len, best_node):
    """The addresses of a verification's accept_len and best_node (None for rounds of chains)."""
    at = _ints(accept_len, "accept_len", rows.B, rows.index)
    if best_node is not None:
        return at, _ints(best_node, "best_node", rows.B, rows.index)
    if rows.kind != ROWS_CHAIN:
        raise ValueError("rounds with trees need best_node")
    return at, None


def history_update(history, rows: RoundRows, accept_len, best_node, bonus, *, slot=None,
                   stream=None) -> None:
    """Enters a verified round's accepted draft tokens and bonus tokens into the history.
    best_node may be None for rounds of chains."""
    slots, V, stride = _history(history)
    if history.get_device() != rows.index:
        raise ValueError(f"history is on {history.device}, the round on {rows.device}")
    if not rows.tokens:
        raise ValueError("the history needs the round's draft tokens (draft_ids and d2t)")
    al, best = _verified(rows, accept_len, best_node)
    bonus_at = _ints(bonus, "bonus", rows.B, rows.index)
    slot_at = None if slot is None else _ints(slot, "slot", rows.B, rows.index)
    raw, ctx = _enter(rows.index, stream)
    try:
        _check(functions().history_update(history.data_ptr(), slots, V, stride, rows.ref, slot_at, al,
                                          best, bonus_at, raw))
    finally:
        _leave(ctx)


# ----------------------------------------------------------------------------- cache


def _cache_call(cache: PageCache, rows: RoundRows, seqs):
    if rows.index != cache.index:
        raise ValueError(f"the round is on {rows.device}, the cache on {cache.device}")
    return None if seqs is None else _ints(seqs, "seqs", rows.B, cache.index)


def _vectors(t, name, rows, heads, cache):
    """Row stride of [rows, heads, head_dim] vectors of the cache's type, each row contiguous."""
    _device_tensor(t, name)
    if t.get_device() != cache.index or t.dtype != cache.dtype:
        raise ValueError(f"{name} must be {cache.dtype} on {cache.device}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != rows or shape[2] != cache.head_dim or \
            (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [{rows}, {heads or 'heads'}, {cache.head_dim}]")
    st = t.stride()
    if st[2] != 1 or (shape[1] > 1 and st[1] != shape[2]):
        raise ValueError(f"each row of {name} must be contiguous")
    return st[0] if rows > 1 else shape[1] * shape[2]


def cache_append(cache: PageCache, rows: RoundRows, k_rows, v_rows, *, layer: int = 0, seqs=None,
                 stream=None) -> None:
    """Puts the rows' keys and values [rows, heads, head_dim] at positions context + i of their
    sequences in one layer.  seqs [B] int32: the cache sequences (None: 0 .. B-1)."""
    seq = _cache_call(cache, rows, seqs)
    ks = _vectors(k_rows, "k_rows", rows.total, cache.heads, cache)
    vs = _vectors(v_rows, "v_rows", rows.total, cache.heads, cache)
    raw, ctx = _enter(cache.index, stream)
    try:
        _check(functions().cache_append(cache.ref, _word(layer, "layer"), rows.ref, seq, k_rows.data_ptr(), ks,
                                        v_rows.data_ptr(), vs, raw))
    finally:
        _leave(ctx)


def attend_workspace_bytes(cache: PageCache, rows: RoundRows, q_heads: int, max_context: int) -> int:
    return functions().attend_workspace_bytes(cache.ref, rows.ref, _word(q_heads, "q_heads"),
                                              _word(max_context, "max_context"))


def attend(q, rows: RoundRows, cache: PageCache, *, layer: int = 0, seqs=None, scale=None,
           max_context=None, out=None, workspace=None, stream=None):
    """Attention of the rows' queries q [rows, q_heads, head_dim] over the cache.  scale: None for
    head_dim ** -0.5; max_context: an upper bound of the sequences' committed lengths that the host
    knows (None: what a table row can hold).  Returns out [rows, q_heads, head_dim]."""
    seq = _cache_call(cache, rows, seqs)
    qs = _vectors(q, "q", rows.total, None, cache)
    heads = q.shape[1]
    if max_context is None:
        max_context = cache.struct.max_pages * cache.struct.page_size
    if scale is None:
        scale = cache.head_dim ** -0.5
    raw, ctx = _enter(cache.index, stream)
    try:
        if out is None:
            out = torch.empty((rows.total, heads, cache.head_dim), dtype=cache.dtype, device=cache.device)
        else:
            _out(out, cache.dtype, rows.total * heads * cache.head_dim, cache.device, "out")
        ws, at, size = _scratch(workspace, attend_workspace_bytes(cache, rows, heads, max_context),
                                cache.device)
        _check(functions().attend(q.data_ptr(), qs, heads, cache.ref, _word(layer, "layer"), rows.ref, seq,
                                  max_context, scale, out.data_ptr(), at, size, raw))
    finally:
        _leave(ctx)
    return out


def cache_compact(cache: PageCache, rows: RoundRows, accept_len, best_node=None, *, seqs=None,
                  next_context=None, stream=None) -> None:
    """Moves each accepted tree path's rows to the front of the round's positions, in every layer,
    and commits accept_len positions: next_context (None: the cache's context, in place) gets
    context + accept_len.  best_node may be None for rounds of chains."""
    seq = _cache_call(cache, rows, seqs)
    al, best = _verified(rows, accept_len, best_node)
    after = None if next_context is None else _ints(next_context, "next_context", cache.seqs, cache.index)
    raw, ctx = _enter(cache.index, stream)
    try:
        _check(functions().cache_compact(cache.ref, rows.ref, seq, al, best, after, raw))
    finally:
        _leave(ctx)


def cache_pages_workspace_bytes(cache: PageCache, n: int) -> int:
    return functions().cache_pages_workspace_bytes(cache.ref, n)


def _pages_call(fn, cache, first, second, names, status, workspace, stream):
    _i32(first, names[0])
    n = first.numel()
    one = _ints(first, names[0], n, cache.index)
    two = _ints(second, names[1], n, cache.index)
    raw, ctx = _enter(cache.index, stream)
    try:
        status = _out(status, _I32, n, cache.device, "status")
        ws, at, size = _scratch(workspace, cache_pages_workspace_bytes(cache, n), cache.device)
        _check(fn(cache.ref, n, one, two, status.data_ptr(), at, size, raw))
    finally:
        _leave(ctx)
    return status


def cache_fork(cache: PageCache, src, dst, *, status=None, workspace=None, stream=None):
    """Makes sequence dst[i] a fork of src[i]: full pages shared, the last partly filled one copied.
    Returns status [n] int32, 1 where done, 0 where refused."""
    return _pages_call(functions().cache_fork, cache, src, dst, ("src", "dst"), status, workspace, stream)


def cache_reserve(cache: PageCache, count, *, seqs, status=None, workspace=None, stream=None):
    """Gives sequence seqs[i] pages for context + count[i] positions.  Returns status [n] int32."""
    return _pages_call(functions().cache_reserve, cache, seqs, count, ("seqs", "count"), status,
                       workspace, stream)


def cache_free(cache: PageCache, seqs, *, stream=None) -> None:
    """Frees the sequences' pages and empties the sequences."""
    _i32(seqs, "seqs")
    n = seqs.numel()
    at = _ints(seqs, "seqs", n, cache.index)
    raw, ctx = _enter(cache.index, stream)
    try:
        _check(functions().cache_free(cache.ref, n, at, raw))
    finally:
        _leave(ctx)
