"""The operators around a verify-and-route round that are measured here, in plain form and as the
framework's calls.

A round's rows (a chain's K + 1 rows, a tree's N rows, or a routed mix of both) pass through:

  process    the rules of decoding applied to the logits: penalties for repeated tokens, biases
             and grammar masks, written out
  constrain  greedy verification under the same rules without writing processed logits, then the
             accepted tokens entered into the sequences' token history
  attend     the rows' keys and values put into a paged cache, then their attention over it
  compact    the cache rows of each accepted tree path moved to the front of the round's rows
  pages      sequences forked (full pages shared, the last one copied), given room for the next
             round, and freed again

Formulas, for row r of sequence b with path tokens P_r (the drafted tokens its prediction follows),
history word h[v] (bit 15: v is in the prompt; low 15 bits: times v was put out):

  c = (h[v] & 0x7fff) + #(P_r == v),  seen = prompt or c > 0
  x = logit;  x = seen ? (x > 0 ? x / rep : x * rep) : x;  x = x - freq * c - pres * [c > 0]
  x = x + bias[v];  x = allowed ? x : -inf
  t[r] = lowest v that holds the maximum, -1 where every x is -inf
  out[r, h] = sum_j softmax_j(scale q[r, h] . k[j]) v[j]  over the committed keys, and those of the
              round's rows that are r or on r's path
"""

import math

import numpy as np
import torch

own = False

HEADS, KV_HEADS, DIM, PAGE = 32, 8, 128, 16
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    heads = {"heads": HEADS, "kv_heads": KV_HEADS, "dim": DIM, "page": PAGE}
    layers = {"kv_heads": KV_HEADS, "dim": DIM, "page": PAGE, "dtype": "bf16", "layers": 36}
    return [
        # One sampled step of a few sequences over a small vocabulary: launches and latency.
        {"name": "process-step-f32", "op": "process", "rows": "chain", "B": 4, "K": 0, "N": 0,
         "V": 32000, "dtype": "f32"},
        # Sampled verification of a serving batch of chains: bandwidth.
        {"name": "process-chains-bf16", "op": "process", "rows": "chain", "B": 64, "K": 16, "N": 0,
         "V": 151936, "dtype": "bf16"},
        # One chain in float32, the single-sequence round.
        {"name": "constrain-chain-f32", "op": "constrain", "rows": "chain", "B": 1, "K": 16, "N": 0,
         "V": 151936, "dtype": "f32"},
        # The routed batch: half chains, half trees.
        {"name": "constrain-routed-bf16", "op": "constrain", "rows": "routed", "B": 128, "K": 16,
         "N": 61, "V": 151936, "dtype": "bf16"},
        # One new token of one sequence with a short context: latency.
        {"name": "attend-token-bf16", "op": "attend", "rows": "chain", "B": 1, "K": 0, "N": 0,
         "context": 1000, "dtype": "bf16", **heads},
        # One new token each of a ragged serving batch.
        {"name": "attend-batch-bf16", "op": "attend", "rows": "chain", "B": 64, "K": 0, "N": 0,
         "context": 8192, "dtype": "bf16", **heads},
        # Trees being verified.
        {"name": "attend-trees-bf16", "op": "attend", "rows": "tree", "B": 8, "K": 0, "N": 61,
         "context": 4096, "dtype": "bf16", **heads},
        # Two chains at the end of very long contexts.
        {"name": "attend-long-bf16", "op": "attend", "rows": "chain", "B": 2, "K": 16, "N": 0,
         "context": 131000, "dtype": "bf16", **heads},
        # A few trees accepted, every layer of the cache.
        {"name": "compact-trees", "op": "compact", "rows": "tree", "B": 8, "K": 0, "N": 61,
         "context": 1000, **layers},
        # A large routed batch accepted.
        {"name": "compact-routed", "op": "compact", "rows": "routed", "B": 128, "K": 16, "N": 61,
         "context": 200, **layers},
        # One sequence forked.
        {"name": "pages-one", "op": "pages", "B": 1, "children": 1, "context": 500, "room": 17, **layers},
        # Every sequence of a batch forked into four.
        {"name": "pages-beams", "op": "pages", "B": 32, "children": 4, "context": 500, "room": 61,
         **layers},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["process", "constrain", "attend", "compact", "pages"])
    kind = rng.choice(["chain", "tree", "routed"])
    case = {"op": op, "rows": kind, "K": rng.randint(0, 24) if kind != "tree" else 0,
            "N": rng.randint(1, 64) if kind != "chain" else 0}
    deepest = max(case["K"] + 1, case["N"])
    if op in ("process", "constrain"):
        case["V"] = _log(rng, 999, 151936)
        case["dtype"] = rng.choice(["f32", "bf16"])
        most = (1088 if op == "process" else 4352) * 151936 // (2 if case["dtype"] == "f32" else 1)
        case["B"] = _log(rng, 1, max(1, min(256, most // (case["V"] * deepest))))
        return case
    case["kv_heads"] = rng.choice([1, 2, 4, 8])
    case["dim"] = rng.choice([64, 128])
    case["page"] = rng.choice([16, 32, 64])
    if op == "attend":
        case["heads"] = case["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
        case["dtype"] = rng.choice(["f32", "bf16"])
        case["B"] = _log(rng, 1, 96)
        # keys x heads x dims stay under the largest listed case's, and scores under its as well
        room = min(131000 * 2 * 1024 // (case["B"] * case["kv_heads"] * case["dim"] * 2),
                   131000 * 2 * 17 * 32 // (case["B"] * deepest * case["heads"]))
        case["context"] = _log(rng, 1, max(2, min(131000, room)))
        return case
    case["dtype"] = rng.choice(["f32", "bf16"])
    case["layers"] = rng.randint(1, 24)
    if op == "compact":
        case["B"] = _log(rng, 1, 128)
        case["context"] = _log(rng, 1, 200)
        return case
    del case["rows"], case["K"], case["N"]
    case["B"] = _log(rng, 1, 32)
    case["children"] = rng.randint(1, 4)
    case["context"] = _log(rng, 1, 500)
    case["room"] = rng.randint(1, 61)
    return case


# ----------------------------------------------------------------------------- inputs


def _choices(case):
    """The drafter of each sequence of a routed batch: trees at every odd place."""
    return [b % 2 for b in range(case["B"])]


def _contexts(case):
    """Committed lengths: evenly spread over the upper half, the longest first."""
    B, top = case["B"], case["context"]
    return [max(0, top - (b * (top // 2)) // B) for b in range(B)]


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _tree(g, B, N):
    """Parents of random trees: each node hangs under one of the ten before it."""
    u = torch.arange(N, device="cuda")
    low = (u - 10).clamp_min(0)
    parent = low + (_rand(g, B, N) * (u - low)).floor().long().minimum((u - low - 1).clamp_min(0))
    return parent.to(torch.int32)


def _round(case, g, V):
    """The round's drafts: what a verify call takes."""
    B, K, N, kind = case["B"], case["K"], case["N"], case["rows"]
    s = {"kind": kind, "K": K, "N": N}
    if kind != "tree":
        s["draft"] = _ints(g, 0, V, B, K)
    if kind != "chain":
        Vd = min(32000, V)
        s["parent"] = _tree(g, B, N)
        s["draft_ids"] = _ints(g, 0, Vd, B, N)
        s["d2t"] = torch.randperm(V, generator=g, device="cuda")[:Vd].to(torch.int32)
    if kind == "routed":
        choice = _choices(case)
        s["choice"] = torch.tensor(choice, dtype=torch.int32, device="cuda")
        starts = np.cumsum([0] + [N if c else K + 1 for c in choice])
        s["row_offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["total_rows"] = int(starts[-1])
    else:
        s["total_rows"] = B * (K + 1 if kind == "chain" else N)
    return s


def _rules(case, g, s, rows_of):
    """History, penalties, biases and masks as a serving batch holds them."""
    B, V, rows = case["B"], case["V"], s["total_rows"]
    S = B + 3
    s["slot"] = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    skew = lambda n: (V * _rand(g, S, n) ** 3).long().clamp_max(V - 1)  # noqa: E731
    counts = torch.zeros(S, V, device="cuda").scatter_add_(1, skew(400), torch.ones(S, 400, device="cuda"))
    prompt = torch.zeros(S, V, device="cuda").scatter_(1, skew(1500), 1.0)
    stride = (V + 7) // 8 * 8
    s["history"] = torch.zeros(S, stride, dtype=torch.int16, device="cuda")[:, :V]
    s["history"].copy_((counts.int() | (prompt.int() << 15)).to(torch.int16))
    on = (_rand(g, B, 1) < 0.8).float()
    top = torch.tensor([0.3, 0.5, 0.5], device="cuda")
    s["penalties"] = (torch.tensor([1.0, 0.0, 0.0], device="cuda") + on * top * _rand(g, B, 3)).contiguous()
    ids = torch.cumsum(_ints(g, 1, max(2, V // 40), B, 48), 1)
    keep = (ids < V) & (_rand(g, B, 1) * 48 > torch.arange(48, device="cuda"))
    s["bias_offsets"] = torch.cat([keep.new_zeros(1).int(), keep.sum(1).cumsum(0).int()])
    s["bias_ids"] = ids[keep].to(torch.int32)
    s["bias_values"] = 2 * torch.randn(B, 48, generator=g, device="cuda")[keep]
    # Half of the sequences follow a grammar that leaves one token in sixteen; a few rows nothing.
    words = (V + 31) // 32
    bits = lambda: torch.randint(-2**31, 2**31, (rows, words), generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    few = bits() & bits() & bits() & bits()
    strict = (rows_of % 2 == 0)[:, None]
    none = _rand(g, rows, 1) < 0.02
    full = torch.full_like(few, -1)
    s["allow"] = torch.where(strict, torch.where(none, torch.zeros_like(few), few), full)


def _round_state(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    V, dtype = case["V"], TYPES[case["dtype"]]
    s = _round(case, g, V)
    lay = _layout(s)
    rows = s["total_rows"]
    stride = (V + 7) // 8 * 8
    logits = torch.zeros(rows, stride, dtype=dtype, device="cuda")[:, :V]
    logits.copy_(torch.randn(rows, V, generator=g, device="cuda", dtype=dtype) * 2)
    # Mostly the model agrees with the first drafted child of a row.
    child = torch.where(lay["par"] >= 0, lay["par"], lay["par"].new_full((), rows))
    first = torch.full((rows + 1,), rows, device="cuda").scatter_reduce_(
        0, child, torch.arange(rows, device="cuda"), "amin")[:rows]
    has = (first < rows) & (_rand(g, rows) < 0.8)
    token = torch.where(has, lay["tok"][first.clamp_max(rows - 1)], _ints(g, 0, V, rows).long())
    logits.scatter_(1, token.clamp_min(0)[:, None], 14 + 4 * _rand(g, rows, 1).to(dtype))
    s["logits"] = logits
    _rules(case, g, s, lay["seq"])
    word, bit = (token >> 5)[:, None], (token & 31)
    with_it = s["allow"].gather(1, word) | (1 << bit).to(torch.int32)[:, None]
    some = (s["allow"] != 0).any(1)
    s["allow"].scatter_(1, word, torch.where(some[:, None], with_it, torch.zeros_like(with_it)))
    return s


def _cache(case, g, sequences, layers, spare, rows):
    """A page pool with `sequences` held ones, their pages scattered over it."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    context = _contexts(case)
    most = (case["context"] + rows + page - 1) // page
    held = [(c + rows + page - 1) // page for c in context]
    S, P = sequences, sum(held) + spare
    shape = ([layers] if layers else []) + [P, heads, page, dim]
    dtype = TYPES[case["dtype"]]
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, most), -1, dtype=torch.int32)
    at = 0
    order_host = order.cpu()
    for b, n in enumerate(held):
        table[b, :n] = order_host[at:at + n]
        at += n
    refs = torch.zeros(P, dtype=torch.int32)
    refs[order_host[:at].long()] = 1
    whole = lambda v: torch.tensor(v + [0] * (S - len(v)), dtype=torch.int32, device="cuda")  # noqa: E731
    return {"k": torch.randn(shape, generator=g, device="cuda", dtype=dtype),
            "v": torch.randn(shape, generator=g, device="cuda", dtype=dtype),
            "table": table.cuda(), "held": whole(held), "context": whole(context), "refs": refs.cuda()}


def prepare(case, seed):
    if case["op"] in ("process", "constrain"):
        s = _round_state(case, seed)
        s["op"] = case["op"]
        return s
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "pages":
        n = case["B"] * case["children"]
        per = (case["context"] + case["room"] + case["page"] - 1) // case["page"]
        s = _cache(case, g, case["B"] + n, case["layers"], n * (2 + case["room"] // case["page"]) + 5,
                   case["room"])
        assert s["table"].shape[1] >= per
        s["src"] = torch.arange(case["B"], device="cuda", dtype=torch.int32).repeat_interleave(case["children"])
        s["dst"] = torch.randperm(n, generator=g, device="cuda").to(torch.int32) + case["B"]
        s["room"] = torch.full((n,), case["room"], dtype=torch.int32, device="cuda")
        s["op"] = "pages"
        return s
    s = _round(case, g, 32000)
    s["op"] = case["op"]
    most = max(case["K"] + 1, case["N"])
    if case["op"] == "attend":
        s |= _cache(case, g, case["B"], 0, 7, most)
        width = (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        # q, k and v of the new rows come as the slices of one projection
        qkv = torch.randn(s["total_rows"], width, generator=g, device="cuda", dtype=TYPES[case["dtype"]])
        q, k, v = qkv.split([case["heads"] * case["dim"]] + 2 * [case["kv_heads"] * case["dim"]], 1)
        s["q"] = q.unflatten(1, (case["heads"], case["dim"]))
        s["k_rows"] = k.unflatten(1, (case["kv_heads"], case["dim"]))
        s["v_rows"] = v.unflatten(1, (case["kv_heads"], case["dim"]))
        s["max_context"] = case["context"]
        return s
    s |= _cache(case, g, case["B"], case["layers"], 7, most)
    # What verification gave: a node, and the tokens up to it.
    lay = _layout(s)
    local = torch.arange(s["total_rows"], device="cuda") - lay["start"][lay["seq"]]
    size = (lay["start"].diff(append=lay["start"].new_tensor([s["total_rows"]])))
    best = (_rand(g, case["B"]) * size).floor().long().minimum(size - 1)
    s["best_node"] = best.to(torch.int32)
    s["accept_len"] = lay["anc"].sum(1)[lay["start"] + best].to(torch.int32)
    s["next_context"] = torch.zeros_like(s["context"])
    assert int(local.max()) < most
    return s


# ----------------------------------------------------------------------------- plain forms


def _layout(s):
    """For every packed row: its sequence, its parent row (-1: a first row), the token its node
    drafted (-1: none) and which rows are on its path; for every sequence its first row."""
    rows, K, N, kind = s["total_rows"], s["K"], s["N"], s["kind"]
    dev = "cuda"
    r = torch.arange(rows, device=dev)
    if kind == "routed":
        start = s["row_offsets"][:-1].long()
        seq = torch.searchsorted(s["row_offsets"][1:].long(), r, right=True)
        tree = s["choice"].long()[seq] == 1
    else:
        each = K + 1 if kind == "chain" else N
        start = torch.arange(0, rows, each, device=dev)
        seq = r // each
        tree = torch.full((rows,), kind == "tree", device=dev)
    i = r - start[seq]
    chain_parent = i - 1
    chain_token = s["draft"].long()[seq, (i - 1).clamp(0, K - 1)] if kind != "tree" and K else torch.full_like(i, -1)
    if kind != "chain":
        node = i.clamp_max(N - 1)
        tree_parent = s["parent"].long()[seq, node]
        tree_token = s["d2t"].long()[s["draft_ids"].long()[seq, node]]
    else:
        tree_parent, tree_token = chain_parent, chain_token
    par = torch.where(i == 0, torch.full_like(i, -1), start[seq] + torch.where(tree, tree_parent, chain_parent))
    tok = torch.where(i == 0, torch.full_like(i, -1), torch.where(tree, tree_token, chain_token))
    # ancestor-or-self of every row among its sequence's rows, by local index
    most = max(K + 1, N)
    up = torch.zeros(rows, most, device=dev)
    up[r, i] = 1
    up[r, (par - start[seq]).clamp_min(0)] += (par >= 0).float()
    grid = torch.zeros(start.numel(), most, most, device=dev)
    grid[seq, i] = up
    return {"seq": seq, "par": par, "tok": tok, "i": i, "start": start,
            "anc": torch.linalg.matrix_power(grid, most)[seq, i] > 0}


def _processed(s, lay):
    """The processed logits in 32 bits."""
    logits, seq, rows = s["logits"], lay["seq"], s["total_rows"]
    V = logits.shape[1]
    word = s["history"][s["slot"].long()].int() & 0xffff
    count = (word & 0x7fff).float()[seq]
    # every row's path tokens: the path's nodes without the first row
    local_tok = torch.full((lay["start"].numel(), lay["anc"].shape[1]), -1, device=seq.device)
    local_tok[seq, lay["i"]] = lay["tok"]
    token = local_tok[seq]
    count.scatter_add_(1, token.clamp_min(0), (lay["anc"] & (token >= 0)).float())
    put_out = count > 0
    seen = put_out | (word >= 0x8000)[seq]
    rep, freq, pres = (s["penalties"][:, k][seq][:, None] for k in range(3))
    x = logits.float()
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * count - pres * put_out.float()
    owner = torch.searchsorted(s["bias_offsets"][1:].long(),
                               torch.arange(s["bias_ids"].numel(), device=seq.device), right=True)
    bias = torch.zeros(s["slot"].numel(), V, device=seq.device)
    bias[owner, s["bias_ids"].long()] = s["bias_values"]
    x = x + bias[seq]
    bit = torch.arange(32, device=seq.device, dtype=torch.int32)
    allowed = ((s["allow"][:, :, None] >> bit) & 1).view(rows, -1)[:, :V] != 0
    return torch.where(allowed, x, x.new_full((), -math.inf))


def _accepted(s, lay, t):
    """Acceptance length, bonus token and best node of every sequence from the rows' tokens t."""
    seq, par, tok, i = lay["seq"], lay["par"], lay["tok"], lay["i"]
    match = (par < 0) | ((tok >= 0) & (tok == t[par.clamp_min(0)]))
    local = torch.zeros(lay["start"].numel(), lay["anc"].shape[1], dtype=torch.bool, device=seq.device)
    local[seq, i] = match
    ok = (local[seq] | ~lay["anc"]).all(1)
    depth = lay["anc"].sum(1)
    key = torch.where(ok, depth * 65536 + 65535 - i, torch.zeros_like(i))
    top = torch.zeros(lay["start"].numel(), dtype=key.dtype, device=seq.device).scatter_reduce_(0, seq, key, "amax")
    best = 65535 - top % 65536
    row = lay["start"] + best
    return top // 65536, t[row], best, row


def _plain_constrain(s):
    lay = _layout(s)
    x = _processed(s, lay)
    top = x.amax(1, keepdim=True)
    V = x.shape[1]
    place = torch.arange(V, device=x.device, dtype=torch.int32)
    t = torch.where(x == top, place, place.new_full((), V)).amin(1).long()
    t = torch.where(top[:, 0] == -math.inf, torch.full_like(t, -1), t)
    al, bonus, best, row = _accepted(s, lay, t)
    # the accepted tokens enter the history: those on the best row's path, then the bonus token
    path_tok = torch.full((al.numel(), lay["anc"].shape[1]), -1, device=x.device)
    path_tok[lay["seq"], lay["i"]] = lay["tok"]
    new = torch.cat([torch.where(lay["anc"][row], path_tok, torch.full_like(path_tok, -1)), bonus[:, None]], 1)
    at = s["slot"].long()
    word = s["history"][at].int() & 0xffff
    count = (word & 0x7fff).scatter_add(1, new.clamp_min(0), (new >= 0).int()).clamp_max(0x7fff)
    s["history"][at] = (count | (word & 0x8000)).to(torch.int16)
    return {"accept_len": al.int(), "bonus": bonus.int(), "best_node": best.int(), "row_argmax": t.int(),
            "history": s["history"]}


def _place(s, position, seq):
    """(page, row within it) of every cache position."""
    page = s["k"].shape[-2]
    return s["table"].long()[seq, position // page], position % page


def _plain_attend(s):
    lay = _layout(s)
    seq, i = lay["seq"], lay["i"]
    context = s["context"].long()
    page, off = _place(s, context[seq] + i, seq)
    s["k"][page, :, off] = s["k_rows"]
    s["v"][page, :, off] = s["v_rows"]
    B, most = lay["start"].numel(), lay["anc"].shape[1]
    Hkv, ps, D = s["k"].shape[1:]
    group = s["q"].shape[1] // Hkv
    table = s["table"].long().clamp_min(0)
    cap = table.shape[1] * ps
    keys = s["k"][table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, cap, D)
    vals = s["v"][table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, cap, D)
    q = torch.zeros(B, most, Hkv, group, D, device=keys.device)
    q[seq, i] = s["q"].float().unflatten(1, (Hkv, group))
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, most * group, D)
    score = torch.matmul(q, keys.transpose(2, 3).contiguous()) * D ** -0.5
    j = torch.arange(cap, device=keys.device) - context[:, None]  # a key's place among the round's rows
    anc = torch.zeros(B, most, most, dtype=torch.bool, device=keys.device)
    anc[seq, i] = lay["anc"]
    mine = anc.gather(2, j.clamp(0, most - 1)[:, None].expand(B, most, cap))
    see = (j < 0)[:, None] | ((j < most)[:, None] & mine)
    score = score.view(B, Hkv, most, group, cap).masked_fill_(~see[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, most * group, cap), vals).view(B, Hkv, most, group, D)
    out = out / total.clamp_min(1e-30)
    out = out.permute(0, 2, 1, 3, 4)[seq, i].flatten(1, 2).to(s["q"].dtype)
    return {"out": out, "k": s["k"], "v": s["v"]}


def _plain_compact(s):
    lay = _layout(s)
    al = s["accept_len"].long()
    path = lay["anc"][lay["start"] + s["best_node"].long()]
    src = torch.argsort((~path).int(), dim=1, stable=True)  # the path's nodes first, in order
    dst = torch.arange(path.shape[1], device=path.device).expand_as(src)
    b, _ = torch.nonzero(moves := dst < al[:, None], as_tuple=True)
    base = s["context"].long()[b]
    from_page, from_row = _place(s, base + src[moves], b)
    to_page, to_row = _place(s, base + dst[moves], b)
    s["k"][:, to_page, :, to_row] = s["k"][:, from_page, :, from_row]
    s["v"][:, to_page, :, to_row] = s["v"][:, from_page, :, from_row]
    s["next_context"].copy_(s["context"] + s["accept_len"])
    return {"k": s["k"], "v": s["v"], "context": s["next_context"]}


def _plain_pages(s):
    table, held, context, refs = s["table"], s["held"], s["context"], s["refs"]
    page = s["k"].shape[-2]
    src, dst = s["src"].long(), s["dst"].long()
    # fork: full pages shared, a partly filled last page copied into the lowest free ones
    c = context.long()[src]
    full, part = c // page, c % page
    need = (part > 0).long()
    free = torch.nonzero(refs == 0)[:, 0]
    before = need.cumsum(0) - need
    forked = (need.cumsum(0) <= free.numel()) | (need == 0)
    column = torch.arange(table.shape[1], device=table.device)
    row = torch.where(column < full[:, None], table[src], table.new_full((), -1))
    refs.index_add_(0, row[row >= 0].long(), torch.ones_like(row[row >= 0]))
    fresh = free[before.clamp_max(free.numel() - 1)]
    entry = torch.nonzero(need, as_tuple=True)[0]
    old = table.long()[src[entry], full[entry]]
    live = torch.arange(page, device=table.device) < part[entry, None]
    e, o = torch.nonzero(live, as_tuple=True)
    s["k"][:, fresh[entry][e], :, o] = s["k"][:, old[e], :, o]
    s["v"][:, fresh[entry][e], :, o] = s["v"][:, old[e], :, o]
    row[entry, full[entry]] = fresh[entry].int()
    refs[fresh[entry]] = 1
    table[dst], held[dst], context[dst] = row, (full + need).int(), c.int()
    forked_table = row.clone()
    # room for the next rows: the lowest free pages again
    want = (c + s["room"] + page - 1) // page
    need = (want - held[dst]).clamp_min(0).long()
    free = torch.nonzero(refs == 0)[:, 0]
    before = need.cumsum(0) - need
    given = (need.cumsum(0) <= free.numel()) | (need == 0)
    inside = (column >= held[dst][:, None]) & (column < (held[dst] + need)[:, None])
    rank = (before[:, None] + column - held[dst][:, None])[inside]
    row[inside] = free[rank].int()
    refs[free[rank]] = 1
    roomy_table = row.clone()
    # and the children freed
    gone = row[row >= 0].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[dst], held[dst], context[dst] = -1, 0, 0
    return {"forked": forked.int(), "given": given.int(), "fork_table": forked_table, "room_table": roomy_table,
            "k": s["k"], "v": s["v"], "table": table, "held": held, "context": context, "refs": refs}


def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op == "process":
        return _processed(s, _layout(s)).to(s["logits"].dtype)
    if op == "constrain":
        return _plain_constrain(s)
    if op == "attend":
        return _plain_attend(s)
    if op == "compact":
        return _plain_compact(s)
    return _plain_pages(s)


# ----------------------------------------------------------------------------- the framework's calls


def _own(s):
    import drafter_routing_verification_amd as wf

    if s["op"] == "pages":
        cache = wf.PageCache(s["k"], s["v"], s["table"], s["held"], s["context"], s["refs"])
        forked = wf.cache_fork(cache, s["src"], s["dst"])
        fork_table = s["table"][s["dst"]]
        given = wf.cache_reserve(cache, s["room"], seqs=s["dst"])
        room_table = s["table"][s["dst"]]
        wf.cache_free(cache, s["dst"])
        return {"forked": forked, "given": given, "fork_table": fork_table, "room_table": room_table,
                "k": s["k"], "v": s["v"], "table": s["table"], "held": s["held"], "context": s["context"],
                "refs": s["refs"]}
    if s["kind"] == "chain":
        rows = wf.chain_rows(s["draft"])
    elif s["kind"] == "tree":
        rows = wf.tree_rows(s["parent"], s["draft_ids"], s["d2t"])
    else:
        rows = wf.routed_rows(s["row_offsets"], s["total_rows"], s["choice"], s["draft"], s["parent"],
                              s["draft_ids"], s["d2t"])
    if s["op"] in ("process", "constrain"):
        rules = wf.LogitRules(history=s["history"], slot=s["slot"], penalties=s["penalties"],
                              bias=(s["bias_offsets"], s["bias_ids"], s["bias_values"]), allow=s["allow"])
        if s["op"] == "process":
            return wf.process_logits(s["logits"], rows, rules, dtype=s["logits"].dtype)
        al, bonus, best, t = wf.verify_constrained(s["logits"], rows, rules)
        wf.history_update(s["history"], rows, al, best, bonus, slot=s["slot"])
        return {"accept_len": al, "bonus": bonus, "best_node": best, "row_argmax": t, "history": s["history"]}
    cache = wf.PageCache(s["k"], s["v"], s["table"], s["held"], s["context"], s["refs"])
    if s["op"] == "attend":
        wf.cache_append(cache, rows, s["k_rows"], s["v_rows"])
        out = wf.attend(s["q"], rows, cache, max_context=s["max_context"])
        return {"out": out, "k": s["k"], "v": s["v"]}
    wf.cache_compact(cache, rows, s["accept_len"], s["best_node"], next_context=s["next_context"])
    return {"k": s["k"], "v": s["v"], "context": s["next_context"]}


# ----------------------------------------------------------------------------- work


def work(case):
    """Each input read once, each output written once."""
    op, B = case["op"], case["B"]
    size = {"f32": 4, "bf16": 2}[case["dtype"]]
    if op == "pages":
        n, page = B * case["children"], case["page"]
        row = case["layers"] * 2 * case["kv_heads"] * case["dim"] * size
        part = sum(c % page for c in _contexts(case)) * case["children"]
        pages = sum(-(-(c + case["room"]) // page) for c in _contexts(case)) * case["children"]
        return {"bytes": 2 * part * row + 24 * pages + 24 * n, "flops": 0}
    K, N, kind = case["K"], case["N"], case["rows"]
    sizes = ([N if c else K + 1 for c in _choices(case)] if kind == "routed"
             else [K + 1 if kind == "chain" else N] * B)
    rows = sum(sizes)
    if op in ("process", "constrain"):
        V = case["V"]
        read = rows * V * size + B * V * 2 + rows * V / 8
        return {"bytes": read + (rows * V * size if op == "process" else 0), "flops": 4.0 * rows * V}
    context = _contexts(case)
    if op == "attend":
        kv = 2 * case["kv_heads"] * case["dim"] * size
        q = case["heads"] * case["dim"] * size
        keys = sum(c + n for c, n in zip(context, sizes))
        flops = sum(4.0 * n * case["heads"] * case["dim"] * (c + n / 2) for c, n in zip(context, sizes))
        return {"bytes": keys * kv + 2 * rows * q + rows * kv, "flops": flops}
    # a random node of such a tree is about a fifth of log(N) * 2 edges deep; a chain moves nothing
    row = case["layers"] * 2 * case["kv_heads"] * case["dim"] * size
    moved = sum(math.log(max(n, 1)) for n, c in zip(sizes, _choices(case)) if kind == "tree" or (kind == "routed" and c))
    return {"bytes": 2 * moved * row + 4 * (rows + 4 * B), "flops": 0}


# ----------------------------------------------------------------------------- in 64 bits


def _paths(s):
    """Per sequence: its first row, its rows and, for each, (token of its node, rows of its path)."""
    found = []
    host = {k: s[k].cpu().tolist() for k in ("parent", "draft_ids", "d2t", "draft", "row_offsets", "choice") if k in s}
    B = len(host["draft"] if "draft" in host else host["parent"])
    at = 0
    for b in range(B):
        tree = s["kind"] == "tree" or (s["kind"] == "routed" and host["choice"][b] == 1)
        tokens, paths = [-1], [[0]]
        for u in range(1, s["N"] if tree else s["K"] + 1):
            p = host["parent"][b][u] if tree else u - 1
            tokens.append(host["d2t"][host["draft_ids"][b][u]] if tree else host["draft"][b][u - 1])
            paths.append(paths[p] + [u])
        found.append((at, tokens, paths))
        at += len(tokens)
    return found


def _exact_rows(s, b, at, tokens, paths):
    """The processed logits of one sequence in 64 bits."""
    n, V = len(tokens), s["logits"].shape[1]
    word = s["history"][int(s["slot"][b])].long() % 65536
    rep, freq, pres = (float(p) for p in s["penalties"][b].double().cpu())
    times = (word % 32768).double().repeat(n, 1)
    place = [(u, tokens[a]) for u in range(n) for a in paths[u] if a]
    if place:
        u, v = torch.tensor(place, device="cuda").T
        times.index_put_((u, v), torch.ones(len(place), dtype=torch.float64, device="cuda"), accumulate=True)
    x = s["logits"][at:at + n].double()
    hit = (times > 0) | (word >= 32768)
    x = torch.where(hit, torch.where(x > 0, x / rep, x * rep), x) - freq * times - pres * (times > 0).double()
    lo, hi = int(s["bias_offsets"][b]), int(s["bias_offsets"][b + 1])
    x[:, s["bias_ids"][lo:hi].long()] += s["bias_values"][lo:hi].double()
    v = torch.arange(V, device="cuda")
    allowed = (s["allow"][at:at + n].long()[:, v // 32] >> (v % 32)) % 2 == 1
    x[~allowed] = -math.inf
    return x


def _exact_attend(s):
    context, table = s["context"].cpu().tolist(), s["table"].cpu()
    ps, D, Hkv = s["k"].shape[2], s["k"].shape[3], s["k"].shape[1]
    group = s["q"].shape[1] // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (at, tokens, paths) in enumerate(_paths(s)):
        n, c = len(tokens), context[b]
        spots = [(int(table[b, (c + u) // ps]), (c + u) % ps) for u in range(n)]
        for u, (pg, o) in enumerate(spots):
            s["k"][pg, :, o], s["v"][pg, :, o] = s["k_rows"][at + u], s["v_rows"][at + u]
        used = table[b, :(c + n + ps - 1) // ps].long().cuda()
        see = torch.zeros(n, c + n, dtype=torch.bool)
        see[:, :c] = True
        for u, path in enumerate(paths):
            see[u, [c + a for a in path]] = True
        see = see.cuda()
        for h in range(Hkv):
            keys = s["k"][used, h].double().reshape(-1, D)[:c + n]
            vals = s["v"][used, h].double().reshape(-1, D)[:c + n]
            for k in range(h * group, (h + 1) * group):
                w = s["q"][at:at + n, k].double() @ keys.T / math.sqrt(D)
                out[at:at + n, k] = torch.softmax(w.masked_fill(~see, -math.inf), 1) @ vals
    return {"out": out, "k": s["k"].double(), "v": s["v"].double()}


def _exact_compact(s):
    context, table = s["context"].cpu().tolist(), s["table"].cpu()
    ps = s["k"].shape[3]
    al, best = s["accept_len"].cpu().tolist(), s["best_node"].cpu().tolist()
    for b, (_, _, paths) in enumerate(_paths(s)):
        for j, u in enumerate(paths[best[b]]):
            f, t = context[b] + u, context[b] + j
            if f != t:
                for x in (s["k"], s["v"]):
                    x[:, int(table[b, t // ps]), :, t % ps] = x[:, int(table[b, f // ps]), :, f % ps]
    return {"k": s["k"].double(), "v": s["v"].double(),
            "context": torch.tensor([c + n for c, n in zip(context, al)], dtype=torch.int32)}


def _exact_pages(s):
    table, held, context, refs = (s[k].cpu().tolist() for k in ("table", "held", "context", "refs"))
    page = s["k"].shape[3]
    pairs = list(zip(s["src"].cpu().tolist(), s["dst"].cpu().tolist()))

    def lowest():
        p = refs.index(0)
        refs[p] = 1
        return p

    for a, d in pairs:
        full = context[a] // page
        for n in range(full):
            table[d][n] = table[a][n]
            refs[table[a][n]] += 1
        if context[a] % page:
            table[d][full] = lowest()
            for x in (s["k"], s["v"]):
                x[:, table[d][full], :, :context[a] % page] = x[:, table[a][full], :, :context[a] % page]
        held[d], context[d] = -(-context[a] // page), context[a]
    fork_table = [list(table[d]) for _, d in pairs]
    for (_, d), room in zip(pairs, s["room"].cpu().tolist()):
        while held[d] * page < context[d] + room:
            table[d][held[d]] = lowest()
            held[d] += 1
    room_table = [list(table[d]) for _, d in pairs]
    for _, d in pairs:
        for n in range(held[d]):
            refs[table[d][n]] -= 1
            table[d][n] = -1
        held[d] = context[d] = 0
    whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    ones = whole([1] * len(pairs))
    return {"forked": ones, "given": ones, "fork_table": whole(fork_table), "room_table": whole(room_table),
            "k": s["k"].double(), "v": s["v"].double(), "table": whole(table), "held": whole(held),
            "context": whole(context), "refs": whole(refs)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "compact":
        return _exact_compact(s)
    if case["op"] == "pages":
        return _exact_pages(s)
    if case["op"] == "process":
        return torch.cat([_exact_rows(s, b, *p) for b, p in enumerate(_paths(s))])
    al, bonus, best, t = [], [], [], []
    for b, (at, tokens, paths) in enumerate(_paths(s)):
        x = _exact_rows(s, b, at, tokens, paths)
        top = x.max(1, keepdim=True).values
        v = torch.arange(x.shape[1], device="cuda")
        low = torch.where((x == top) & (top > -math.inf), v, x.shape[1]).min(1).values.cpu().tolist()
        low = [u if u < x.shape[1] else -1 for u in low]
        good = [all(tokens[c] >= 0 and tokens[c] == low[a] for a, c in zip(p, p[1:])) for p in paths]
        u = max((u for u in range(len(paths)) if good[u]), key=lambda u: (len(paths[u]), -u))
        word = s["history"][int(s["slot"][b])]
        for new in [tokens[a] for a in paths[u][1:]] + [low[u]]:
            if new >= 0 and int(word[new]) % 32768 < 32767:
                word[new] += 1
        al.append(len(paths[u]))
        bonus.append(low[u])
        best.append(u)
        t += low
    whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"accept_len": whole(al), "bonus": whole(bonus), "best_node": whole(best), "row_argmax": whole(t),
            "history": s["history"]}
