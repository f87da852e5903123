"""Operators of a decoding step around the rounds that are measured here, in plain form and as the
framework's calls: rotary positions, a paged cache held in 8 bits, the attention over it, and the log
probabilities of tokens.

The rows of a round are chains of K + 1 rows or trees of N rows; row r of sequence b has the position
context[b] + depth(r), depth being the edges between it and the first row.

  rotate    queries and keys turned by their positions.  For pair i (elements i and i + pairs, or 2 i
            and 2 i + 1) with angle a = position * frequency[i] and magnitude m:
              x' = m (x cos a - y sin a),  y' = m (y cos a + x sin a)
  append    keys and values of the rows written in 8 bits, and the blocks that hold them read back.
            A block of positions of one head has one exponent e, the least with
            max |x| <= 448 * 2^e (from -100 to 119) over its committed and new values;
            it holds c = e4m3(x / 2^e), which stands for c * 2^e
  read      the committed positions of whole sequences read back (zeros behind them)
  attend    out[r, h] = sum_j softmax_j(scale q[r, h] . k[j]) v[j] over the committed positions and
            those of the round's rows on r's path, k and v as the cache's 8 bits stand for them
  logprobs  log softmax of given tokens, entropy, and the most likely tokens, of selected rows
"""

import math

import torch

own = False

HEADS, KV_HEADS, DIM, PAGE = 32, 8, 128, 16
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LEAST, MOST = -100, 119  # exponents of a block


def listed():
    heads = {"heads": HEADS, "kv_heads": KV_HEADS, "dim": DIM}
    cache = {"kv_heads": KV_HEADS, "dim": DIM}
    return [
        # One new token of one sequence: latency.
        {"name": "rotate-token-bf16", "op": "rotate", "rows": "chain", "B": 1, "K": 0, "N": 0, "context": 5000,
         "pairs": 64, "layout": "half", "dtype": "bf16", **heads},
        # A batch of trees, half of each head turned, pairs side by side, far positions.
        {"name": "rotate-trees-f32", "op": "rotate", "rows": "tree", "B": 64, "K": 0, "N": 61, "context": 131000,
         "pairs": 32, "layout": "interleaved", "dtype": "f32", **heads},
        # Parts of prompts, 1,024 rows a sequence: bandwidth.
        {"name": "rotate-prompts-bf16", "op": "rotate", "rows": "chain", "B": 32, "K": 1023, "N": 0, "context": 4096,
         "pairs": 64, "layout": "half", "dtype": "bf16", **heads},
        # A serving batch's verified chains written into blocks that hold committed positions: latency.
        {"name": "append-chains-bf16", "op": "append", "rows": "chain", "B": 64, "K": 16, "N": 0, "context": 4096,
         "page": PAGE, "block": 16, "dtype": "bf16", **cache},
        # Parts of prompts written, a scale for every position.
        {"name": "append-prompts-bf16", "op": "append", "rows": "chain", "B": 32, "K": 1023, "N": 0,
         "context": 2000, "page": 64, "block": 1, "dtype": "bf16", **cache},
        # Two long sequences read back whole.
        {"name": "read-long-bf16", "op": "read", "B": 2, "context": 131000, "page": PAGE, "block": 16,
         "dtype": "bf16", **cache},
        # One new token of one sequence with a short context: latency.
        {"name": "attend-token-bf16", "op": "attend", "rows": "chain", "B": 1, "K": 0, "N": 0, "context": 1000,
         "page": PAGE, "block": 1, "dtype": "bf16", **heads},
        # One new token each of a ragged serving batch.
        {"name": "attend-batch-bf16", "op": "attend", "rows": "chain", "B": 64, "K": 0, "N": 0, "context": 8192,
         "page": PAGE, "block": 16, "dtype": "bf16", **heads},
        # Trees being verified.
        {"name": "attend-trees-bf16", "op": "attend", "rows": "tree", "B": 8, "K": 0, "N": 61, "context": 4096,
         "page": PAGE, "block": 1, "dtype": "bf16", **heads},
        # Two chains at the end of very long contexts.
        {"name": "attend-long-bf16", "op": "attend", "rows": "chain", "B": 2, "K": 16, "N": 0, "context": 131000,
         "page": 64, "block": 32, "dtype": "bf16", **heads},
        # The sampled rows of a few sequences over a small vocabulary, some under a grammar: latency.
        {"name": "logprobs-step-f32", "op": "logprobs", "n": 4, "every": 17, "V": 32000, "given": 1, "top": 5,
         "dtype": "f32"},
        # Every row of a batch of chains: bandwidth.
        {"name": "logprobs-chains-bf16", "op": "logprobs", "n": 4352, "every": 1, "V": 151936, "given": 2,
         "top": 20, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "read", "attend", "attend", "logprobs"])
    case = {"op": op, "dtype": rng.choice(["f32", "bf16", "bf16"])}
    size = 4 if case["dtype"] == "f32" else 2
    if op == "logprobs":
        case["V"] = _log(rng, 999, 151936)
        case["n"] = _log(rng, 1, max(1, min(4352, 4352 * 151936 * 2 // (case["V"] * size))))
        case["every"] = rng.choice([1, 1, 3, 17]) if case["n"] <= 256 else 1
        case["given"], case["top"] = rng.randint(0, 3), rng.randint(0, 32)
        return case
    case["kv_heads"] = rng.choice([1, 2, 4, 8])
    case["dim"] = rng.choice([64, 128])
    if op != "read":
        case["rows"] = rng.choice(["chain", "tree"])
        long = op != "attend" and rng.random() < 0.3
        case["K"] = (rng.randint(100, 1023) if long else rng.randint(0, 24)) if case["rows"] == "chain" else 0
        case["N"] = rng.randint(1, 64) if case["rows"] == "tree" else 0
    deepest = max(case["K"] + 1, case["N"]) if op != "read" else 1
    if op in ("rotate", "attend"):
        case["heads"] = case["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
    if op == "rotate":
        case["pairs"] = rng.choice([case["dim"] // 2, case["dim"] // 4, rng.randint(1, case["dim"] // 2)])
        case["layout"] = rng.choice(["half", "interleaved"])
        width = (case["heads"] + case["kv_heads"]) * case["dim"]
        case["B"] = _log(rng, 1, max(1, min(64, 32 * 1024 * 5120 * 2 // (deepest * width * size))))
        case["context"] = _log(rng, 1, 1000000)
        return case
    case["page"] = rng.choice([16, 32, 64])
    case["block"] = rng.choice([1, 16, case["page"], rng.choice([2, 4, 8])])
    if op == "append":
        case["B"] = _log(rng, 1, min(64, 32 * 1024 // deepest))
        case["context"] = _log(rng, 1, 2000)
    elif op == "read":
        case["B"] = _log(rng, 1, 64)
        width = case["kv_heads"] * case["dim"] * size
        case["context"] = _log(rng, 1, 2 * 131000 * 2048 // (case["B"] * width))
    else:
        case["B"] = _log(rng, 1, 96)
        # keys x heads x dims stay under the largest listed case's, and scores under its as well
        room = min(131000 * 2 * 1024 // (case["B"] * case["kv_heads"] * case["dim"] * 2),
                   131000 * 2 * 17 * 32 // (case["B"] * deepest * case["heads"]))
        case["context"] = _log(rng, 1, max(2, min(131000, room)))
    return case


# ----------------------------------------------------------------------------- inputs


def _contexts(case):
    """Committed lengths: evenly spread over the upper half, the longest first."""
    B, top = case["B"], case["context"]
    return [max(0, top - (b * (top // 2)) // B) for b in range(B)]


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _round(case, g, s):
    """The round's drafts, as a verify call takes them."""
    B, K, N = case["B"], case["K"], case["N"]
    s |= {"kind": case["rows"], "K": K, "N": N, "total_rows": B * (K + 1 if case["rows"] == "chain" else N)}
    if case["rows"] == "chain":
        s["draft"] = torch.randint(0, 32000, (B, K), generator=g, device="cuda", dtype=torch.int32)
    else:  # random trees: each node hangs under one of the ten before it
        u = torch.arange(N, device="cuda")
        low = (u - 10).clamp_min(0)
        parent = low + (_rand(g, B, N) * (u - low)).floor().long().minimum((u - low - 1).clamp_min(0))
        s["parent"] = parent.to(torch.int32)


def _vectors(g, rows, heads, dim, dtype):
    """Projected vectors: some channels of a head are larger than others, and so are some rows."""
    x = torch.randn(rows, heads, dim, generator=g, device="cuda")
    channel = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device="cuda"))
    row = torch.exp(0.3 * torch.randn(rows, 1, 1, generator=g, device="cuda"))
    return (x * channel * row).to(dtype)


def _cache(case, g, s, room):
    """One layer's page pool, the sequences' pages scattered over it."""
    page, heads, dim, block = case["page"], case["kv_heads"], case["dim"], case["block"]
    context = _contexts(case)
    held = [(c + room + page - 1) // page for c in context]
    P = sum(held) + 7
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    most = (case["context"] + room + page - 1) // page
    table = torch.full((case["B"], most), -1, dtype=torch.int32)
    order_host, at = order.cpu(), 0
    for b, n in enumerate(held):
        table[b, :n] = order_host[at:at + n]
        at += n
    refs = torch.zeros(P, dtype=torch.int32)
    refs[order_host[:at].long()] = 1
    for name in ("k", "v"):
        x = _vectors(g, P * page, heads, dim, torch.bfloat16).float().view(P, page, heads, dim).transpose(1, 2)
        x = x.contiguous().view(P, heads, page // block, block, dim)
        e = _exponent(x.abs().amax((-1, -2)))
        s[name] = (x * _power(-e)[..., None, None]).to(torch.float8_e4m3fn).view(P, heads, page, dim)
        s[name + "_scale"] = (e + 127).to(torch.uint8)
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s |= {"table": table.cuda(), "held": whole(held), "context": whole(context), "refs": refs.cuda(), "block": block}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], TYPES[case["dtype"]]
    s = {"op": op}
    if op == "logprobs":
        n, every, V = case["n"], case["every"], case["V"]
        per = 16 // dtype.itemsize
        logits = torch.zeros(n * every, (V + per - 1) // per * per, dtype=dtype, device="cuda")[:, :V]
        logits.normal_(generator=g).mul_(2.5)
        # a likely token in each row, sharply so in some
        lead = torch.randint(0, V, (n * every, 1), generator=g, device="cuda")
        logits.scatter_(1, lead, (10 + 12 * _rand(g, n * every, 1)).to(dtype))
        if case["dtype"] == "f32":  # processed logits: a grammar leaves every second row one token in sixteen
            masked = (_rand(g, n * every, V) < 15 / 16) & (torch.arange(n * every, device="cuda") % 2 == 1)[:, None]
            logits.masked_fill_(masked, -math.inf)
        s |= {"logits": logits, "top": case["top"]}
        s["rows"] = None
        if every > 1:
            s["rows"] = (torch.arange(n, device="cuda") * every + torch.randint(0, every, (n,), generator=g, device="cuda")).int()
        tokens = torch.randint(0, V, (n, case["given"]), generator=g, device="cuda")
        picked = lead if s["rows"] is None else lead[s["rows"].long()]
        if case["given"]:
            tokens[:, :1] = torch.where(_rand(g, n, 1) < 0.7, picked, tokens[:, :1])
        s["tokens"] = tokens.int()
        return s
    if op == "read":
        _cache(case, g, s, 1)
        s |= {"count": case["context"], "pending": 0, "dtype": dtype}
        return s
    _round(case, g, s)
    rows, kv, dim = s["total_rows"], case["kv_heads"], case["dim"]
    if op == "append":
        _cache(case, g, s, max(case["K"] + 1, case["N"]))
        s["k_rows"], s["v_rows"] = (_vectors(g, rows, kv, dim, dtype) for _ in range(2))
        s["first"] = (s["context"] // s["block"] * s["block"]).int()
        s["pending"] = max(case["K"] + 1, case["N"])
        s["count"] = s["pending"] + case["block"] - 1
        s["dtype"] = dtype
        return s
    # q, k and v of the new rows come as the slices of one projection
    qkv = _vectors(g, rows, case["heads"] + 2 * kv, dim, dtype)
    s["q"], s["k_rows"] = qkv[:, :case["heads"]], qkv[:, case["heads"]:case["heads"] + kv]
    if op == "rotate":
        s["context"] = torch.tensor(_contexts(case), dtype=torch.int32, device="cuda")
        i = torch.arange(case["pairs"], dtype=torch.float64, device="cuda")
        s["frequency"] = 10000.0 ** (-i / case["pairs"])
        s |= {"layout": case["layout"], "magnitude": 1.0 if case["layout"] == "half" else 1.25}
        return s
    _cache(case, g, s, max(case["K"] + 1, case["N"]))
    s["max_context"] = case["context"]
    return s


# ----------------------------------------------------------------------------- plain forms


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, from LEAST to MOST."""
    part, e = torch.frexp(amax)  # amax = part * 2^e, part in [0.5, 1)
    e = torch.where(part <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, torch.full_like(e, LEAST)).clamp(LEAST, MOST)


def _power(e):
    """2^e in 32 bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _layout(s):
    """For every row its sequence, its place there, and which of the sequence's rows are on its path."""
    each = s["K"] + 1 if s["kind"] == "chain" else s["N"]
    r = torch.arange(s["total_rows"], device="cuda")
    seq, i = r // each, r % each
    B = s["total_rows"] // each
    u = torch.arange(each, device="cuda")
    if s["kind"] == "chain":
        return seq, i, (u[:, None] >= u).expand(B, each, each)
    up = torch.eye(each, device="cuda").repeat(B, 1, 1)
    b = torch.arange(B, device="cuda")[:, None]
    up[b, u[1:], s["parent"].long()[:, 1:]] = 1
    return seq, i, torch.linalg.matrix_power(up, each) > 0


def _plain_rotate(s):
    seq, i, path = _layout(s)
    position = s["context"].long()[seq] + path[seq, i].sum(1) - 1
    angle = position.double()[:, None] * s["frequency"]
    pairs = s["frequency"].numel()
    c, d = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))

    def turned(x):
        x = x.float()
        part = x[..., :2 * pairs]
        if s["layout"] == "half":
            a, b = part[..., :pairs], part[..., pairs:]
            part = torch.cat([a * c - b * d, b * c + a * d], -1)
        else:
            a, b = part[..., 0::2], part[..., 1::2]
            part = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
        return torch.cat([part, x[..., 2 * pairs:]], -1).to(s["q"].dtype)

    return {"q": turned(s["q"]), "k": turned(s["k_rows"])}


def _values(s, name, page, row):
    """What the cache's bytes at (page, row of it) stand for, [..., heads, dim] in 32 bits."""
    e = s[name + "_scale"][page, :, row // s["block"]].int() - 127
    return s[name][page, :, row].float() * _power(e)[..., None]


def _plain_read(s):
    B, count, ps = s["table"].shape[0], s["count"], s["k"].shape[2]
    j = torch.arange(count, device="cuda") + (s["first"].long()[:, None] if "first" in s else 0)
    j = j.expand(B, count)
    there = (j < s["context"].long()[:, None] + s["pending"])[..., None, None]
    page = s["table"].long().gather(1, (j // ps).clamp_max(s["table"].shape[1] - 1)).clamp_min(0)
    return {name: torch.where(there, _values(s, name, page, j % ps), 0.0).to(s["dtype"])
            for name in ("k", "v")}


def _plain_append(s):
    seq, i, path = _layout(s)
    B, each = path.shape[:2]
    block, ps = s["block"], s["k"].shape[2]
    heads, dim = s["k_rows"].shape[1:]
    context = s["context"].long()[:, None]
    blocks = (each + 2 * block - 2) // block
    # the positions of every block that gets a row
    j = context // block * block + torch.arange(blocks * block, device="cuda")
    live, new = j < context + each, j >= context
    page = s["table"].long().gather(1, (j // ps).clamp_max(s["table"].shape[1] - 1)).clamp_min(0)
    row = (torch.arange(B, device="cuda")[:, None] * each + (j - context).clamp(0, each - 1))
    put = live & (j // block * block < context + each)
    for name in ("k", "v"):
        x = torch.where(new[..., None, None], s[name + "_rows"].float()[row], _values(s, name, page, j % ps))
        x = torch.where(live[..., None, None], x, 0.0)
        e = _exponent(x.abs().view(B, blocks, block, heads, dim).amax((2, 4)))
        e = e.repeat_interleave(block, 1)
        c = (x * _power(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s[name].view(torch.uint8)[page[put], :, j[put] % ps] = c.view(torch.uint8)[put]
        s[name + "_scale"][page[put], :, j[put] % ps // block] = (e[put] + 127).to(torch.uint8)
    return _plain_read(s)


def _plain_attend(s):
    seq, i, path = _layout(s)
    context = s["context"].long()
    B, most = path.shape[:2]
    heads, ps, D = s["k"].shape[1:]
    group = s["q"].shape[1] // heads
    table = s["table"].long().clamp_min(0)
    cap = table.shape[1] * ps

    def whole(name):
        e = s[name + "_scale"][table].int() - 127
        x = s[name][table].float() * _power(e).repeat_interleave(s["block"], 3)[..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, heads, cap, D)

    q = s["q"].float().view(B, most, heads, group, D).permute(0, 2, 1, 3, 4).reshape(B, heads, most * group, D)
    score = torch.matmul(q, whole("k").transpose(2, 3).contiguous()) * D ** -0.5
    j = torch.arange(cap, device="cuda") - context[:, None]  # a position's place among the round's rows
    mine = path.gather(2, j.clamp(0, most - 1)[:, None].expand(B, most, cap))
    see = (j < 0)[:, None] | ((j >= 0) & (j < most))[:, None] & mine
    score = score.view(B, heads, most, group, cap).masked_fill_(~see[:, None, :, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, heads, most * group, cap), whole("v")).view(B, heads, most, group, D) / total
    return out.permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(s["q"].dtype)


def _plain_logprobs(s):
    x = (s["logits"] if s["rows"] is None else s["logits"][s["rows"].long()]).float()
    V = x.shape[1]
    z = x - x.amax(1, keepdim=True)
    p = torch.exp(z)
    total = p.sum(1, keepdim=True)
    norm = torch.log(total)
    entropy = norm[:, 0] - (torch.where(p > 0, z, 0.0) * p).sum(1) / total[:, 0]
    given = z.gather(1, s["tokens"].long()) - norm
    # one number a token that falls with its logit, and among equal ones with its index
    bits = (x + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * 2**32 + (V - 1 - torch.arange(V, device="cuda"))
    ids = V - 1 - torch.topk(order, s["top"], dim=1).values % 2**32
    likely = z.gather(1, ids) - norm
    return {"logprob": given, "entropy": entropy,
            "top_tokens": torch.where(likely > -math.inf, ids, -1).int(), "top_logprobs": likely}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "rotate":
        return _plain_rotate(s)
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "read":
        return _plain_read(s)
    if s["op"] == "attend":
        return _plain_attend(s)
    return _plain_logprobs(s)


# ----------------------------------------------------------------------------- the framework's calls


def _own(s):
    import drafter_routing_verification_amd as wf

    op = s["op"]
    if op == "logprobs":
        logprob, entropy, ids, likely = wf.token_logprobs(s["logits"], s["tokens"], rows=s["rows"], top=s["top"])
        return {"logprob": logprob, "entropy": entropy, "top_tokens": ids, "top_logprobs": likely}
    if op != "read":
        rows = wf.chain_rows(s["draft"]) if s["kind"] == "chain" else wf.tree_rows(s["parent"])
    if op == "rotate":
        rotary = wf.Rotary(s["frequency"], layout=s["layout"], magnitude=s["magnitude"])
        q, k = wf.rotate(s["q"], s["k_rows"], rows, rotary, s["context"])
        return {"q": q, "k": k}
    cache = wf.PageCache8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["held"], s["context"],
                          s["refs"])
    if op == "attend":
        return wf.attend(s["q"], rows, cache, max_context=s["max_context"])
    if op == "append":
        wf.cache_append(cache, rows, s["k_rows"], s["v_rows"])
    k, v = wf.cache_read(cache, s["count"], first=s.get("first"), pending=s["pending"], dtype=s["dtype"])
    return {"k": k, "v": v}


# ----------------------------------------------------------------------------- work


def work(case):
    """Each input read once, each output written once."""
    op, size = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "logprobs":
        n, V = case["n"], case["V"]
        return {"bytes": n * (V * size + 8 * case["given"] + 8 * case["top"] + 4), "flops": 5.0 * n * V}
    width = case["kv_heads"] * case["dim"]
    scale = 2 * case["kv_heads"]  # bytes of a block's two exponents
    context = _contexts(case)
    if op == "read":
        held = sum(context)
        return {"bytes": 2 * held * width + scale * held / case["block"] + 2 * case["B"] * case["context"] * width * size,
                "flops": 2.0 * held * width}
    each = max(case["K"] + 1, case["N"])
    rows = case["B"] * each
    if op == "rotate":
        moved = rows * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * moved * case["dim"] * size, "flops": 6.0 * moved * case["pairs"]}
    if op == "append":
        block = case["block"]
        kept = sum(c % block for c in context)
        count = case["B"] * (each + block - 1)
        return {"bytes": 2 * width * (rows * (size + 1) + kept) + scale * (rows / block + case["B"])
                + 2 * width * (count + count * size), "flops": 8.0 * rows * width}
    keys = sum(c + each for c in context)
    flops = sum(4.0 * each * case["heads"] * case["dim"] * (c + each / 2) for c in context)
    return {"bytes": 2 * keys * width + scale * keys / case["block"] + 2 * rows * case["heads"] * case["dim"] * size,
            "flops": flops}


# ----------------------------------------------------------------------------- in 64 bits


def _depths(s, B, each):
    """Per sequence, the rows on each row's path, last first."""
    if s["kind"] == "chain":
        return [[list(range(u, -1, -1)) for u in range(each)]] * B
    found = []
    for parent in s["parent"].cpu().tolist():
        paths = [[0]]
        for u in range(1, each):
            paths.append([u] + paths[parent[u]])
        found.append(paths)
    return found


def _exact_rotate(s, B, each):
    paths = _depths(s, B, each)
    context = s["context"].cpu().tolist()
    place = torch.tensor([context[b] + len(p) - 1 for b in range(B) for p in paths[b]], dtype=torch.float64,
                         device="cuda")
    w = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device="cuda"),
                    place[:, None, None] * s["frequency"])
    pairs = s["frequency"].numel()
    out = {}
    for name, x in (("q", s["q"]), ("k", s["k_rows"])):
        x = x.double().clone()
        one, two = ((slice(0, pairs), slice(pairs, 2 * pairs)) if s["layout"] == "half" else
                    (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)))
        y = torch.complex(x[..., one], x[..., two]) * w
        x[..., one], x[..., two] = y.real, y.imag
        out[name] = x
    return out


def _two_to(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stands_for(s, name, pages):
    """The values of whole pages in 64 bits, [positions, heads, dim]."""
    bytes_, e = s[name][pages].double(), s[name + "_scale"][pages].long() - 127
    e = e[:, :, :, None].expand(*e.shape, s["block"]).flatten(2)
    return (bytes_ * _two_to(e[..., None])).transpose(1, 2).flatten(0, 1)


def _exact_append(s, B, each):
    block, ps = s["block"], s["k"].shape[2]
    out = {n: torch.zeros(B, s["count"], *s["k_rows"].shape[1:], dtype=torch.float64, device="cuda") for n in ("k", "v")}
    for b, c in enumerate(s["context"].cpu().tolist()):
        lo, end = c - c % block, c + each
        pages = s["table"][b, lo // ps:(end + ps - 1) // ps].long()
        for name in ("k", "v"):
            y = torch.zeros((end - lo + block - 1) // block * block, *out[name].shape[2:], dtype=torch.float64, device="cuda")
            y[:c - lo] = _stands_for(s, name, pages)[lo % ps:][:c - lo]
            y[c - lo:end - lo] = s[name + "_rows"][b * each:(b + 1) * each]
            y = y.view(-1, block, *y.shape[1:])
            part, e = torch.frexp(y.abs().amax((1, 3), keepdim=True) / 448)
            e = (e - (part == 0.5).int()).masked_fill_(part == 0, LEAST).clamp_(LEAST, MOST)
            # e4m3 numbers have three bits behind the leading one, and none below 2^-9
            lead = torch.frexp(y)[1] - 1 - e
            step = _two_to(lead.clamp_min(-6) - 3 + e)
            out[name][b, :end - lo] = (torch.round(y / step) * step).flatten(0, 1)[:end - lo]
    return out


def _exact_read(s):
    B, count, ps = s["table"].shape[0], s["count"], s["k"].shape[2]
    out = {n: torch.zeros(B, count, s["k"].shape[1], s["k"].shape[3], dtype=torch.float64, device="cuda") for n in ("k", "v")}
    for b, c in enumerate(s["context"].cpu().tolist()):
        for name in ("k", "v"):
            out[name][b, :c] = _stands_for(s, name, s["table"][b, :(c + ps - 1) // ps].long())[:c]
    return out


def _exact_attend(s, B, each):
    paths = _depths(s, B, each)
    context = s["context"].cpu().tolist()
    heads, ps, D = s["k"].shape[1:]
    group = s["q"].shape[1] // heads
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, c in enumerate(context):
        pages = s["table"][b, :(c + each + ps - 1) // ps].long()
        see = torch.zeros(each, c + each, dtype=torch.bool)
        see[:, :c] = True
        for u, p in enumerate(paths[b]):
            see[u, [c + a for a in p]] = True
        see = see.cuda().repeat_interleave(group, 0)
        keys, vals = (_stands_for(s, n, pages)[:c + each].transpose(0, 1).contiguous() for n in ("k", "v"))
        q = s["q"][b * each:(b + 1) * each].double()
        for h in range(heads):
            mine = q[:, h * group:(h + 1) * group].reshape(-1, D)
            w = (mine @ keys[h].T / math.sqrt(D)).masked_fill_(~see, -math.inf)
            out[b * each:(b + 1) * each, h * group:(h + 1) * group] = (torch.softmax(w, 1) @ vals[h]).view(each, group, D)
    return out


def _exact_logprobs(s):
    n = s["tokens"].shape[0]
    at = torch.arange(n, device="cuda") if s["rows"] is None else s["rows"].long()
    V, top = s["logits"].shape[1], s["top"]
    out = {"logprob": [], "entropy": [], "top_tokens": [], "top_logprobs": []}
    for lo in range(0, n, 256):
        x = s["logits"][at[lo:lo + 256]]
        logp = torch.log_softmax(x.double(), 1)
        out["logprob"].append(logp.gather(1, s["tokens"][lo:lo + 256].long()))
        out["entropy"].append(-torch.where(logp > -math.inf, logp * logp.exp(), 0.0).sum(1))
        first = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
        likely = logp.gather(1, first)
        out["top_tokens"].append(torch.where(likely > -math.inf, first, -1).int())
        out["top_logprobs"].append(likely)
    return {k: torch.cat(v) for k, v in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    B, each = case.get("B", 0), max(case.get("K", 0) + 1, case.get("N", 0))
    if case["op"] == "rotate":
        return _exact_rotate(s, B, each)
    if case["op"] == "append":
        return _exact_append(s, B, each)
    if case["op"] == "read":
        return _exact_read(s)
    if case["op"] == "attend":
        return _exact_attend(s, B, each)
    return _exact_logprobs(s)
