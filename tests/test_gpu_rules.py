"""process_logits and verify_constrained against the oracle.  The rules are defined in float32,
operation by operation, so processed logits and tokens are compared exactly."""

import numpy as np
import pytest
import torch

import drafter_routing_verification_amd as wf
from gpu_helpers import DEV, dev, host
from oracle import rounds as orc
from round_helpers import Round, bits, i32, make_logits, make_rules, stored, to_bf16

pytestmark = pytest.mark.gpu

# (kind, B, K, N, V): one row, single tokens, vocabularies around the vector and chunk sizes,
# full chains and trees, the largest chain.
SHAPES = [
    ("chain", 1, 0, 0, 1), ("chain", 3, 0, 0, 7), ("chain", 2, 4, 0, 8), ("tree", 1, 0, 1, 97),
    ("tree", 3, 0, 13, 4099), ("routed", 5, 6, 9, 4096), ("chain", 4, 16, 0, 8193),
    ("routed", 4, 3, 17, 20011), ("tree", 2, 0, 61, 32768), ("chain", 1, 1023, 0, 33),
    ("tree", 1, 0, 1024, 50), ("chain", 70, 2, 0, 260), ("chain", 2, 1, 0, 151936),
]


def _expected(r, raw, dtype, rules):
    """Processed float32 rows; rows of no well-formed sequence are NaN."""
    x = np.full((r.total, r.V), np.nan, np.float32)
    for b, q in enumerate(r.seqs):
        if q.n:
            x[q.row0:q.row0 + q.n] = orc.process_rows(bits(raw[q.row0:q.row0 + q.n], dtype), b, q, rules)
    return x


def _verified(r, x):
    al, bonus, best = (np.zeros(r.B, np.int64) for _ in range(3))
    t = np.full(r.total, -9)
    for b, q in enumerate(r.seqs):
        if q.n:
            t[q.row0:q.row0 + q.n] = orc.constrained_tokens(x[q.row0:q.row0 + q.n])
        al[b], bonus[b], best[b] = orc.verify_seq(q, t[q.row0:q.row0 + q.n])
    return al, bonus, best, t


def _check(r, raw, dtype, o_rules, rules, stride=None):
    stride = stride or (r.V + 7) // 8 * 8 + 8
    x = _expected(r, raw, dtype, o_rules)
    mine = r.owned()
    logits = stored(raw, dtype, stride)
    # verification
    t = torch.full((r.total,), -9, dtype=torch.int32, device=DEV)
    got = wf.verify_constrained(logits, r.rows, rules, row_argmax=t)
    for a, e in zip(got, _verified(r, x)):
        assert np.array_equal(host(a), e)
    # written: float32, bfloat16, in place
    for name, stored_out in (("f32", lambda y: y), ("bf16", to_bf16)):
        sentinel = {"f32": np.float32(-77), "bf16": np.uint16(0x4321)}[name]
        want = np.where(mine[:, None], stored_out(np.nan_to_num(x, nan=0, neginf=-np.inf, posinf=np.inf)),
                        sentinel)
        out = stored(np.full((r.total, r.V), sentinel), name, stride, fill=sentinel)
        base = out._base if out._base is not None else out
        wf.process_logits(logits, r.rows, rules, out=out)
        got = host(base.view(torch.int16) if name == "bf16" else base).reshape(r.total, stride)
        got = got.view(np.uint16) if name == "bf16" else got
        assert np.array_equal(got[:, :r.V], want), name
        assert np.all(got[:, r.V:] == sentinel), f"{name}: entries past V written"
    before = bits(raw, dtype)
    wf.process_logits(logits, r.rows, rules, out=logits)
    want = np.where(mine[:, None], x if dtype == "f32" else bits(to_bf16(np.nan_to_num(
        x, nan=0, neginf=-np.inf, posinf=np.inf)), "bf16"), before)
    assert np.array_equal(host(logits.float()), want), "in place"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rules_against_oracle(shape, dtype):
    print(f"rules {shape} {dtype}", flush=True)
    r = Round(*shape, seed=sum(shape[1:]))
    o, rules = make_rules(r, seed=shape[4] + 1)
    _check(r, make_logits(r, dtype, 7), dtype, o, rules)


@pytest.mark.parametrize("on", ["history", "penalties", "bias", "allow", "none"])
def test_each_rule_alone(on):
    r = Round("routed", 6, 5, 12, 8200, seed=3)
    names = ("history", "penalties", "bias", "allow")
    o, rules = make_rules(r, 5, **{n: n == on or (on == "history" and n == "penalties") for n in names})
    _check(r, make_logits(r, "bf16", 8), "bf16", o, rules)


@pytest.mark.parametrize("kind", ["chain", "tree", "routed"])
def test_bad_data_has_its_defined_result(kind):
    r = Round(kind, 9, 6, 14, 999, seed=11, bad=True)
    o, rules = make_rules(r, 12)
    _check(r, make_logits(r, "f32", 13), "f32", o, rules)


@pytest.mark.parametrize("kind", ["chain", "tree", "routed"])
def test_no_rules_equal_the_plain_calls(kind):
    r = Round(kind, 5, 6, 14, 5003, seed=21)
    raw = make_logits(r, "bf16", 22)
    logits = stored(raw, "bf16", 5008)
    al, bonus, best, t = wf.verify_constrained(logits, r.rows, wf.LogitRules())
    ten = r.rows.tensors
    if kind == "chain":
        e_al, e_bo, e_t = wf.verify_chain(logits, ten["chain_draft"])
        e_be = e_al - 1
    elif kind == "tree":
        e_al, e_bo, e_be, e_t = wf.verify_tree(logits, ten["parent"], ten["draft_ids"], ten["d2t"])
    else:
        e_al, e_bo, e_be, e_t = wf.verify_routed(logits, ten["row_offsets"], r.total, ten["choice"],
                                                 ten["chain_draft"], ten["parent"], ten["draft_ids"], ten["d2t"])
    mine = torch.from_numpy(r.owned()).to(DEV)
    for a, e in ((al, e_al), (bonus, e_bo), (best, e_be), (t[mine], e_t[mine])):
        assert torch.equal(a, e)


def test_rows_that_nothing_is_left_of():
    # Row 0 of sequence 0 allows nothing: no token, nothing accepted, although the draft holds -1.
    # Sequence 1 has only -inf logits.  Sequence 2 allows one token, whose logit is the lowest.
    V, K = 600, 2
    x = np.zeros((3 * (K + 1), V), np.float32)
    x[3:6] = -np.inf
    x[6:9, 77] = np.finfo(np.float32).min
    allow = np.full((9, 19), -1, np.int32)
    allow[0] = 0
    allow[6:9] = 0
    allow[6:9, 77 // 32] = 1 << (77 % 32)
    draft = np.array([[-1, -1], [-1, 3], [77, 77]])
    rows = wf.chain_rows(i32(draft))
    rules = wf.LogitRules(allow=i32(allow))
    for dt in (torch.float32, torch.bfloat16):
        al, bonus, best, t = wf.verify_constrained(dev(x).to(dt), rows, rules)
        # (the lowest float32 rounds to -inf in bfloat16: nothing is left there either)
        low = 77 if dt == torch.float32 else -1
        assert host(t).tolist() == [-1, 0, 0, -1, -1, -1, low, low, low]
        assert host(al).tolist() == [1, 1, 3 if low == 77 else 1]
        assert host(bonus).tolist() == [-1, -1, low]
        assert host(best).tolist() == [0, 0, 2 if low == 77 else 0]


def test_infinite_logits_and_masked_nan_positions():
    V = 300
    x = np.random.default_rng(0).normal(0, 1, (4, V)).astype(np.float32)
    x[0, 5] = np.inf
    x[1, 9] = np.nan       # masked away
    x[2, :] = -np.inf
    x[2, 250] = -5
    allow = np.full((4, 10), -1, np.int32)
    allow[1, 9 // 32] &= ~(1 << 9)
    rows = wf.chain_rows(i32(np.zeros((4, 0))))
    _, _, _, t = wf.verify_constrained(stored(x, "f32", 304), rows, wf.LogitRules(allow=i32(allow)))
    y = x.copy()
    y[1, 9] = -np.inf
    assert host(t).tolist() == np.argmax(y, 1).tolist()


def test_repeated_tokens_on_the_path_count_each_time():
    V, K = 64, 6
    draft = np.array([[5, 5, 5, 9, 5, 9]])
    r = Round("chain", 1, K, 0, V, seed=1)
    r.draft = draft
    r.seqs = [orc.chain_seq(0, draft[0], V)]
    r.rows = wf.chain_rows(i32(draft))
    pen = np.array([[1.5, 0.25, 0.5]], np.float32)
    h = np.zeros((1, V), np.uint16)
    h[0, 5] = 0x7FFF          # a full count still grows by the path's tokens
    h[0, 9] = 0x8000
    raw = np.random.default_rng(2).normal(0, 2, (K + 1, V)).astype(np.float32)
    _check(r, raw, "f32", orc.Rules(history=h, penalties=pen),
           wf.LogitRules(torch.from_numpy(h.view(np.int16)).to(DEV), penalties=dev(pen)))


def test_sequences_sharing_a_slot_and_many_biases():
    r = Round("chain", 4, 3, 0, 9000, seed=31)
    o, _ = make_rules(r, 32, allow=False, slots=2)
    ids = np.sort(np.random.default_rng(3).permutation(9000)[:4000])
    o.bias = (np.array([0, 4000, 4000, 4000, 4000]), ids, np.linspace(-4, 4, 4000).astype(np.float32))
    rules = wf.LogitRules(torch.from_numpy(o.history.view(np.int16)).to(DEV), slot=i32(o.slot),
                          penalties=dev(o.penalties), bias=(i32(o.bias[0]), i32(ids), dev(o.bias[2])))
    _check(r, make_logits(r, "bf16", 4), "bf16", o, rules)


def test_offsets_past_32_bits():
    # 40,000 rows of 56,000 float32 logits end past 8 GiB and 2^31 elements.
    B, V = 40000, 56000
    logits = torch.zeros(B, V, device=DEV)
    put = torch.arange(B, device=DEV) % V
    logits[torch.arange(B, device=DEV), put] = 2.0
    rows = wf.chain_rows(torch.zeros(B, 0, dtype=torch.int32, device=DEV))
    al, bonus, _, t = wf.verify_constrained(logits, rows, wf.LogitRules())
    assert torch.equal(t.long(), put) and bool((al == 1).all()) and torch.equal(bonus, t)
    wf.process_logits(logits, rows, wf.LogitRules(), out=logits)
    assert float(logits[-1].sum()) == 2.0 and float(logits[-1, put[-1]]) == 2.0


def test_another_stream_and_empty_batch():
    r = Round("tree", 3, 0, 12, 4100, seed=41)
    o, rules = make_rules(r, 42)
    raw = make_logits(r, "bf16", 43)
    logits = stored(raw, "bf16", 4104)
    e = _verified(r, _expected(r, raw, "bf16", o))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [wf.verify_constrained(logits, r.rows, rules, stream=s) for _ in range(3)]
    s.synchronize()
    for g in got:
        for a, b in zip(g[:3], e[:3]):
            assert np.array_equal(host(a), b)
    none = wf.chain_rows(torch.zeros(0, 4, dtype=torch.int32, device=DEV))
    al, bonus, best, t = wf.verify_constrained(torch.zeros(0, 64, device=DEV), none, wf.LogitRules())
    assert al.numel() == bonus.numel() == best.numel() == 0
    assert wf.process_logits(torch.zeros(0, 64, device=DEV), none, wf.LogitRules()).numel() == 0
