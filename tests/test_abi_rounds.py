"""Host-side checks of the calls around a round (no GPU): argument errors come back as statuses
before anything is launched, and workspace sizes answer."""

import ctypes

import pytest

from drafter_routing_verification_amd import _rounds as rd

A = 1 << 20   # a fake, aligned device address: every call here is refused before it is used
V = 151936


def _rows(**kw):
    s = rd._RowsStruct(kind=0, B=4, K=16, N=61, Vd=32000, total_rows=68, chain_draft=A, parent=A,
                       draft_ids=A, d2t=A, row_offsets=A, choice=A)
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def _rules(**kw):
    s = rd._RulesStruct(history=A, history_stride=V, slots=4, bias_count=3, slot=A, penalties=A,
                        bias_offsets=A, bias_ids=A, bias_values=A, allow=A, allow_stride=V // 32)
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def _cache(**kw):
    s = rd._CacheStruct(k=A, v=A, layer_stride=100 * 8 * 16 * 128, page_stride=8 * 16 * 128, dtype=1,
                        layers=2, pages=100, heads=8, page_size=16, head_dim=128, seqs=4, max_pages=30,
                        table=A, held=A, context=A, refs=A)
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


@pytest.fixture(scope="module")
def fn():
    return rd.functions()


def test_constrained_refusals(fn):
    def call(rows=None, rules=None, **kw):
        a = dict(logits=A, dtype=1, V=V, stride=V, al=A, bonus=A, best=None, argmax=None, ws=A, size=1 << 30)
        a.update(kw)
        return fn.verify_constrained(a["logits"], a["dtype"], a["V"], a["stride"], rows or _rows(),
                                     rules or _rules(), a["al"], a["bonus"], a["best"], a["argmax"],
                                     a["ws"], a["size"], None)

    assert call(dtype=2) == -3 and call(logits=None) == -1 and call(logits=A + 2) == -4
    assert call(V=0) == -2 and call(stride=V - 8) == -2 and call(V=101, stride=101) == -4
    assert call(V=(1 << 30) + 8, stride=1 << 31) == -2
    for bad in (dict(kind=3), dict(kind=-1), dict(B=-1), dict(K=-1), dict(K=1024),
                dict(kind=1, N=0), dict(kind=1, N=1025), dict(kind=2, total_rows=-1),
                dict(kind=1, Vd=0), dict(B=1 << 22, K=1023)):
        assert call(rows=_rows(**bad)) == -2, bad
    for bad in (dict(chain_draft=None), dict(kind=1, parent=None), dict(kind=1, draft_ids=None),
                dict(kind=1, d2t=None), dict(kind=2, row_offsets=None), dict(kind=2, choice=None)):
        assert call(rows=_rows(**bad)) == -1, bad
    for bad, status in ((dict(slots=-1), -2), (dict(history_stride=V - 8), -2), (dict(history=A + 2), -4),
                        (dict(history_stride=V + 4), -4), (dict(bias_count=-1), -2),
                        (dict(bias_ids=None), -1), (dict(allow_stride=V // 32 - 1), -2),
                        (dict(allow=A + 2), -4)):
        assert call(rules=_rules(**bad)) == status, bad
    assert call(al=None) == -1 and call(bonus=None) == -1
    need = fn.verify_constrained_workspace_bytes(_rows(), V)
    assert need % 256 == 0 and need >= 68 * 8
    assert call(ws=None) == -5 and call(size=need - 1) == -5 and call(ws=A + 64) == -5
    assert call(rows=_rows(B=0)) == 0
    assert fn.verify_constrained_workspace_bytes(_rows(B=0), V) == 0
    assert fn.verify_constrained_workspace_bytes(_rows(K=5000), V) == 0
    assert fn.verify_constrained_workspace_bytes(_rows(), 0) == 0


def test_process_and_history_refusals(fn):
    def process(out=A, dtype=1, stride=V, rows=None):
        return fn.process_logits(A * 8, 1, V, V, rows or _rows(), _rules(), out, dtype, stride, None)

    assert process(out=None) == -1 and process(dtype=7) == -3 and process(stride=V - 8) == -2
    assert process(out=A + 2) == -4 and process(rows=_rows(B=0)) == 0
    assert process(out=A * 8, dtype=0) == -2 and process(out=A * 8, stride=V + 8) == -2   # in place, laid out else
    prompt = lambda h=A, S=4, n=V, st=V, B=2, t=A, o=A, c=9: fn.history_prompt(h, S, n, st, B, None, t, o, c, None)  # noqa: E731
    assert prompt(h=None) == -1 and prompt(S=-1) == -2 and prompt(st=V + 4) == -4 and prompt(B=-1) == -2
    assert prompt(t=None) == -1 and prompt(o=None) == -1 and prompt(c=-1) == -2
    assert prompt(B=0) == 0 and prompt(c=0) == 0
    update = lambda rows, al=A, best=A, bonus=A: fn.history_update(A, 4, V, V, rows, None, al, best, bonus, None)  # noqa: E731
    assert update(_rows(), al=None) == -1 and update(_rows(), bonus=None) == -1
    assert update(_rows(kind=1), best=None) == -1 and update(_rows(B=0)) == 0 and update(_rows(K=-2)) == -2


def test_cache_refusals(fn):
    free = lambda **kw: fn.cache_free(_cache(**kw), 1, None, None)  # noqa: E731
    assert free() == -1                                       # no sequences given
    for bad, status in ((dict(dtype=5), -3), (dict(layers=0), -2), (dict(pages=0), -2), (dict(heads=0), -2),
                        (dict(page_size=8), -2), (dict(page_size=24), -2), (dict(page_size=2048), -2),
                        (dict(head_dim=96), -2), (dict(seqs=0), -2), (dict(max_pages=0), -2),
                        (dict(max_pages=1 << 28), -2), (dict(page_stride=100), -2), (dict(layer_stride=5), -2),
                        (dict(k=None), -1), (dict(table=None), -1), (dict(refs=None), -1),
                        (dict(k=A + 8), -4), (dict(page_stride=8 * 16 * 128 + 4), -4)):
        assert free(**bad) == status, bad
    assert fn.cache_free(_cache(), 0, None, None) == 0 and fn.cache_free(_cache(), -1, A, None) == -2
    size = fn.cache_pages_workspace_bytes(_cache(), 5)
    assert size >= 4 * (5 + 8 + 100) and fn.cache_pages_workspace_bytes(_cache(), 0) == 0
    for call in (fn.cache_fork, fn.cache_reserve):
        assert call(_cache(), -1, A, A, A, A, size, None) == -2 and call(_cache(), 0, None, None, None, None, 0, None) == 0
        assert call(_cache(), 5, None, A, A, A, size, None) == -1 and call(_cache(), 5, A, A, None, A, size, None) == -1
        assert call(_cache(), 5, A, A, A, A, size - 1, None) == -5 and call(_cache(), 5, A, A, A, None, size, None) == -5
    compact = lambda rows, al=A, best=A: fn.cache_compact(_cache(), rows, None, al, best, None, None)  # noqa: E731
    assert compact(_rows(kind=1), best=None) == -1 and compact(_rows(), al=None) == -1
    assert compact(_rows(B=0), al=None) == 0 and compact(_rows(kind=1, N=2000)) == -2
    append = lambda layer=0, k=A, ks=1024, v=A, vs=1024, rows=None: fn.cache_append(  # noqa: E731
        _cache(), layer, rows or _rows(chain_draft=None), None, k, ks, v, vs, None)
    assert append(layer=2) == -2 and append(layer=-1) == -2 and append(k=None) == -1 and append(ks=1000) == -2
    assert append(v=A + 8) == -4 and append(vs=1025) == -4 and append(rows=_rows(B=0)) == 0


def test_attend_refusals(fn):
    def call(**kw):
        a = dict(q=A, qs=4096, heads=32, layer=0, rows=_rows(chain_draft=None), most=400, scale=1.0, out=A,
                 ws=A, size=1 << 30)
        a.update(kw)
        return fn.attend(a["q"], a["qs"], a["heads"], _cache(), a["layer"], a["rows"], None, a["most"],
                         a["scale"], a["out"], a["ws"], a["size"], None)

    assert call(q=None) == -1 and call(q=A + 8) == -4 and call(qs=4088) == -2 and call(qs=4100) == -4
    assert call(heads=0) == -2 and call(heads=12) == -2 and call(layer=2) == -2 and call(most=-1) == -2
    assert call(scale=float("inf")) == -2 and call(scale=float("nan")) == -2
    assert call(out=None) == -1 and call(out=A + 4) == -4
    assert call(rows=_rows(B=0), q=None, out=None) in (0, -1)
    need = fn.attend_workspace_bytes(_cache(), _rows(), 32, 400)
    assert need > 0 and call(size=need - 1) == -5 and call(ws=None) == -5 and call(ws=A + 16) == -5
    assert fn.attend_workspace_bytes(_cache(), _rows(), 33, 400) == 0
    assert fn.attend_workspace_bytes(_cache(head_dim=80), _rows(), 32, 400) == 0


def test_python_refuses_host_tensors():
    import torch
    import drafter_routing_verification_amd as wf
    i = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: wf.chain_rows(i), lambda: wf.tree_rows(i), lambda: wf.LogitRules(i.short()),
                 lambda: wf.PageCache(i, i, i, i, i, i)):
        with pytest.raises(TypeError):
            call()


def test_a_stream_of_another_gpu_is_refused():
    from types import SimpleNamespace
    with pytest.raises(ValueError, match="GPU 1"):
        rd._enter(0, SimpleNamespace(device_index=1, cuda_stream=0))


def test_sizes_past_32_bits_are_refused_by_the_binding():
    handle = lambda ref: type("Handle", (), {"ref": ref})()  # noqa: E731
    cache, rows = handle(_cache()), handle(_rows())
    assert rd.attend_workspace_bytes(cache, rows, 32, 131000) > 0
    for heads, context in ((32, 1 << 32), ((1 << 32) + 32, 131000), (32, -1 - (1 << 31))):
        with pytest.raises(ValueError, match="32 bits"):
            rd.attend_workspace_bytes(cache, rows, heads, context)
    with pytest.raises(ValueError, match="32 bits"):
        rd.verify_constrained_workspace_bytes(rows, (1 << 32) + V)
