"""Host-side checks of a decoding step's calls (no GPU): argument errors come back as statuses before
anything is launched, and workspace sizes answer."""

import ctypes
import math

import pytest

import drafter_routing_verification_amd as wf
from drafter_routing_verification_amd import _decode as de
from drafter_routing_verification_amd import _rounds as rd
from test_abi_rounds import A, V, _cache, _rows


def _cache8(block=16, k_scale=A, v_scale=A, scale_layer_stride=100 * 8, scale_page_stride=8, **kw):
    pages = rd._CacheStruct(k=A, v=A, layer_stride=100 * 8 * 16 * 128, page_stride=8 * 16 * 128, dtype=2, layers=2,
                            pages=100, heads=8, page_size=16, head_dim=128, seqs=4, max_pages=30, table=A, held=A,
                            context=A, refs=A)
    for k, v in kw.items():
        setattr(pages, k, v)
    return de._Cache8Struct(pages, k_scale, v_scale, scale_layer_stride, scale_page_stride, block)


def _ref(**kw):
    return ctypes.byref(_cache8(**kw))


@pytest.fixture(scope="module")
def fn():
    return de.functions()


def test_rotate_refusals(fn):
    def call(dtype=1, dim=128, rows=None, context=A, seqs=4, q=(A, A, 4096, 4096, 32), k=(A, A, 1024, 1024, 8), **kw):
        t = dict(frequency=A, pairs=64, layout=0, magnitude=1.0)
        t.update(kw)
        one = None if q is None else ctypes.byref(de._RotaryRowsStruct(*q))
        two = None if k is None else ctypes.byref(de._RotaryRowsStruct(*k))
        return fn.rotate(ctypes.byref(de._RotaryStruct(**t)), dtype, dim, rows or _rows(chain_draft=None), None, context, seqs,
                         one, two, None)

    assert fn.rotate(None, 1, 128, _rows(), None, A, 4, None, None, None) == -1 and call(q=None) == -1
    assert call(dtype=2) == -3 and call(dim=0) == -2 and call(dim=516) == -2 and call(dim=1024) == -2
    assert call(dim=4, pairs=1) == -2                                           # 8 bytes a head
    assert call(pairs=0) == -2 and call(pairs=65) == -2 and call(layout=2) == -2 and call(layout=-1) == -2
    assert call(magnitude=math.inf) == -2 and call(magnitude=math.nan) == -2 and call(seqs=-1) == -2
    assert call(frequency=None) == -1 and call(context=None) == -1
    for which in ("q", "k"):
        ok = (A, 2 * A, 4096, 4096, 8)
        for at, value, status in ((0, None, -1), (1, None, -1), (0, A + 8, -4), (1, A + 2, -4), (2, 1000, -2),
                                  (3, 1000, -2), (2, 4100, -4), (3, 4100, -4), (4, 0, -2), (4, 4097, -2)):
            bad = list(ok)
            bad[at] = value
            assert call(**{which: tuple(bad)}) == status, (which, at, value)
        assert call(**{which: (A, A, 4096, 4104, 8)}) == -2                      # in place, laid out else
    assert call(rows=_rows(B=0), context=None) == 0 and call(rows=_rows(K=-1)) == -2
    assert call(rows=_rows(kind=1, parent=None)) == -1 and call(rows=_rows(B=1 << 22, K=1)) == -2


def test_cache8_refusals(fn):
    def append(cache=None, layer=0, rows=None, dtype=1, k=A, ks=1024, v=A, vs=1024):
        return fn.cache8_append(cache or _ref(), layer, rows or _rows(chain_draft=None), None, dtype, k, ks, v, vs, None)

    for bad, status in ((dict(dtype=1), -3), (dict(dtype=0), -3), (dict(layers=0), -2), (dict(pages=0), -2),
                        (dict(page_size=8), -2), (dict(head_dim=96), -2), (dict(max_pages=1 << 28), -2),
                        (dict(page_stride=100), -2), (dict(layer_stride=5), -2), (dict(k=None), -1), (dict(refs=None), -1),
                        (dict(k=A + 8), -4), (dict(page_stride=8 * 16 * 128 + 8), -4), (dict(block=0), -2),
                        (dict(block=3), -2), (dict(block=32), -2), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
                        (dict(scale_page_stride=7), -2), (dict(scale_layer_stride=3), -2),
                        (dict(block=1, scale_page_stride=100), -2)):
        assert append(_ref(**bad)) == status, bad
    assert append(dtype=2) == -3 and append(dtype=-1) == -3 and append(layer=2) == -2 and append(layer=-1) == -2
    assert append(k=None) == -1 and append(ks=1000) == -2 and append(v=A + 8) == -4 and append(vs=1028) == -4
    assert append(rows=_rows(B=0)) == 0 and append(rows=_rows(kind=1, N=2000)) == -2
    assert append(_ref(block=1, scale_page_stride=128, scale_layer_stride=12800), rows=_rows(B=4097, K=1023)) == -2

    def read(cache=None, layer=0, B=4, count=5, pending=0, dtype=1, k=A, v=A):
        return fn.cache8_read(cache or _ref(), layer, B, None, None, count, pending, dtype, k, v, None)

    assert read(_ref(block=0)) == -2 and read(dtype=2) == -3 and read(layer=2) == -2 and read(B=-1) == -2
    assert read(count=-1) == -2 and read(pending=-1) == -2 and read(count=(1 << 30) + 1) == -2
    assert read(k=A + 8) == -4 and read(v=A + 8) == -4 and read(B=1 << 20, count=1 << 10) == -2
    assert read(B=0) == 0 and read(count=0) == 0 and read(k=None, v=None) == 0
    compact = lambda rows, al=A, best=A: fn.cache8_compact(_ref(), rows, None, al, best, None, None)  # noqa: E731
    assert compact(_rows(kind=1), best=None) == -1 and compact(_rows(), al=None) == -1 and compact(_rows(B=0), al=None) == 0
    size = rd.functions().cache_pages_workspace_bytes(ctypes.byref(_cache8().pages), 5)
    assert size >= 4 * (5 + 8 + 100)
    fork = lambda n=5, src=A, dst=A, st=A, ws=A, size=size: fn.cache8_fork(_ref(), n, src, dst, st, ws, size, None)  # noqa: E731
    assert fork(n=-1) == -2 and fork(n=0, src=None) == 0 and fork(src=None) == -1 and fork(st=None) == -1
    assert fork(size=size - 1) == -5 and fork(ws=None) == -5


def test_the_other_caches_calls_take_an_8_bit_cache_for_its_pages_alone():
    old, pages = rd.functions(), _cache8().pages
    ref = ctypes.byref(pages)
    assert old.cache_free(ref, 1, None, None) == -1 and old.cache_free(ref, 0, None, None) == 0
    assert old.cache_reserve(ref, 5, None, A, A, A, 1 << 20, None) == -1
    assert old.cache_append(ref, 0, _rows(), None, A, 1024, A, 1024, None) == -3
    assert old.cache_compact(ref, _rows(), None, A, A, None, None) == -3
    assert old.cache_fork(ref, 5, A, A, A, A, 1 << 20, None) == -3
    assert old.attend(A, 4096, 32, ref, 0, _rows(), None, 400, 1.0, A, A, 1 << 30, None) == -3
    assert old.attend_workspace_bytes(ref, _rows(), 32, 400) == 0
    assert old.cache_free(_cache(dtype=5), 1, A, None) == -3


def test_attend8_refusals(fn):
    def call(cache=None, **kw):
        a = dict(q=A, qs=4096, heads=32, dtype=1, layer=0, rows=_rows(chain_draft=None), most=400, scale=1.0, out=A,
                 ws=A, size=1 << 30)
        a.update(kw)
        return fn.attend8(a["q"], a["qs"], a["heads"], a["dtype"], cache or _ref(), a["layer"], a["rows"], None, a["most"],
                          a["scale"], a["out"], a["ws"], a["size"], None)

    assert call(q=None) == -1 and call(q=A + 8) == -4 and call(qs=4088) == -2 and call(qs=4100) == -4
    assert call(heads=0) == -2 and call(heads=12) == -2 and call(layer=2) == -2 and call(most=-1) == -2
    assert call(dtype=2) == -3 and call(_ref(dtype=1)) == -3 and call(_ref(block=5)) == -2
    assert call(scale=math.inf) == -2 and call(scale=math.nan) == -2 and call(out=None) == -1 and call(out=A + 4) == -4
    assert call(rows=_rows(B=0), q=None, out=None) in (0, -1)
    size = fn.attend8_workspace_bytes(_ref(), _rows(), 1, 32, 400)
    if size:
        assert call(size=size - 1) == -5 and call(ws=None) == -5 and call(ws=A + 16) == -5
    assert fn.attend8_workspace_bytes(_ref(), _rows(), 1, 33, 400) == 0
    assert fn.attend8_workspace_bytes(_ref(), _rows(), 2, 32, 400) == 0


def test_token_logprobs_refusals(fn):
    def call(**kw):
        a = dict(logits=A, dtype=1, total=68, V=V, stride=V, n=68, rows=None, given=1, tokens=A, top=5, lp=A, h=A,
                 ids=A, top_lp=A, ws=A, size=1 << 30)
        a.update(kw)
        return fn.token_logprobs(*(a[k] for k in ("logits", "dtype", "total", "V", "stride", "n", "rows", "given",
                                                  "tokens", "top", "lp", "h", "ids", "top_lp", "ws", "size")), None)

    assert call(logits=None) == -1 and call(dtype=2) == -3 and call(total=-1) == -2 and call(V=0) == -2
    assert call(stride=V - 8) == -2 and call(logits=A + 4) == -4 and call(V=101, stride=101) == -4
    assert call(V=(1 << 30) + 8, stride=1 << 31) == -2
    assert call(n=-1) == -2 and call(n=69) == -2 and call(given=-1) == -2 and call(given=65537) == -2
    assert call(top=-1) == -2 and call(top=65) == -2 and call(n=(1 << 22) + 1, rows=A) == -2
    assert call(tokens=None) == -1 and call(lp=None) == -1 and call(ids=None) == -1 and call(top_lp=None) == -1
    size = fn.token_logprobs_workspace_bytes(68, V, 5)
    assert size > 0 and call(size=size - 1) == -5 and call(ws=None) == -5 and call(ws=A + 16) == -5
    assert call(n=0) == 0 and call(n=0, logits=None, total=0) == 0
    for bad in ((0, V, 5), (68, 0, 5), (68, V, 65), (68, V, -1), (1 << 23, V, 1)):
        assert fn.token_logprobs_workspace_bytes(*bad) == 0


def test_sizes_past_32_bits_are_refused_by_the_binding():
    cache = type("Handle", (wf.PageCache8,), {"__init__": lambda self: None})()
    struct = _cache8()
    cache.ref = ctypes.byref(struct)
    rows = type("Handle", (), {"ref": _rows()})()
    for heads, context in ((32, 1 << 32), ((1 << 32) + 32, 131000)):
        with pytest.raises(ValueError, match="32 bits"):
            rd.attend_workspace_bytes(cache, rows, heads, context)
    for bad in ((1 << 32, V, 1), (1, (1 << 32) + V, 1), (1, V, 1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            wf.token_logprobs_workspace_bytes(*bad)


def test_python_refuses_host_tensors():
    import torch
    f = torch.zeros(4, dtype=torch.float64)
    i = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: wf.Rotary(f), lambda: wf.PageCache8(i, i, i, i, i, i, i, i), lambda: wf.token_logprobs(i),
                 lambda: wf.cache_read(None, 4)):
        with pytest.raises(TypeError):
            call()


def test_rotary_frequencies():
    plain, m = wf.rotary_frequencies(4, 10000.0)
    assert plain == pytest.approx([1, 0.1, 0.01, 0.001]) and m == 1
    assert wf.rotary_frequencies(4, 10000.0, ("linear", 4.0))[0] == pytest.approx([x / 4 for x in plain])
    based, _ = wf.rotary_frequencies(4, 10000.0, ("base", 8.0))
    assert based[0] == 1 and based[3] == pytest.approx(plain[3] / 8) and plain[1] / 8 < based[1] < plain[1]
    # 64 pairs, trained over 8,192: the fastest as they are, the slowest slowed, each in between
    plain, _ = wf.rotary_frequencies(64, 500000.0)
    waved, _ = wf.rotary_frequencies(64, 500000.0, ("wavelength", 8.0, 1.0, 4.0, 8192))
    for f, g in zip(plain, waved):
        length = 2 * math.pi / f
        if length < 8192 / 4:
            assert g == pytest.approx(f)
        elif length > 8192:
            assert g == pytest.approx(f / 8)
        else:
            assert f / 8 < g < f
    turned, m = wf.rotary_frequencies(64, 10000.0, ("turns", 16.0, 1.0, 32.0, 4096))
    assert m == pytest.approx(1 + 0.1 * math.log(16)) and wf.rotary_frequencies(64, 10000.0, ("turns", 1.0, 1.0, 32.0, 4096))[1] == 1
    plain, _ = wf.rotary_frequencies(64, 10000.0)
    turns = [f * 4096 / (2 * math.pi) for f in plain]
    assert all(g == pytest.approx(f) for f, g, n in zip(plain, turned, turns) if n > 34)
    assert all(g == pytest.approx(f / 16) for f, g, n in zip(plain, turned, turns) if n < 0.9)
    assert all(a >= b for a, b in zip(turned, turned[1:]))
    for bad in ((0, 1e4, None), (4, -1.0, None), (4, 1e4, ("linear", 0.0)), (4, 1e4, ("x", 2.0)),
                (4, 1e4, ("wavelength", 8.0, 4.0, 1.0, 8192)), (4, 1e4, ("turns", 8.0, 4.0, 1.0, 8192))):
        with pytest.raises(ValueError):
            wf.rotary_frequencies(*bad)
