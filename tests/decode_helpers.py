"""Caches of 8 bits for the tests of a decoding step, on the host and on the GPU."""

import numpy as np
import torch

import drafter_routing_verification_amd as wf
from gpu_helpers import DEV, dev
from oracle import decode as dec
from round_helpers import bits, i32, to_bf16


def make_cache8(layers, heads, page, dim, block, context, room, seed, *, spare=3, empty=0, spread=1.0):
    """(oracle cache, library cache): sequences with the given committed lengths and room for `room`
    more, their pages scattered over the pool, then `empty` sequences that hold nothing.  Every block
    has a scale of its own; spread: the standard deviation of the logarithms of their sizes."""
    rng = np.random.default_rng(seed)
    held = [-(-(c + room) // page) for c in context]
    S, P, most = len(context) + empty, sum(held) + spare, max(held + [1]) + 1
    order = rng.permutation(P)
    table = np.full((S, most), -1, np.int32)
    refs = np.zeros(P, np.int32)
    at = 0
    for s, n in enumerate(held):
        table[s, :n] = order[at:at + n]
        refs[order[at:at + n]] = 1
        at += n
    shape = (layers, P, heads, page // block)
    parts = []
    for _ in range(2):
        x = rng.normal(0, 1, (*shape, block, dim)) * np.exp(spread * rng.normal(0, 1, (*shape, 1, 1)))
        top = np.abs(x).max((-1, -2))
        e = np.ceil(np.log2(top / 448)).astype(int)
        e += top > 448 * 2.0 ** e
        parts += [dec.round_e4m3(x * 2.0 ** -e[..., None, None]).reshape(layers, P, heads, page, dim),
                  (e + 127).astype(np.uint8)]
    whole = lambda x: np.array(list(x) + [0] * empty, np.int32)  # noqa: E731
    o = dec.Cache8(parts[0], parts[2], table, whole(held), whole(context), refs, parts[1], parts[3])
    return o, device_cache8(o)


def to_e4m3(x):
    """Device tensor of e4m3 numbers given as float32."""
    return dev(torch.from_numpy(np.array(x, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()).view(
        torch.float8_e4m3fn)


def device_cache8(o):
    return wf.PageCache8(to_e4m3(o.k), to_e4m3(o.v), dev(o.k_scale), dev(o.v_scale), i32(o.table), i32(o.held),
                         i32(o.context), i32(o.refs))


def same_cache8(o, cache):
    """The library's cache equals the oracle's, number for number."""
    for name in ("table", "held", "context", "refs", "k_scale", "v_scale"):
        got = getattr(cache, name).cpu().numpy()
        want = getattr(o, name)
        assert np.array_equal(got, want), (name, np.argwhere(got != want)[:5])
    for name in ("k", "v"):
        got = getattr(cache, name).float().cpu().numpy()
        want = getattr(o, name)
        assert np.array_equal(got, want, equal_nan=True), (name, np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:5])


def vectors(total, heads, dim, dtype, seed, scale=1.0, parts=1):
    """`parts` [rows, heads, dim] tensors as slices of one wider projection, and their exact values."""
    x = (np.random.default_rng(seed).normal(0, 1, (total, parts * heads + 1, dim)) * scale).astype(np.float32)
    t = dev(to_bf16(x)) if dtype == "bf16" else dev(x)
    x = bits(to_bf16(x), "bf16") if dtype == "bf16" else x
    cut = [slice(n * heads, (n + 1) * heads) for n in range(parts)]
    return [t[:, c] for c in cut], [x[:, c] for c in cut]


TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def full(shape, value, dtype):
    return torch.full(shape, value, dtype=TORCH[dtype], device=DEV)
