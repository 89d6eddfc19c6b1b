"""The quantised key/value cache in plain numpy and 64 bits: what the tests compare with.

Written from the definitions in include/qmm.h (block rules, byte layout,
attention formula), without the library. ggml's block rules are binary32 steps,
so the quantiser is numpy float32; everything else is float64.
"""
from __future__ import annotations

import numpy as np

Q8, Q4 = 0, 1
BLOCK, GROUP = 32, 16


def part_bytes(d, qt):
    return GROUP * (d if qt == Q8 else d // 2) + GROUP * (d // BLOCK) * 2


def page_bytes(hkv, d, page, kt, vt):
    return hkv * (page // GROUP) * (part_bytes(d, kt) + part_bytes(d, vt))


def runs(nb, qt):
    """(first, n) of every block, as the header lays them out: 4 (Q4_0) or 2 (Q8_0) together, then 2, then 1."""
    out, first = [], 0
    for n in (4, 2, 1) if qt == Q4 else (2, 1):
        while nb - first >= n:
            out += [(first, n)] * n
            first += n
    return out


def code_place(d, qt, val, tok, b, x):
    """Byte offset in a group's part of code byte x of block b of token tok: the header's formula."""
    first, n = runs(d // BLOCK, qt)[b]
    if not val:
        row = 8 * (tok // 8) + 2 * (tok % 4) + tok // 4 % 2
        if qt == Q8:
            return 512 * first + ((4 * row + x % 16 // 4) * n + b - first) * 8 + x // 16 * 4 + x % 4
        return 256 * first + ((4 * row + x // 4) * n + b - first) * 4 + x % 4
    u, g = (4 if qt == Q8 else 2), x % 16 // 2
    c = (64 * (g // 4) + 4 * tok + g % 4) * 8 if n * u == 8 else (8 * tok + g) * n * u
    return 128 * u * first + c + (b - first) * u + x // 16 * 2 + x % 2


def scale_place(d, qt, tok, b):
    return GROUP * (d if qt == Q8 else d // 2) + (tok % 4 * (d // BLOCK) + b) * 8 + tok // 4 * 2


def quantise(x, qt):
    """float32 [..., d] -> (code bytes uint8 [..., nb, 32 or 16], scales float16 [..., nb])."""
    f = np.float32
    x = np.ascontiguousarray(x, dtype=f).reshape(*x.shape[:-1], -1, BLOCK)
    top = np.take_along_axis(x, np.abs(x).argmax(-1)[..., None], -1)  # argmax: the first of the largest
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        d = np.abs(top) / f(127) if qt == Q8 else top / f(-8)
        inv = np.where(d != 0, f(1) / d, f(0)).astype(f)
        y = (x * inv).astype(f)
        scale = d[..., 0].astype(np.float16)
    if qt == Q8:
        q = np.copysign(np.floor(np.abs(y.astype(np.float64)) + 0.5), y).clip(-127, 127).astype(np.int8)
        return q.view(np.uint8), scale
    q = np.floor((y + f(8.5)).astype(f)).clip(0, 15).astype(np.uint8)
    return q[..., :16] | (q[..., 16:] << 4), scale


def values(codes, scale, qt):
    """float64 [..., d]."""
    if qt == Q8:
        q = codes.view(np.int8).astype(np.float64)
    else:
        q = np.concatenate((codes & 15, codes >> 4), -1).astype(np.float64) - 8
    v = q * scale.astype(np.float64)[..., None]
    return v.reshape(*v.shape[:-2], -1)


class Cache:
    """A cache held as bytes in the documented layout, written and read byte by byte."""

    def __init__(self, pages, hkv, d, page, kt, vt, fill=0):
        self.hkv, self.d, self.page, self.kt, self.vt = hkv, d, page, kt, vt
        self.bytes = np.full((pages, page_bytes(hkv, d, page, kt, vt)), fill, dtype=np.uint8)
        nb = d // BLOCK
        self.at = []
        for val, qt in ((False, kt), (True, vt)):
            start = part_bytes(d, kt) if val else 0
            n = 32 if qt == Q8 else 16
            code = np.array([[[start + code_place(d, qt, val, t, b, x) for x in range(n)] for b in range(nb)]
                             for t in range(GROUP)])
            scale = np.array([[start + scale_place(d, qt, t, b) for b in range(nb)] for t in range(GROUP)])
            self.at.append((qt, code, np.stack((scale, scale + 1), -1)))

    def _base(self, slot, head):
        pg, place = divmod(int(slot), self.page)
        size = part_bytes(self.d, self.kt) + part_bytes(self.d, self.vt)
        return pg, (head * (self.page // GROUP) + place // GROUP) * size, place % GROUP

    def write(self, slots, k, v):
        for (qt, code, scale), x in zip(self.at, (k, v)):
            codes, d = quantise(x, qt)
            for i, s in enumerate(slots):
                if s < 0:
                    continue
                for h in range(self.hkv):
                    pg, base, t = self._base(s, h)
                    self.bytes[pg, base + code[t]] = codes[i, h]
                    self.bytes[pg, base + scale[t]] = d[i, h][:, None].view(np.uint8)

    def read(self, slots):
        """float64 (K, V) [T, hkv, d]."""
        out = []
        for qt, code, scale in self.at:
            rows = np.zeros((len(slots), self.hkv, self.d))
            for i, s in enumerate(slots):
                for h in range(self.hkv):
                    pg, base, t = self._base(s, h)
                    d = np.ascontiguousarray(self.bytes[pg, base + scale[t]]).view(np.float16)[:, 0]
                    rows[i, h] = values(self.bytes[pg, base + code[t]], d, qt)
            out.append(rows)
        return out


def attention(q, k, v, length, scale, window=0):
    """One sequence. q [M, Hq, d], k, v [length, Hkv, d], all float64 -> (out, A, S, floor): the result, sum p|v| / sum p
    per output, per row the largest sum |scale q_d k_jd| over its keys, and the weights' floor (assert_attention)."""
    m, hq, d = q.shape
    out, a, s = np.zeros(q.shape), np.zeros(q.shape), np.zeros((m, hq, 1))
    floor = np.abs(v).max(initial=0.0) * min(len(v) * 2.0 ** -28, np.sqrt(len(v)) * 2.0 ** -25)
    ratio = hq // (k.shape[1] if k.ndim == 3 else 1)
    for i in range(m):
        last = length - m + i
        low = max(0, last - window + 1) if window else 0
        if last < low:
            continue
        for h in range(hq):
            kk, vv = k[low:last + 1, h // ratio], v[low:last + 1, h // ratio]
            z = kk @ q[i, h] * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h], a[i, h] = p @ vv, p @ np.abs(vv)
            s[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, a, s, floor


def assert_attention(got, ref, what="", bf16=False):
    """fp32 against 64 bits.

    A score is a sum of D products; its roundings (u = 2^-24 each, of terms whose
    magnitudes sum to S) add up like a random walk, about sqrt(D) u S, and 8 times
    that covers the largest of the many scores of a case. A score that is off by e
    turns its weight by the factor exp(e); after the division an output is off by
    at most 2 e A, A = sum p|v| / sum p. The exponentials, the sums over the keys,
    the division and the two-term products (22 bits: 2^-23 each) add at most
    16 u sqrt(1 + D) A to that in the same sense. Over a whole output the errors
    do not line up: its 2-norm is held to 1e-5 of A's, the library's fp32
    tolerance. With bf16 queries the weights p and their products p d_v are rounded
    to fp16, 2^-11 of each and so 2^-10 A, and the outputs to bf16, 2^-8 of the
    value.

    The weights p d_v 2^13 are held as fp16 terms. fp16's smallest step is 2^-24,
    and the terms lose at most half of one where p is split and twice half of one
    where the product is: less than 2^-23 (d_v < 2). The largest d_v of the keys
    taken together is 2^-7 at least, by a power of two where need be, so that
    is 2^-23 / 2^(13 - 7) = 2^-29 of the largest d_v at most, and with a code c
    2^-29 |c| max d_v <= 2^-29 128/127 max|v| (the largest |c| is 8 or 127 and
    belongs to the largest |v| of its block). Each of the keys may add one such
    error to an output, and sum p >= 1 divides them: F 2^-28 with F = keys *
    max|v| is the bound. It lines up nowhere: as above, 8 sqrt(keys) of them are
    taken, F / sqrt(keys) 2^-25, where that is less.
    """
    out, a, s, floor = ref
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == out.shape, (what, got.shape, out.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite outputs"
    u, d = 2.0 ** -24, got.shape[-1]
    bound = (16 * u * np.sqrt(d) * s + 16 * u * np.sqrt(1 + d)) * a + floor + (2.0 ** -10 * a + 2.0 ** -8 * np.abs(out) if bf16 else 0)
    err = np.abs(got - out)
    bad = err > bound
    if bad.any():
        i = np.unravel_index(np.argmax(err - bound), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outputs outside; worst at {i}: {got[i]!r} for "
                             f"{out[i]!r}, off {err[i]:.3e} of {bound[i]:.3e}")
    if not bf16:
        off, norm = np.linalg.norm(got - out), np.linalg.norm(a)
        assert off <= 1e-5 * norm, f"{what}: off by {off / norm:.2e} of the norm"
