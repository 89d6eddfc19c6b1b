"""qmm_kv_attn over caches whose values differ widely in size or are not finite: each output against 64-bit attention
over the keys its row sees, with a bound that only those keys enter."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from parity import dev, host
from test_kv_attn_gpu import Case

pytestmark = pytest.mark.gpu

qmm = pytest.importorskip("decode_gemv_qmm_b200")

U = 2.0 ** -24


def refill(c, k, v):
    """Writes other keys and values [tokens, hkv, d] of the one sequence of a case, and takes what the cache then holds."""
    n, page = c.lens[0], c.form["page"]
    pos = np.arange(n)
    c.slots = c.table[0, pos // page].astype(np.int64) * page + pos % page
    qmm.qmm_kv_write(c.cache, dev(k.astype(np.float32)), dev(v.astype(np.float32)), dev(c.slots), **c.form)
    take(c, k.shape[1], k.shape[2])


def take(c, hkv, d):
    c.kv = [tuple(host(t).astype(np.float64) for t in qmm.qmm_kv_read(c.cache, dev(c.slots), hkv, d, **c.form))]


def check_rows(c, y, what=""):
    """Per output, with A = sum p|v| / sum p over the keys the row sees and S the row's largest sum |scale q_d k_jd|:
    (16 u sqrt(D) S + 16 u sqrt(1 + D)) A as kv_reference.assert_attention derives it, and the floor of fp16 terms. There
    a weight's terms lose at most half of fp16's smallest step, 2^-25, where p 2^13 is split and twice where its product
    with d_v is, 2^-38 (d_v + 2) of p d_v's unit; for scales d_v of 2^-7 and more (or brought there by a power of two,
    which goes into both) and a code c that is 2^-38 (1 + 2 / d_v) |c| d_v <= 2^-38 257 |v| < 2^-29 |v|, of every key the
    row sees. bf16: 2^-10 A (weights) and 2^-8 of the output besides. Where a seen value is not finite, what 64 bits give:
    the same infinity, or NaN."""
    y = y.double().cpu().numpy()[0]
    q, (k, v), n = c.q[0], c.kv[0], c.lens[0]
    m, hq, d = q.shape
    ratio = hq // k.shape[1]
    for i in range(m):
        last = n - m + i
        low = max(0, last - c.window + 1) if c.window else 0
        for h in range(hq):
            got = y[i, h]
            if last < low:
                assert (got == 0).all()
                continue
            kk, vv = k[low:last + 1, h // ratio], v[low:last + 1, h // ratio]
            z = kk @ q[i, h] * c.scale
            p = np.exp(z - z.max())
            p /= p.sum()
            with np.errstate(invalid="ignore", over="ignore"):
                out, a = p @ vv, p @ np.abs(vv)
            fine = np.isfinite(vv).all(0)
            # (a product with an infinity in it: column by column, as the formula adds it up)
            for x in np.flatnonzero(~fine):
                with np.errstate(invalid="ignore"):
                    out[x] = (p * vv[:, x]).sum()
            assert np.array_equal(got[~fine], out[~fine], equal_nan=True), (what, i, h, got[~fine], out[~fine])
            s = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(c.scale)
            bound = (16 * U * np.sqrt(d) * s + 16 * U * np.sqrt(1 + d)) * a + 2.0 ** -29 * np.abs(vv).sum(0)
            if c.dtype == torch.bfloat16:
                bound = bound + 2.0 ** -10 * a + 2.0 ** -8 * np.abs(out)
            err = np.abs(np.where(fine, got, 0) - np.where(fine, out, 0))
            bad = fine & ~(err <= bound)
            if bad.any():
                x = int(np.argmax(np.where(bad, err / np.maximum(bound, 1e-300), 0)))
                raise AssertionError(f"{what}: query {i} head {h}: {int(bad.sum())} of {d} outside; dim {x}: {got[x]!r} for "
                                     f"{out[x]!r}, off {err[x]:.3e} of {bound[x]:.3e}")
    assert qmm.device_status() == 0


TYPES = [(0, 0), (1, 1), (0, 1), (1, 0)]


@pytest.mark.parametrize("kt,vt", TYPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,hq,m", [(64, 2, 4), (96, 4, 4), (128, 5, 4), (128, 8, 4), (256, 4, 3)])
def test_infinite_values_reach_only_the_rows_that_see_them(d, hq, m, kt, vt, dtype):
    """A drafted token, and one that a window leaves behind, whose finite values overflow the fp16 scale."""
    g = np.random.default_rng(d + hq + 2 * kt + vt)
    for window in (0, 30):
        for n, big in ((70, [69]), (70, [68, 67]), (300, [299]), (70, [37, 39] if window else [69, 68])):
            c = Case([n], m, hq, 1, d, kt, vt, dtype=dtype, window=window, seed=n)
            k, v = g.standard_normal((n, 1, d)), g.standard_normal((n, 1, d))
            for i, at in enumerate(big):
                v[at, 0, 32 * i:32 * i + 32] *= 1e8
            refill(c, k, v)
            assert not np.isfinite(c.kv[0][1][big]).all()
            check_rows(c, c.run(), f"{n} tokens, {big}, window {window}")


@pytest.mark.parametrize("bits", [0x7c00, 0xfc00, 0x7e00, 0xffff])
@pytest.mark.parametrize("vt", [0, 1])
def test_scales_that_are_not_finite(bits, vt):
    """Infinities of either sign and NaN as a value's scale, in one block of a token that half of the rows see."""
    n, m, d = 90, 4, 128
    c = Case([n], m, 3, 1, d, 1, vt, seed=3)
    g = np.random.default_rng(4)
    refill(c, g.standard_normal((n, 1, d)), g.standard_normal((n, 1, d)))
    plain = ref.Cache(0, 1, d, 16, 1, vt)
    pg, base, t = plain._base(c.slots[n - 2], 0)
    at = base + plain.at[1][2][t, 2]
    c.cache[int(pg), dev(at)] = dev(np.array([bits & 255, bits >> 8], np.uint8))
    take(c, 1, d)
    assert not np.isfinite(c.kv[0][1][n - 2, 0, 64:96]).any() and np.isfinite(c.kv[0][1][n - 2, 0, :64]).all()
    check_rows(c, c.run(), hex(bits))


@pytest.mark.parametrize("vt", [0, 1])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_nothing_but_infinities(d, vt):
    """Every scale that a step holds, alone and between tokens of the usual size."""
    g = np.random.default_rng(2)
    for n, odd in ((1, [0]), (3, [0, 1, 2]), (64, range(64)), (130, range(64, 128)), (131, [130])):
        c = Case([n], 2, 18 if d < 256 else 9, 1, d, 1, vt, seed=n)
        v = g.standard_normal((n, 1, d))
        v[list(odd)] = 1e9 * (1 + g.random((len(odd), 1, d)))
        refill(c, g.standard_normal((n, 1, d)), v)
        check_rows(c, c.run(), f"{n} tokens")


@pytest.mark.parametrize("vt", [0, 1])
@pytest.mark.parametrize("big", [1, 4, 8, 11, 16, 20])
def test_a_large_block_beside_small_ones(big, vt):
    """32 dims 2^big in size, the others 2^-7: each block's outputs are as near as its own values allow."""
    n, d = 150, 128
    g = np.random.default_rng(big)
    for at in (0, 64):
        c = Case([n], 2, 4, 1, d, 1, vt, seed=5)
        v = g.standard_normal((n, 1, d)) * 2.0 ** -7
        v[..., at:at + 32] *= 2.0 ** (big + 7 - (4 if big > 15 else 0))
        refill(c, g.standard_normal((n, 1, d)), v)
        check_rows(c, c.run(), f"2^{big}, dims {at}")


@pytest.mark.parametrize("vt", [0, 1])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 14, 2.0 ** 18])
def test_a_large_token_hidden_from_some_rows(size, vt):
    """The window leaves token 22 to the first two of four rows, or the causal limit the last token to the last row."""
    g = np.random.default_rng(6)
    for window, at in ((40, 22), (0, 63)):
        c = Case([64], 4, 4, 1, 64, 1, vt, window=window, seed=12)
        v = g.standard_normal((64, 1, 64)) * 2.0 ** -8
        v[at] *= size
        refill(c, g.standard_normal((64, 1, 64)), v)
        low = max(0, 63 - window + 1) if window else 0
        assert at < low if window else at > 62
        check_rows(c, c.run(), f"window {window}")


@pytest.mark.parametrize("vt", [0, 1])
@pytest.mark.parametrize("down", [0.0, 4.0, 12.0, 30.0])
def test_a_large_token_of_little_weight(down, vt):
    """Seen by all, 2^22 times the others' size, with a weight of about exp(-down) of theirs."""
    n, d = 64, 128
    g = np.random.default_rng(7)
    c = Case([n], 1, 4, 1, d, 0, vt, seed=8)
    c.qd = torch.ones_like(c.qd)
    c.q = c.qd.double().cpu().numpy()
    k = g.standard_normal((n, 1, d)) * 0.01
    v = g.standard_normal((n, 1, d)) * 2.0 ** -8
    k[30] = -down / d ** 0.5
    v[30] *= 2.0 ** 22
    refill(c, k, v)
    check_rows(c, c.run(), f"down {down}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,hq,m,kt,vt", [(64, 1, 1, 1, 1), (64, 14, 1, 0, 0), (96, 3, 2, 1, 0), (96, 5, 3, 0, 1),
                                           (128, 5, 1, 1, 1), (128, 6, 4, 1, 1), (128, 5, 8, 1, 0), (192, 4, 2, 0, 1),
                                           (256, 4, 1, 1, 1), (256, 3, 8, 0, 0)])
def test_scales_all_over_the_range(d, hq, m, kt, vt, dtype):
    """Every block of every token of a size of its own, from 2^-23 to 2^15, zeros among them; then only some tokens."""
    g = np.random.default_rng(d + hq)
    for n, some in ((33, 1.0), (500, 1.0), (500, 0.05), (2100, 0.01)):
        c = Case([n], m, hq, 1, d, kt, vt, dtype=dtype, window=0 if n < 2000 else 900, seed=n)
        size = 2.0 ** np.where(g.random((n, 1, d // 32, 1)) < some, g.uniform(-20, 15, (n, 1, d // 32, 1)), 0)
        size *= g.random((n, 1, d // 32, 1)) > 0.1
        v = (g.standard_normal((n, 1, d // 32, 32)) * size).reshape(n, 1, d)
        refill(c, g.standard_normal((n, 1, d)), v)
        check_rows(c, c.run(), f"{n} tokens, {some}")


def test_small_values_of_one_size():
    """Scales of one size anywhere in fp16's range, subnormal ones among them: a power of two brings them up."""
    g = np.random.default_rng(9)
    for vt in (0, 1):
        for size in (2.0 ** -17, 2.0 ** -12, 2.0 ** -6, 1.0, 2.0 ** 6, 2.0 ** 13):
            c = Case([200], 2, 5, 1, 128, 1, vt, seed=10)
            refill(c, g.standard_normal((200, 1, 128)), g.standard_normal((200, 1, 128)) * size)
            check_rows(c, c.run(), f"size {size}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("exp", range(16, 33, 2))
def test_steep_scores(exp, sign, dtype):
    """Finite scores up to 2^32: where the largest is far above the others its value is the output."""
    n, hq, d, seen = 200, 6, 128, 0
    for seed in range(4):
        g = np.random.default_rng(100 * exp + seed)
        c = Case([n], 2, hq, 1, d, 0, 1, dtype=dtype, seed=seed)
        size = 2.0 ** (exp / 2)
        refill(c, g.standard_normal((n, 1, d)) * size, g.standard_normal((n, 1, d)))
        q = torch.from_numpy((g.standard_normal((1, 2, hq, d)) * size).astype(np.float32)).to(dtype)
        c.q, c.qd = q.double().numpy(), q.cuda()
        c.scale = sign * d ** -0.5
        y = c.run().double().cpu().numpy()[0]
        assert np.isfinite(y).all()
        k, v = c.kv[0]
        for i in range(2):
            for h in range(hq):
                z = k[:n - 1 + i, 0] @ c.q[0, i, h] * c.scale
                at = np.argsort(z)[-2:]
                # scores are off by 16 u sqrt(D) S at most (check_rows); 40 apart leaves 2^-57 for the rest
                s = (np.abs(k[:n - 1 + i, 0]) @ np.abs(c.q[0, i, h])).max() * abs(c.scale)
                if z[at[1]] - z[at[0]] > 40 + 32 * U * np.sqrt(d) * s:
                    want = v[at[1], 0]
                    seen += 1
                    assert (np.abs(y[i, h] - want) <= (16 * U * np.sqrt(1 + d) + (2.0 ** -8 + 2.0 ** -10 if dtype == torch.bfloat16 else 0)) * np.abs(want) + 2.0 ** -29).all()
    assert seen > 10
    assert qmm.device_status() == 0


@pytest.mark.parametrize("kt", [0, 1])
@pytest.mark.parametrize("bits", [0x7c00, 0xfc00, 0x7e00])
def test_key_scales_that_are_not_finite_stay_with_their_rows(bits, kt):
    """A key that only the last two of four rows see, and one that the window leaves to the first."""
    n, m, d = 90, 4, 128
    for window, at, rows in ((0, n - 2, (0, 1)), (40, n - m - 39, (1, 2, 3))):
        c = Case([n], m, 3, 1, d, kt, 1, seed=3, window=window)
        g = np.random.default_rng(4)
        refill(c, g.standard_normal((n, 1, d)), g.standard_normal((n, 1, d)))
        plain = ref.Cache(0, 1, d, 16, kt, 1)
        pg, base, t = plain._base(c.slots[at], 0)
        c.cache[int(pg), dev(base + plain.at[0][2][t, 1])] = dev(np.array([bits & 255, bits >> 8], np.uint8))
        y = c.run().double().cpu().numpy()[0]
        want = ref.attention(c.q[0], *c.kv[0], n, c.scale, window)    # (of the finite key: the rows below do not see it)
        for i in rows:
            ref.assert_attention(y[i:i + 1], tuple(x[i:i + 1] if isinstance(x, np.ndarray) and x.ndim else x for x in want), f"row {i}")
    assert qmm.device_status() == 0
