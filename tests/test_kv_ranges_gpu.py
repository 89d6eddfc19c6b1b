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
    a weight p d_v is off by less than 2^-36 for scales d_v in [2^-7, 2) (and where scales are brought there by a power
    of two, that much of it); a code c makes that 2^-36 |c| <= 2^-29 |c| d_v = 2^-29 |v|, of every key the row sees. bf16:
    2^-10 A (weights) and 2^-8 of the output besides. Where a seen value is not finite, what 64 bits give: the same
    infinity, or NaN."""
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
