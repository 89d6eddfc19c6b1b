"""qmm_kv_attn against 64-bit attention over the values that the cache holds."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from parity import dev, host

pytestmark = pytest.mark.gpu

qmm = pytest.importorskip("decode_gemv_qmm_b200")


class Case:
    """A filled cache, page tables and queries; every unused byte of the cache is `junk`."""

    def __init__(self, lens, m, hq, hkv, d, kt, vt, page=16, dtype=torch.float32, window=0, seed=0, spread=1.0, junk=0xFF):
        g = np.random.default_rng(seed)
        self.lens, self.m, self.hkv, self.window, self.dtype = list(lens), m, hkv, window, dtype
        self.form = dict(page=page, ktype=kt, vtype=vt)
        held = [-(-n // page) for n in lens]
        pages = sum(held) + 1
        size = qmm.qmm_kv_page_bytes(hkv, d, **self.form)
        # 0xFF bytes are NaN scales: nothing outside the tokens may be used
        self.cache = torch.full((pages, size), junk, dtype=torch.uint8, device="cuda")
        order, at = g.permutation(pages), 0
        self.table = np.full((len(lens), max(held + [1]) + 1), -1, np.int32)
        self.kv, slots = [], []
        for s, n in enumerate(lens):
            self.table[s, :held[s]] = order[at:at + held[s]]
            at += held[s]
            pos = np.arange(n)
            slots.append((self.table[s, pos // page].astype(np.int64) * page + pos % page))
        slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
        x = [torch.from_numpy(g.standard_normal((len(slots), hkv, d)).astype(np.float32)
                              * np.exp(0.4 * g.standard_normal((1, hkv, d))).astype(np.float32)) for _ in range(2)]
        qmm.qmm_kv_write(self.cache, x[0].cuda(), x[1].cuda(), dev(slots), **self.form)
        k, v = (host(t).astype(np.float64) for t in
                qmm.qmm_kv_read(self.cache, dev(slots), hkv, d, **self.form))
        at = 0
        for n in lens:
            self.kv.append((k[at:at + n], v[at:at + n]))
            at += n
        q = torch.from_numpy((g.standard_normal((len(lens), m, hq, d)) * 1.5 * spread).astype(np.float32)).to(dtype)
        self.q, self.qd = q.double().numpy(), q.cuda()
        self.scale = d ** -0.5

    def run(self, **kw):
        a = dict(scale=self.scale, window=self.window) | kw
        return qmm.qmm_kv_attn(self.qd, self.cache, dev(self.table), dev(np.array(self.lens, np.int32)), self.hkv,
                               **a, **self.form)

    def check(self, y, what=""):
        y = y.double().cpu().numpy()
        for s, n in enumerate(self.lens):
            want = ref.attention(self.q[s], *self.kv[s], n, self.scale, self.window)
            ref.assert_attention(y[s], want, f"{what} sequence {s} of {n}", self.dtype == torch.bfloat16)
        assert qmm.device_status() == 0


TYPES = [(0, 0), (1, 1), (0, 1), (1, 0)]


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kt,vt", TYPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_types_and_head_sizes(d, kt, vt, dtype):
    c = Case([70, 1, 33], 1, 10, 2, d, kt, vt, dtype=dtype, seed=d + kt)
    c.check(c.run())


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4097])
def test_lengths(n):
    """Around the ends of groups, pages and tiles, and none at all."""
    c = Case([n], 1, 14, 2, 64, 1, 1, page=64, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 6), (4, 2), (10, 2), (14, 2), (8, 1), (9, 1), (16, 1), (33, 1), (71, 1)])
def test_queries_and_ratios(m, hq, hkv):
    """Every sequence's first queries see no key where it is shorter than M."""
    c = Case([5, 40, 0, 1, 131], m, hq, hkv, 64, 1, 0, seed=m * 100 + hq)
    y = c.run()
    c.check(y)
    assert (y[2] == 0).all()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1 << 20, 1 << 40])
@pytest.mark.parametrize("m", [1, 5])
def test_windows(window, m):
    c = Case([3, 16, 130, 517], m, 8, 2, 128, 0, 1, page=32, window=window, seed=window % 1000)
    c.check(c.run())


@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
def test_pages(page):
    c = Case([1, 16, 100, 700, 2049], 2, 10, 2, 128, 1, 1, page=page, seed=page)
    c.check(c.run())


def test_many_sequences_of_uneven_lengths():
    g = np.random.default_rng(3)
    c = Case([int(n) for n in np.exp(g.uniform(0, 7.5, 100))] + [0, 0, 3], 1, 8, 2, 64, 1, 1, page=16)
    c.check(c.run())


@pytest.mark.parametrize("n,hkv,d,kt", [(33, 1, 64, 1), (257, 1, 64, 1), (700, 2, 64, 1), (300, 1, 256, 0), (129, 2, 256, 0)])
def test_more_sequences_than_lanes_and_threads(n, hkv, d, kt):
    """Sequences are looked up by lanes, then threads, then several a thread; empty ones lie in between."""
    g = np.random.default_rng(n)
    c = Case([int(v) for v in g.integers(0, 40, n) * g.integers(0, 2, n)], 1, hkv * 3, hkv, d, kt, kt, page=16, seed=n)
    y = c.run()
    c.check(y)
    for s in range(n):
        if not c.lens[s]:
            assert (y[s] == 0).all()


@pytest.mark.parametrize("batch", [1, 3, 40])
def test_no_keys_anywhere(batch):
    c = Case([0] * batch, 2, 4, 2, 64, 1, 1)
    y = torch.full((batch, 2, 4, 64), float("nan"), device="cuda")
    c.run(Y=y)
    assert (y == 0).all() and qmm.device_status() == 0


def test_one_scratch_for_calls_of_different_sizes():
    """A scratch that other calls have used, larger and smaller, and one filled with ones or zeros."""
    a = Case([4000, 10, 900], 1, 10, 2, 128, 1, 1, page=64, seed=21)
    b = Case([700], 4, 16, 2, 128, 1, 1, page=64, seed=22, dtype=torch.bfloat16)
    ws = torch.full((max(qmm.qmm_kv_attn_workspace(3, 1, 10, 2, 128), qmm.qmm_kv_attn_workspace(1, 4, 16, 2, 128)),), 255,
                    dtype=torch.uint8, device="cuda")
    wa, wb = a.run(), b.run()
    for _ in range(3):
        assert torch.equal(a.run(ws=ws), wa) and torch.equal(b.run(ws=ws), wb)
    ws.zero_()
    assert torch.equal(b.run(ws=ws), wb) and torch.equal(a.run(ws=ws), wa)


def test_two_graphs_replayed_at_once():
    """Each with the scratch of its own capture; replayed side by side on two streams, again and again."""
    cases = [Case([3000, 900], 1, 10, 2, 128, 1, 1, page=64, seed=23), Case([1500, 2900], 1, 10, 2, 128, 1, 1, page=64, seed=24)]
    want, graphs, outs, keep = [], [], [], []
    for c in cases:
        want.append(c.run())
        t, n = dev(c.table), dev(np.array(c.lens, np.int32))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qmm.qmm_kv_attn(c.qd, c.cache, t, n, 2, scale=c.scale, **c.form))
        graphs.append(g)
        keep.append((t, n))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_first_call_of_a_process_is_captured():
    """Nothing has to run before a capture."""
    import subprocess
    import sys
    code = """
import torch, decode_gemv_qmm_b200 as qmm
f = dict(page=16)
cache = torch.zeros(4, qmm.qmm_kv_page_bytes(2, 64, **f), dtype=torch.uint8, device="cuda")
x = torch.randn(20, 2, 64, device="cuda"); slots = torch.arange(20, device="cuda")
q = torch.randn(1, 1, 4, 64, device="cuda"); lens = torch.full((1,), 20, dtype=torch.int32, device="cuda")
table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    qmm.qmm_kv_write(cache, x, x, slots, **f)
    k, v = qmm.qmm_kv_read(cache, slots, 2, 64, **f)
    y = qmm.qmm_kv_attn(q, cache, table, lens, 2, **f)
g.replay(); torch.cuda.synchronize()
w = torch.softmax(torch.einsum("hd,nhd->hn", q[0, 0].double(), k.repeat_interleave(2, 1).double()) / 8, -1)
assert torch.allclose(y[0, 0].double(), torch.einsum("hn,nhd->hd", w, v.repeat_interleave(2, 1).double()), atol=1e-5)
assert qmm.device_status() == 0
print("ok")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_calls_from_threads_on_streams_of_their_own():
    import threading
    cases = [Case([500 + 300 * i, 20], 1, 10, 2, 128, 1, 1, page=64, seed=40 + i) for i in range(3)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        c, s = cases[i], torch.cuda.Stream()
        t, n = dev(c.table), dev(np.array(c.lens, np.int32))
        torch.cuda.synchronize()
        for _ in range(20):
            y = qmm.qmm_kv_attn(c.qd, c.cache, t, n, 2, scale=c.scale, stream=s, **c.form)
            s.synchronize()
            if not torch.equal(y, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("d,kt,vt,n", [(128, 1, 1, 40000), (64, 0, 0, 30011), (256, 1, 0, 9000)])
def test_long_context_of_one_sequence(d, kt, vt, n):
    c = Case([n], 1, 5, 1, d, kt, vt, page=64, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("m,hq,hkv,d", [(8, 64, 4, 128), (8, 16, 2, 256), (3, 40, 8, 128)])
def test_long_contexts_with_many_rows(m, hq, hkv, d):
    c = Case([3000, 777, 2], m, hq, hkv, d, 1, 1, page=64, dtype=torch.bfloat16, seed=m)
    c.check(c.run())


def test_peaked_and_flat_scores():
    for spread in (0.0, 1e-3, 30.0):          # equal weights; one key that takes all
        c = Case([300, 2000], 1, 7, 1, 128, 1, 1, spread=spread, seed=4)
        c.check(c.run(), f"spread {spread}")


def test_small_and_large_values():
    """Scales of the values over the whole range of fp16, keys and queries large and small in turn."""
    for kv, q in ((2.0 ** -18, 2.0 ** 10), (2.0 ** 10, 2.0 ** -12), (1.0, 1e-30), (1e-3, 1e3)):
        c = Case([150], 1, 4, 1, 64, 1, 0, seed=11)
        x = [torch.randn(150, 1, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(k)) * kv for k in (1, 2)]
        pos = np.arange(150)
        slots = dev(c.table[0, pos // 16].astype(np.int64) * 16 + pos % 16)
        qmm.qmm_kv_write(c.cache, *x, slots, **c.form)
        c.kv = [tuple(host(t).astype(np.float64) for t in qmm.qmm_kv_read(c.cache, slots, 1, 64, **c.form))]
        c.qd = c.qd * q
        c.q = c.qd.double().cpu().numpy()
        c.check(c.run(), f"kv {kv} q {q}")


def test_values_of_uneven_scale_in_one_sequence():
    """One token whose values are 2^20 times the others', seen by some rows and hidden from others by the window."""
    c = Case([64], 4, 4, 1, 64, 1, 1, window=40, seed=12)
    x = torch.randn(64, 1, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(5)) * 2.0 ** -8
    x[24] *= 2.0 ** 20
    pos = np.arange(64)
    slots = dev(c.table[0, pos // 16].astype(np.int64) * 16 + pos % 16)
    k = torch.randn(64, 1, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    qmm.qmm_kv_write(c.cache, k, x, slots, **c.form)
    c.kv = [tuple(host(t).astype(np.float64) for t in qmm.qmm_kv_read(c.cache, slots, 1, 64, **c.form))]
    c.check(c.run())


def test_scale_of_either_sign_and_zero():
    c = Case([90], 1, 4, 2, 64, 0, 0, seed=5)
    for scale in (-0.3, 0.0, 2.0, 1e-20):
        c.scale = scale
        c.check(c.run(), f"scale {scale}")


def test_query_rows_of_zeros():
    """With any scale: equal weights over the keys a row sees, whatever lies behind them."""
    for dtype in (torch.float32, torch.bfloat16):
        c = Case([37, 5], 3, 4, 2, 64, 1, 0, seed=17, dtype=dtype)
        c.qd = c.qd.clone()
        c.qd[:, :, ::2] = 0
        c.q = c.qd.double().cpu().numpy()
        for scale in (0.125, 1e-12, 1e-38, -1e-30, 0.0):
            c.scale = scale
            c.check(c.run(), f"scale {scale}")


def test_strided_queries_and_tables():
    c = Case([50, 20, 80], 2, 6, 2, 64, 1, 1, seed=6)
    want = c.run()
    y = torch.zeros(3, 2, 10 * 64, device="cuda")
    y[..., : 6 * 64] = c.qd.flatten(2)
    c.qd = y[..., : 6 * 64].unflatten(2, (6, 64))                       # a slice of the fused projection
    assert torch.equal(c.run(), want)
    c.qd = c.qd.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)   # heads outermost
    assert torch.equal(c.run(), want)
    wide = np.full((3, 40), -1, np.int32)
    wide[:, : c.table.shape[1]] = c.table
    got = qmm.qmm_kv_attn(c.qd, c.cache, dev(wide)[:, : c.table.shape[1]], dev(np.array(c.lens, np.int32)), 2,
                          scale=c.scale, **c.form)
    assert torch.equal(got, want)


def test_pages_shared_by_sequences_and_repeated():
    c = Case([64], 1, 4, 2, 64, 1, 1, page=16, seed=7)
    c.check(c.run())
    t = c.table.copy()
    c.qd = c.qd.expand(3, -1, -1, -1)                                  # a common prefix, queries alike (stride 0)
    c.q, c.kv = np.repeat(c.q, 3, 0), c.kv * 3
    c.table, c.lens = np.repeat(c.table, 3, 0), [64, 64, 64]
    c.check(c.run())                                                   # (how a sequence is split goes by the whole call)
    t[0, 1] = t[0, 0]                                                  # the same page twice in a sequence
    c2 = Case([64], 1, 4, 2, 64, 1, 1, page=16, seed=7)
    k, v = c2.kv[0]
    c2.kv = [(np.concatenate((k[:16], k[:16], k[32:])), np.concatenate((v[:16], v[:16], v[32:])))]
    c2.table = t
    c2.check(c2.run())


def test_bad_pages_and_lengths_are_left_out_and_recorded():
    c = Case([60, 30], 1, 4, 2, 64, 1, 1, page=16, seed=8)
    k, v = c.kv[0]
    pages = c.cache.shape[0]
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        c.table[0, 1] = bad                                            # positions 16..31 do not exist
        y = c.run()
        assert qmm.device_status() == 8
        want = ref.attention(c.q[0], np.delete(k, np.s_[16:32], 0), np.delete(v, np.s_[16:32], 0), 44, c.scale)
        ref.assert_attention(host(y)[0], want)
        ref.assert_attention(host(y)[1], ref.attention(c.q[1], *c.kv[1], 30, c.scale))
    c.table[0, :] = -1                                                 # no page at all
    y = c.run()
    assert qmm.device_status() == 8 and (y[0] == 0).all()
    c.lens = [-5, 30]                                                  # taken as 0
    y = c.run()
    assert qmm.device_status() == 8 and (y[0] == 0).all()
    ref.assert_attention(host(y)[1], ref.attention(c.q[1], *c.kv[1], 30, c.scale))
    d = Case([64, 64], 1, 4, 2, 64, 1, 1, page=16, seed=9)
    d.table = d.table[:, :4].copy()
    want = d.run()
    d.lens = [10 ** 9, 64]                                             # taken as the table's 64
    y = d.run()
    assert qmm.device_status() == 8 and torch.equal(y, want)


def test_nothing_behind_the_length_is_used():
    """The same result whatever lies behind the last token, in its group, page and further pages."""
    for n in (1, 17, 50, 64):
        got = []
        for junk in (0x00, 0xFF, 0x7C):
            c = Case([n], 1, 5, 1, 128, 0, 1, page=64, seed=10, junk=junk)
            c.table[:] = np.where(c.table < 0, c.cache.shape[0] - 1, c.table)
            got.append(c.run())
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_no_cache_and_empty_calls():
    form = dict(page=16)
    size = qmm.qmm_kv_page_bytes(2, 64, **form)
    q = torch.randn(2, 1, 4, 64, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = qmm.qmm_kv_attn(q, torch.zeros(0, size, dtype=torch.uint8, device="cuda"),
                        torch.zeros(2, 0, dtype=torch.int32, device="cuda"), lens, 2, **form)
    assert (y == 0).all() and qmm.device_status() == 0
    e = qmm.qmm_kv_attn(q[:0], torch.zeros(1, size, dtype=torch.uint8, device="cuda"),
                        torch.zeros(0, 3, dtype=torch.int32, device="cuda"), lens[:0], 2, **form)
    assert e.shape == (0, 1, 4, 64)
    e = qmm.qmm_kv_attn(q[:, :0], torch.zeros(1, size, dtype=torch.uint8, device="cuda"),
                        torch.zeros(2, 3, dtype=torch.int32, device="cuda"), lens, 2, **form)
    assert e.shape == (2, 0, 4, 64)


def test_same_result_every_time():
    c = Case([5000, 100, 2500], 2, 10, 2, 128, 1, 1, page=64, seed=13)
    want = c.run()
    for _ in range(5):
        assert torch.equal(c.run(), want)


def test_two_streams_at_once():
    """Two calls at once, each with a workspace of its own (the default)."""
    a = Case([3000, 900], 1, 10, 2, 128, 1, 1, page=64, seed=14)
    b = Case([1500, 2900], 1, 10, 2, 128, 1, 1, page=64, seed=15)
    wa, wb = a.run(), b.run()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    table = [dev(c.table) for c in (a, b)]
    lens = [dev(np.array(c.lens, np.int32)) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        ya = qmm.qmm_kv_attn(a.qd, a.cache, table[0], lens[0], 2, scale=a.scale, stream=sa, **a.form)
        yb = qmm.qmm_kv_attn(b.qd, b.cache, table[1], lens[1], 2, scale=b.scale, stream=sb.cuda_stream, **b.form)
        torch.cuda.synchronize()
        assert torch.equal(ya, wa) and torch.equal(yb, wb)


def test_captured_step_replays_with_new_lengths_and_tokens():
    """Projection, write, attention, output projection: a decode step as it is used, captured once and replayed as the
    sequences grow; each step against the plain cache and 64-bit attention, and the last product against the library's
    own on those attention outputs."""
    import synthetic as syn
    g = syn.rng(20)
    hq, hkv, d, page, nseq, steps = 14, 2, 64, 16, 3, 20
    k = 896
    wqkv = dev(syn.q8_0_weights(g, (hq + 2 * hkv) * d, k, dscale=1.0 / (73.6 * k ** 0.5))[0])
    wo = dev(syn.q8_0_weights(g, k, hq * d, dscale=1.0 / (73.6 * k ** 0.5))[0])
    form = dict(page=page, ktype=0, vtype=1)
    cache = torch.full((12, qmm.qmm_kv_page_bytes(hkv, d, **form)), 0xFF, dtype=torch.uint8, device="cuda")
    plain = ref.Cache(12, hkv, d, page, 0, 1, fill=0xFF)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    x, slots = torch.zeros(nseq, k, device="cuda"), torch.full((nseq,), -1, dtype=torch.int64, device="cuda")
    lens, tab = torch.zeros(nseq, dtype=torch.int32, device="cuda"), dev(table)
    y = torch.zeros(nseq, (hq + 2 * hkv) * d, device="cuda")
    z, out = torch.zeros(nseq, 1, hq, d, device="cuda"), torch.zeros(nseq, k, device="cuda")
    ws = torch.empty(qmm.qmm_kv_attn_workspace(nseq, 1, hq, hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        qmm.qmm_q8_gemv(wqkv, x, (hq + 2 * hkv) * d, y)
        qkv = y.unflatten(1, (hq + 2 * hkv, d))
        qmm.qmm_kv_write(cache, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], slots, **form)
        qmm.qmm_kv_attn(qkv[:, :hq].unsqueeze(1), cache, tab, lens, hkv, z, ws, **form)
        qmm.qmm_q8_gemv(wo, z.view(nseq, hq * d), k, out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    start = np.array([0, 5, 40])
    pre = g.standard_normal((45, hkv, d)).astype(np.float32)
    pre_slots = np.concatenate((table[1, 0] * page + np.arange(5), table[2][np.arange(40) // page] * page + np.arange(40) % page))
    qmm.qmm_kv_write(cache, dev(pre), dev(pre), dev(pre_slots.astype(np.int64)), **form)
    plain.write(pre_slots, pre, pre)
    for i in range(steps):
        at = start + i
        s = table[np.arange(3), at // page].astype(np.int64) * page + at % page
        x.copy_(dev(g.standard_normal((nseq, k)).astype(np.float32)))
        slots.copy_(dev(s))
        lens.copy_(dev((at + 1).astype(np.int32)))
        z.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        qkv = host(y).reshape(nseq, hq + 2 * hkv, d)
        plain.write(s, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:])
        assert np.array_equal(host(cache), plain.bytes), i
        for n in range(nseq):
            pos = np.arange(at[n] + 1)
            kk, vv = plain.read(table[n, pos // page].astype(np.int64) * page + pos % page)
            want = ref.attention(qkv[n:n + 1, :hq].astype(np.float64), kk, vv, int(at[n]) + 1, d ** -0.5)
            ref.assert_attention(host(z)[n], want, f"step {i} sequence {n}")
        assert torch.equal(out, qmm.qmm_q8_gemv(wo, z.view(nseq, hq * d).clone(), k))
    assert qmm.device_status() == 0


def test_workspace_too_small_is_refused():
    c = Case([100], 1, 4, 2, 64, 1, 1)
    need = qmm.qmm_kv_attn_workspace(1, 1, 4, 2, 64)
    with pytest.raises(qmm.QmmError) as e:
        c.run(ws=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == qmm.QMM_ERR_SHAPE
    c.check(c.run(ws=torch.empty(need, dtype=torch.uint8, device="cuda")))


def test_offsets_past_32_bits():
    """Pages behind the first 4 GiB of the cache."""
    form = dict(page=64)
    size = qmm.qmm_kv_page_bytes(8, 128, **form)
    pages = (1 << 32) // size + 8
    c = Case([130], 1, 8, 8, 128, 1, 1, page=64, seed=16)
    big = torch.empty(pages, size, dtype=torch.uint8, device="cuda")
    big[pages - c.cache.shape[0]:] = c.cache
    want = c.run()
    c.table = np.where(c.table >= 0, c.table + pages - c.cache.shape[0], c.table).astype(np.int32)
    c.cache = big
    assert torch.equal(c.run(), want)
