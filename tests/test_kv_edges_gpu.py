"""The key/value cache's calls at the ends of what their arguments may be."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from parity import dev, host
from test_kv_attn_gpu import Case

pytestmark = pytest.mark.gpu

qmm = pytest.importorskip("decode_gemv_qmm_b200")


def test_largest_pages():
    """Pages of 65536 tokens: written, read back and attended to over the end of one."""
    hkv, d, page = 1, 64, 65536
    form = dict(page=page, ktype=0, vtype=1)
    cache = torch.zeros(3, qmm.qmm_kv_page_bytes(hkv, d, **form), dtype=torch.uint8, device="cuda")
    table = np.array([[2, 0]], np.int32)
    n = page + 37
    g = np.random.default_rng(1)
    x = [dev(g.standard_normal((n, hkv, d)).astype(np.float32)) for _ in range(2)]
    pos = np.arange(n)
    slots = dev(table[0, pos // page].astype(np.int64) * page + pos % page)
    qmm.qmm_kv_write(cache, *x, slots, **form)
    k, v = (host(t).astype(np.float64) for t in qmm.qmm_kv_read(cache, slots, hkv, d, **form))
    at = np.array([0, 5, page - 1, page, n - 1])
    small = ref.Cache(1, hkv, d, 16, 0, 1)
    small.write(np.arange(5), *(host(t)[at] for t in x))
    for a, b in zip((k, v), small.read(np.arange(5))):
        assert np.array_equal(a[at], b)
    q = g.standard_normal((1, 2, 3, d)).astype(np.float32)
    y = qmm.qmm_kv_attn(dev(q), cache, dev(table), dev(np.array([n], np.int32)), hkv, **form)
    ref.assert_attention(host(y)[0], ref.attention(q[0].astype(np.float64), k, v, n, d ** -0.5))
    assert qmm.device_status() == 0


@pytest.mark.parametrize("m,hq,hkv,d,dtype", [(8, 128, 1, 64, torch.float32), (8, 128, 1, 256, torch.bfloat16),
                                               (1, 1024, 1024, 64, torch.float32), (2, 1024, 512, 96, torch.bfloat16)])
def test_most_rows_and_heads(m, hq, hkv, d, dtype):
    c = Case([21, 0, 3], m, hq, hkv, d, 1, 0, dtype=dtype, seed=m)
    c.check(c.run())


def test_most_sequences():
    """65536 sequences, most of them empty, the last two not."""
    n, hkv, d = 65536, 2, 64
    form = dict(page=16)
    g = np.random.default_rng(2)
    cache = torch.zeros(6, qmm.qmm_kv_page_bytes(hkv, d, **form), dtype=torch.uint8, device="cuda")
    x = [dev(g.standard_normal((96, hkv, d)).astype(np.float32)) for _ in range(2)]
    slots = torch.arange(96, device="cuda")
    qmm.qmm_kv_write(cache, *x, slots, **form)
    k, v = (host(t).astype(np.float64) for t in qmm.qmm_kv_read(cache, slots, hkv, d, **form))
    lens = np.zeros(n, np.int32)
    held = {0: 20, 1: 1, 255: 7, 256: 32, 40000: 31, n - 2: 17, n - 1: 32}
    for s, ln in held.items():
        lens[s] = ln
    table = np.tile(np.array([[4, 1]], np.int32), (n, 1))
    q = g.standard_normal((n, 1, 4, d)).astype(np.float32)
    y = qmm.qmm_kv_attn(dev(q), cache, dev(table), dev(lens), hkv, **form)
    at = np.concatenate((np.arange(64, 80), np.arange(16, 32)))
    for s, ln in held.items():
        ref.assert_attention(host(y[s]), ref.attention(q[s].astype(np.float64), k[at[:ln]], v[at[:ln]], ln, d ** -0.5), f"{s}")
    empty = torch.ones(n, dtype=torch.bool, device="cuda")
    empty[list(held)] = False
    assert (y[empty] == 0).all() and qmm.device_status() == 0


def test_rows_that_broadcast():
    """One token's rows, or one head's, written to every slot (strides of 0)."""
    g = np.random.default_rng(3)
    hkv, d, t = 3, 64, 20
    slots = torch.arange(t, device="cuda")
    size = qmm.qmm_kv_page_bytes(hkv, d, page=16)
    one = dev(g.standard_normal((1, hkv, d)).astype(np.float32)).expand(t, hkv, d)
    head = dev(g.standard_normal((t, 1, d)).astype(np.float32)).expand(t, hkv, d)
    a, b = (torch.zeros(2, size, dtype=torch.uint8, device="cuda") for _ in range(2))
    qmm.qmm_kv_write(a, one, head, slots, page=16)
    qmm.qmm_kv_write(b, one.contiguous(), head.contiguous(), slots, page=16)
    assert torch.equal(a, b)


def test_one_scratch_for_two_graphs_and_calls_between():
    """Two captured calls that share a scratch, replayed one after the other on two streams, and eager calls between."""
    cases = [Case([3000, 900], 1, 10, 2, 128, 1, 1, page=64, seed=23), Case([1500, 2900, 7], 4, 10, 2, 128, 1, 1, page=64, seed=24)]
    ws = torch.empty(max(qmm.qmm_kv_attn_workspace(len(c.lens), c.m, 10, 2, 128) for c in cases), dtype=torch.uint8, device="cuda")
    want, graphs, outs, keep = [], [], [], []
    for c in cases:
        want.append(c.run())
        t, n = dev(c.table), dev(np.array(c.lens, np.int32))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qmm.qmm_kv_attn(c.qd, c.cache, t, n, 2, ws=ws, scale=c.scale, **c.form))
        graphs.append(g)
        keep.append((t, n))
    streams = [torch.cuda.Stream() for _ in cases]
    for i in range(10):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
            s.synchronize()
            assert torch.equal(cases[i % 2].run(ws=ws), want[i % 2])
            torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_lengths_that_shrink_and_pages_given_back():
    """One captured call whose sequences end, begin again and change places between replays."""
    g = np.random.default_rng(5)
    c = Case([700, 300, 50], 1, 6, 2, 64, 1, 1, page=16, seed=25)
    table, lens = dev(c.table), dev(np.array(c.lens, np.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = qmm.qmm_kv_attn(c.qd, c.cache, table, lens, 2, scale=c.scale, **c.form)
    for _ in range(12):
        perm = g.permutation(3)
        cut = np.array([int(g.integers(0, len(c.kv[s][0]) + 1)) for s in perm])
        table.copy_(dev(c.table[perm]))
        lens.copy_(dev(cut.astype(np.int32)))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for i, s in enumerate(perm):
            k, v = (x[:cut[i]] for x in c.kv[s])
            ref.assert_attention(host(y)[i], ref.attention(c.q[i], k, v, int(cut[i]), c.scale), f"{cut[i]}")
    assert qmm.device_status() == 0
