"""qmm_kv_write and qmm_kv_read against the plain cache (bytes and values bit for bit)."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from parity import dev, host

pytestmark = pytest.mark.gpu

qmm = pytest.importorskip("decode_gemv_qmm_b200")


def rows(g, t, hkv, d, dtype):
    """fp32 values of the element type, zero and extreme blocks among them, as numpy and on the device."""
    x = g.standard_normal((t, hkv, d)).astype(np.float32) * np.exp(g.standard_normal((t, hkv, 1))).astype(np.float32)
    if t > 2:
        x[0, 0, :32] = 0.0
        x[1, 0, :32] = np.where(np.arange(32) % 2, -3.0, 3.0)     # ties: the first of the largest decides
        x[2, -1, -32:] = np.arange(-16, 16) + 0.5                 # halves
        x[2, 0, :32] *= np.float32(2.0 ** -20)                    # subnormal scales
    xt = torch.from_numpy(x).to(dtype)
    return xt.float().numpy(), xt.cuda()


def scatter(g, t, pages, page):
    return g.permutation(pages * page)[:t].astype(np.int64)


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kt,vt", [(0, 0), (1, 1), (0, 1), (1, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_write_then_read(d, kt, vt, dtype):
    g = np.random.default_rng(d + 2 * kt + vt)
    t, hkv, page, pages = 37, 3, 16, 5
    k, kd = rows(g, t, hkv, d, dtype)
    v, vd = rows(g, t, hkv, d, dtype)
    slots = scatter(g, t, pages, page)
    plain = ref.Cache(pages, hkv, d, page, kt, vt, fill=0xA5)
    cache = dev(plain.bytes)
    form = dict(page=page, ktype=kt, vtype=vt)
    qmm.qmm_kv_write(cache, kd, vd, dev(slots), **form)
    plain.write(slots, k, v)
    assert np.array_equal(host(cache), plain.bytes)          # the tokens' bytes, and no other
    want = plain.read(slots)
    got = qmm.qmm_kv_read(cache, dev(slots), hkv, d, dtype=dtype, **form)
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), torch.from_numpy(b).float().to(dtype))
    assert qmm.device_status() == 0


@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 63, 64, 65, 300])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_prompts_of_any_length(t, page):
    """Runs of consecutive slots that begin and end inside a group, pages in any order."""
    g = np.random.default_rng(t + page)
    hkv, d = 2, 128
    for first in (0, 5):
        held = -(-(t + first) // page)
        order = g.permutation(held + 2)
        at = np.arange(first, first + t)
        slots = (order[at // page] * page + at % page).astype(np.int64)
        plain = ref.Cache(held + 2, hkv, d, page, ref.Q8, ref.Q4)
        cache = dev(plain.bytes)
        k, kd = rows(g, t, hkv, d, torch.float32)
        v, vd = rows(g, t, hkv, d, torch.float32)
        qmm.qmm_kv_write(cache, kd, vd, dev(slots), page=page, ktype=0, vtype=1)
        plain.write(slots, k, v)
        assert np.array_equal(host(cache), plain.bytes), (t, page, first)
        got = qmm.qmm_kv_read(cache, dev(slots), hkv, d, page=page, ktype=0, vtype=1)
        for a, b in zip(got, plain.read(slots)):
            assert np.array_equal(host(a), b.astype(np.float32))


@pytest.mark.parametrize("hkv,d,kt,vt", [(64, 128, 0, 1), (100, 64, 1, 1), (33, 256, 0, 0), (1, 96, 1, 0)])
def test_many_heads(hkv, d, kt, vt):
    """More units of a token than a block has threads, for one of the two types or for both."""
    g = np.random.default_rng(hkv)
    t, page, pages = 7, 16, 2
    k, kd = rows(g, t, hkv, d, torch.float32)
    v, vd = rows(g, t, hkv, d, torch.float32)
    slots = scatter(g, t, pages, page)
    plain = ref.Cache(pages, hkv, d, page, kt, vt, fill=0x3C)
    cache = dev(plain.bytes)
    qmm.qmm_kv_write(cache, kd, vd, dev(slots), page=page, ktype=kt, vtype=vt)
    plain.write(slots, k, v)
    assert np.array_equal(host(cache), plain.bytes)
    got = qmm.qmm_kv_read(cache, dev(slots), hkv, d, page=page, ktype=kt, vtype=vt)
    for a, b in zip(got, plain.read(slots)):
        assert np.array_equal(host(a), b.astype(np.float32))


def test_bf16_blocks_with_ties():
    """bf16 rows have many pairs of the same magnitude: the first of the largest decides, in every place."""
    g = np.random.default_rng(12)
    t, hkv, d = 64, 2, 128
    x = torch.from_numpy(g.integers(-3, 4, (t, hkv, d)).astype(np.float32))
    plain = ref.Cache(4, hkv, d, 16, 1, 1)
    cache = dev(plain.bytes)
    slots = np.arange(64)
    qmm.qmm_kv_write(cache, x.bfloat16().cuda(), (-x).cuda().bfloat16(), dev(slots), page=16)
    plain.write(slots, x.numpy(), -x.numpy())
    assert np.array_equal(host(cache), plain.bytes)


def test_strided_rows_slices_of_a_projection():
    g = np.random.default_rng(5)
    t, hkv, d, hq = 21, 2, 64, 14
    y = dev(g.standard_normal((t, (hq + 2 * hkv) * d)).astype(np.float32))
    kd = y[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    vd = y[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    heads_first = kd.transpose(0, 1).contiguous().transpose(0, 1)      # token stride d, head stride t d
    slots = dev(scatter(g, t, 3, 16))
    size = qmm.qmm_kv_page_bytes(hkv, d, page=16)
    a, b, c = (torch.zeros(3, size, dtype=torch.uint8, device="cuda") for _ in range(3))
    qmm.qmm_kv_write(a, kd, vd, slots, page=16)
    qmm.qmm_kv_write(b, kd.contiguous(), vd.contiguous(), slots, page=16)
    qmm.qmm_kv_write(c, heads_first, vd, slots, page=16)
    assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(qmm.QmmError) as e:                              # rows off the 16-byte grid
        qmm.qmm_kv_write(a, y[:, 1:1 + hkv * d].unflatten(1, (hkv, d)), vd, slots, page=16)
    assert e.value.status == qmm.QMM_ERR_ALIGN


def test_left_out_and_missing_slots():
    g = np.random.default_rng(6)
    t, hkv, d, page, pages = 12, 2, 96, 16, 2
    k, kd = rows(g, t, hkv, d, torch.float32)
    slots = np.array([3, -1, 31, 32, 5, 1 << 40, -7, 0, 17, 2, 9, 30], np.int64)   # 32 and 2^40 do not exist
    plain = ref.Cache(pages, hkv, d, page, 1, 0)
    cache = dev(plain.bytes)
    assert qmm.device_status() == 0
    qmm.qmm_kv_write(cache, kd, kd, dev(slots), page=page, ktype=1, vtype=0)
    assert qmm.device_status() == 8 and qmm.device_status() == 0
    there = (slots >= 0) & (slots < pages * page)
    plain.write(np.where(there, slots, -1), k, k)
    assert np.array_equal(host(cache), plain.bytes)
    K = torch.full((t, hkv, d), 7.0, device="cuda")
    V = K.clone()
    qmm.qmm_kv_read(cache, dev(slots), hkv, d, K, V, page=page, ktype=1, vtype=0)
    assert qmm.device_status() == 8
    for got, want in zip((K, V), plain.read(np.where(there, slots, 0))):
        assert np.array_equal(host(got)[there], want[there].astype(np.float32))
        assert (host(got)[~there] == 7.0).all()
    qmm.qmm_kv_read(cache, dev(np.full(3, -1, np.int64)), hkv, d, page=page, ktype=1, vtype=0)
    assert qmm.device_status() == 0


def test_same_slot_read_twice_and_no_token():
    size = qmm.qmm_kv_page_bytes(1, 64, page=16)
    g = np.random.default_rng(7)
    cache = torch.zeros(1, size, dtype=torch.uint8, device="cuda")
    x = dev(g.standard_normal((16, 1, 64)).astype(np.float32))
    qmm.qmm_kv_write(cache, x, x, torch.arange(16, device="cuda"), page=16)
    K, _ = qmm.qmm_kv_read(cache, torch.tensor([4, 4, 9, 4], device="cuda"), 1, 64, page=16)
    assert torch.equal(K[0], K[1]) and torch.equal(K[0], K[3])
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    before = cache.clone()
    qmm.qmm_kv_write(cache, x[:0], x[:0], none, page=16)
    K, V = qmm.qmm_kv_read(cache, none, 1, 64, page=16)
    assert K.shape == V.shape == (0, 1, 64) and torch.equal(cache, before)


def test_offsets_past_32_bits():
    """A slot whose bytes lie behind the first 4 GiB of the cache."""
    hkv, d, page = 8, 128, 64
    size = qmm.qmm_kv_page_bytes(hkv, d, page=page)
    pages = (1 << 32) // size + 40
    cache = torch.empty(pages, size, dtype=torch.uint8, device="cuda")
    g = np.random.default_rng(8)
    k, kd = rows(g, 3, hkv, d, torch.float32)
    slots = np.array([pages * page - 1, 5, (pages - 20) * page + 18], np.int64)
    qmm.qmm_kv_write(cache, kd, kd, dev(slots), page=page)
    got = qmm.qmm_kv_read(cache, dev(slots), hkv, d, page=page)
    small = ref.Cache(1, hkv, d, page, 1, 1)
    small.write([0, 1, 2], k, k)
    for a, b in zip(got, small.read([0, 1, 2])):
        assert np.array_equal(host(a), b.astype(np.float32))
    assert qmm.device_status() == 0


def test_other_stream():
    """On a stream of the caller's: ordered there, results the same."""
    g = np.random.default_rng(9)
    hkv, d, t = 4, 128, 512
    x = dev(g.standard_normal((t, hkv, d)).astype(np.float32))
    slots = dev(scatter(g, t, 8, 64))
    size = qmm.qmm_kv_page_bytes(hkv, d, page=64)
    a, b = (torch.zeros(8, size, dtype=torch.uint8, device="cuda") for _ in range(2))
    qmm.qmm_kv_write(a, x, x, slots, page=64)
    want = qmm.qmm_kv_read(a, slots, hkv, d, page=64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        b.zero_()
        torch.cuda.synchronize()
        qmm.qmm_kv_write(b, x, x, slots, page=64, stream=stream)
        got = qmm.qmm_kv_read(b, slots, hkv, d, page=64, stream=stream)
        side.synchronize()
        assert torch.equal(a, b) and all(torch.equal(p, q) for p, q in zip(got, want))
