"""The key/value cache on the host (no GPU): layout, sizes and refusals."""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as ref

qmm = pytest.importorskip("decode_gemv_qmm_b200")
lib = qmm.lib

P16, P_ODD = 0x1000, 0x1008


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("qt", [ref.Q8, ref.Q4])
@pytest.mark.parametrize("val", [False, True])
def test_layout_is_a_permutation_of_the_part(d, qt, val):
    nb, n = d // 32, 32 if qt == ref.Q8 else 16
    at = [ref.code_place(d, qt, val, t, b, x) for t in range(16) for b in range(nb) for x in range(n)]
    at += [ref.scale_place(d, qt, t, b) + e for t in range(16) for b in range(nb) for e in range(2)]
    assert sorted(at) == list(range(ref.part_bytes(d, qt)))


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 64, 65536])
def test_page_bytes(d, page):
    for kt in (ref.Q8, ref.Q4):
        for vt in (ref.Q8, ref.Q4):
            assert qmm.qmm_kv_page_bytes(3, d, page=page, ktype=kt, vtype=vt) == ref.page_bytes(3, d, page, kt, vt)


@pytest.mark.parametrize("qt", [ref.Q8, ref.Q4])
def test_reference_quantiser_is_within_half_a_step(qt):
    """|x - value| <= d / 2 (Q8_0), d (Q4_0: the side away from the largest value ends at 7), and the scale's own
    rounding, half a unit of 2^-11 of the largest value."""
    x = np.random.default_rng(1).standard_normal((50, 128)).astype(np.float32)
    codes, d = ref.quantise(x, qt)
    v = ref.values(codes, d, qt).reshape(50, 4, 32)
    x = x.reshape(50, 4, 32)
    step = np.abs(x).max(-1, keepdims=True) / (127 if qt == ref.Q8 else 8)
    most = step * (0.5 if qt == ref.Q8 else 1.0) + np.abs(x).max(-1, keepdims=True) * 2.0 ** -10
    assert (np.abs(x - v) <= most).all()


def test_reference_quantiser_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [-8, 8, 0.5, -0.5]          # the first of the largest gives the sign: d = 1
    codes, d = ref.quantise(x, ref.Q4)
    assert d[0, 0] == 1 and list(codes[0, 0, :4] & 15) == [0, 15, 9, 8]   # 8.5 + 8 is held at 15; trunc(8.0) = 8
    x[0, :4] = [127, 2.5, -2.5, 0.49999997]
    codes, d = ref.quantise(x, ref.Q8)
    assert d[0, 0] == 1 and list(codes.view(np.int8)[0, 0, :4]) == [127, 3, -3, 0]
    codes, d = ref.quantise(np.zeros((1, 32), np.float32), ref.Q4)
    assert d[0, 0] == 0 and (codes == 0x88).all()


def page_bytes(**kw):
    a = dict(kt=1, vt=1, hkv=2, d=64, block=32, page=64) | kw
    out = ctypes.c_int64(0)
    return lib.qmm_kv_page_bytes(a["kt"], a["vt"], a["hkv"], a["d"], a["block"], a["page"], ctypes.addressof(out))


def write(**kw):
    a = dict(kt=1, vt=1, dt=0, T=4, hkv=2, d=64, block=32, pages=4, page=64, K=P16, ks=128, kh=64, V=P16, vs=128, vh=64,
             slots=P16, cache=P16) | kw
    return lib.qmm_kv_write(*a.values(), 0)


def read(**kw):
    a = dict(kt=1, vt=1, dt=0, T=4, hkv=2, d=64, block=32, pages=4, page=64, slots=P16, cache=P16, K=P16, V=P16) | kw
    return lib.qmm_kv_read(*a.values(), 0)


def attn(**kw):
    a = dict(kt=1, vt=1, dt=0, B=2, M=1, hq=4, hkv=2, d=64, block=32, pages=4, page=64, Q=P16, qs=256, qt=256, qh=64,
             cache=P16, table=P16, ts=2, mp=2, lens=P16, scale=1.0, window=0, Y=P16, ws=P16, wsb=1 << 40) | kw
    return lib.qmm_kv_attn(*a.values(), 0)


FORM = [(dict(kt=2), "DTYPE"), (dict(vt=-1), "DTYPE"), (dict(hkv=0), "SHAPE"), (dict(hkv=1025), "SHAPE"),
        (dict(d=32), "SHAPE"), (dict(d=80), "SHAPE"), (dict(d=288), "SHAPE"), (dict(page=8), "SHAPE"),
        (dict(page=48), "SHAPE"), (dict(page=0), "SHAPE"), (dict(page=131072), "SHAPE"), (dict(block=16), "BLOCK")]
CACHE = FORM + [(dict(pages=-1), "SHAPE"), (dict(pages=1 << 31), "SHAPE"), (dict(dt=2), "DTYPE"),
                (dict(cache=0), "NULL"), (dict(cache=P_ODD), "ALIGN")]
TOKENS = CACHE + [(dict(T=-1), "SHAPE"), (dict(T=1 << 31), "SHAPE"), (dict(slots=0), "NULL"), (dict(slots=P16 + 4), "ALIGN"),
                  (dict(K=0), "NULL"), (dict(V=P_ODD), "ALIGN")]


@pytest.mark.parametrize("call,kw,expect",
                         [(page_bytes, *c) for c in FORM] + [(write, *c) for c in TOKENS] + [(read, *c) for c in TOKENS]
                         + [(attn, *c) for c in CACHE]
                         + [(write, dict(ks=-128), "SHAPE"), (write, dict(kh=66), "ALIGN"), (write, dict(vs=130), "ALIGN"),
                            (write, dict(dt=1, vh=4), "ALIGN"),
                            (attn, dict(B=-1), "SHAPE"), (attn, dict(B=65537), "SHAPE"), (attn, dict(M=9), "SHAPE"),
                            (attn, dict(M=-1), "SHAPE"), (attn, dict(hq=3), "SHAPE"), (attn, dict(hq=0), "SHAPE"),
                            (attn, dict(hq=258), "SHAPE"), (attn, dict(Q=0), "NULL"), (attn, dict(Q=P_ODD), "ALIGN"),
                            (attn, dict(qs=2), "ALIGN"), (attn, dict(qt=6), "ALIGN"), (attn, dict(qh=-4), "SHAPE"),
                            (attn, dict(table=0), "NULL"), (attn, dict(ts=-1), "SHAPE"), (attn, dict(mp=-1), "SHAPE"),
                            (attn, dict(mp=1 << 24), "SHAPE"), (attn, dict(lens=0), "NULL"),
                            (attn, dict(lens=P16 + 2), "ALIGN"), (attn, dict(scale=float("nan")), "SHAPE"),
                            (attn, dict(scale=float("inf")), "SHAPE"), (attn, dict(window=-1), "SHAPE"),
                            (attn, dict(Y=0), "NULL"), (attn, dict(Y=P_ODD), "ALIGN"), (attn, dict(ws=0), "NULL"),
                            (attn, dict(ws=P_ODD), "ALIGN"), (attn, dict(wsb=0), "SHAPE")])
def test_refusals_before_any_cuda_call(call, kw, expect):
    assert qmm.STATUS_NAMES[call(**kw)] == "QMM_ERR_" + expect, lib.qmm_last_error_string()
    assert lib.qmm_last_error_string()


@pytest.mark.parametrize("wait_ns", [0, 999, 2_000_000_001])
def test_withheld_copy_limits(wait_ns):
    a = (1, 1, 0, 2, 1, 4, 2, 64, 32, 4, 64, P16, 256, 256, 64, P16, P16, 2, 2, P16, 1.0, 0, P16, P16, 1 << 40, wait_ns, 0)
    assert lib.qmm_test_kv_withheld_copy(*a) == qmm.QMM_ERR_SHAPE


def test_empty_calls():
    assert write(T=0, K=0, V=0, slots=0, cache=0) == 0
    assert read(T=0, K=0, V=0, slots=0, cache=0) == 0
    assert attn(B=0, Q=0, table=0, lens=0, Y=0, ws=0, wsb=0, cache=0) == 0
    assert attn(M=0, Q=0, table=0, lens=0, Y=0, ws=0, wsb=0, cache=0) == 0
    assert lib.qmm_kv_page_bytes(1, 1, 2, 64, 32, 64, 0) == qmm.QMM_ERR_NULL
    assert lib.qmm_kv_attn_workspace(1, 1, 4, 2, 64, 0) == qmm.QMM_ERR_NULL


def test_workspace_sizes():
    assert qmm.qmm_kv_attn_workspace(0, 0, 4, 2, 64) >= 0
    a = qmm.qmm_kv_attn_workspace(1, 1, 8, 8, 128)
    assert a % 4 == 0 and a <= qmm.qmm_kv_attn_workspace(64, 8, 64, 8, 128) < 1 << 32
    for bad in ((1, 9, 8, 8, 128), (1, 1, 8, 3, 128), (1, 1, 8, 8, 80), (70000, 1, 8, 8, 128)):
        with pytest.raises(qmm.QmmError):
            qmm.qmm_kv_attn_workspace(*bad)


def binding():
    """CPU tensors of a call that is right but for its device."""
    form = dict(page=16, ktype=0, vtype=1, stream=0)
    cache = torch.zeros(3, qmm.qmm_kv_page_bytes(2, 64, page=16, ktype=0, vtype=1), dtype=torch.uint8)
    return form, cache, torch.zeros(5, 2, 64), torch.zeros(5, dtype=torch.int64)


def test_binding_refusals():
    form, cache, x, slots = binding()
    for bad in (dict(K=x[:, :, ::2]), dict(K=x.half()), dict(V=x[:4]), dict(V=x.bfloat16()), dict(slots=slots.int()),
                dict(slots=slots[:3]), dict(slots=torch.zeros(10, dtype=torch.int64)[::2]), dict(cache=cache[:, :-16]),
                dict(cache=cache.view(torch.int8)), dict(K=torch.zeros(5, 3, 64), V=torch.zeros(5, 3, 64))):
        a = dict(cache=cache, K=x, V=x, slots=slots) | bad
        with pytest.raises(ValueError):
            qmm.qmm_kv_write(a["cache"], a["K"], a["V"], a["slots"], **form)
    for bad in (dict(K=x[:4]), dict(K=x, V=x.bfloat16()), dict(K=x.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(slots=slots.view(5, 1)), dict(Hkv=1), dict(dtype=torch.float16)):
        a = dict(slots=slots, Hkv=2, D=64) | bad
        with pytest.raises(ValueError):
            qmm.qmm_kv_read(cache, a.pop("slots"), a.pop("Hkv"), a.pop("D"), **a, **form)
    q, table, lens = torch.zeros(4, 1, 6, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for bad in (dict(Q=q[0]), dict(Q=q.half()), dict(table=table.long()), dict(table=table[:3]), dict(lens=lens.long()),
                dict(lens=lens[:3]), dict(table=torch.zeros(2, 4, dtype=torch.int32).T), dict(Y=q[:3]),
                dict(Y=q.bfloat16()), dict(ws=torch.zeros(64)), dict(Hkv=1)):
        a = dict(Q=q, cache=cache, table=table, lens=lens, Hkv=2) | bad
        with pytest.raises(ValueError):
            qmm.qmm_kv_attn(**a, **form)
    with pytest.raises(qmm.QmmError) as e:
        qmm.qmm_kv_attn(torch.zeros(4, 9, 6, 64), cache, table, lens, 2, **form)
    assert e.value.status == qmm.QMM_ERR_SHAPE
