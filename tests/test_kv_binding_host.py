"""What the Python entry of the key/value cache's calls refuses before the library is called (no GPU)."""
import pytest
import torch

qmm = pytest.importorskip("decode_gemv_qmm_b200")

FORM = dict(page=16, ktype=0, vtype=1)


def host_cache():
    return torch.zeros(3, qmm.qmm_kv_page_bytes(2, 64, **FORM), dtype=torch.uint8)


@pytest.mark.parametrize("stream", [None, 0])
def test_tensors_in_host_memory_are_refused(stream):
    """Calls that are right but for their device: no host address reaches a kernel."""
    cache, x, slots = host_cache(), torch.zeros(5, 2, 64), torch.zeros(5, dtype=torch.int64)
    q, table, lens = torch.zeros(4, 1, 6, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        qmm.qmm_kv_write(cache, x, x, slots, stream=stream, **FORM)
    for out in ((None, None), (x, x.clone())):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            qmm.qmm_kv_read(cache, slots, 2, 64, *out, stream=stream, **FORM)
    ws = torch.zeros(qmm.qmm_kv_attn_workspace(4, 1, 6, 2, 64), dtype=torch.uint8)
    for out in ((None, None), (q.clone(), ws)):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            qmm.qmm_kv_attn(q, cache, table, lens, 2, *out, stream=stream, **FORM)


def test_older_calls_pass_no_address_of_host_memory():
    """The matmuls' entry points: the library is given NULL for a tensor in pageable host memory, and says so."""
    w8, w4 = torch.zeros(4 * 2 * 34, dtype=torch.uint8), torch.zeros(4 * 2 * 18, dtype=torch.uint8)
    x, q, d = torch.zeros(1, 64), torch.zeros(1, 64, dtype=torch.int8), torch.zeros(1, 2)
    calls = [lambda: qmm.qmm_q8_gemv(w8, x, 4, stream=0),
             lambda: qmm.qmm_q8_gemv(w8, x, 4, flags=qmm.QMM_FLAG_EARLY_WEIGHTS, stream=0),
             lambda: qmm.qmm_quantize_act_q8_0(x, stream=0),
             lambda: qmm.qmm_q8q8_gemv_q8_0(w8, w8[:68].view(1, 68), 64, 4, stream=0),
             lambda: qmm.qmm_q8_gemv_auto(w8, x, 4, stream=0),
             lambda: qmm.qmm_q8_gemv_multi([w8, w8], x, [4, 4], stream=0),
             lambda: qmm.qmm_quantize_act_q8(x, stream=0),
             lambda: qmm.qmm_q8q8_gemv(w8, q, d, 4, stream=0),
             lambda: qmm.qmm_q8q8_gemv_fused(w8, x, 4, stream=0),
             lambda: qmm.qmm_q8q8_block_dots(w8, q, 4, stream=0),
             lambda: qmm.qmm_q8q8_gemv_fused_dots(w8, x, 4, stream=0),
             lambda: qmm.qmm_q8q8_block_dots_q8_0(w8, w8[:68].view(1, 68), 64, 4, stream=0),
             lambda: qmm.qmm_q4_gemv(w4, x, 4, stream=0),
             lambda: qmm.qmm_q4_swiglu_gateup(w4, w4, x, 4, stream=0),
             lambda: qmm.qmm_q4_gateup_unfused(w4, w4, x, 4, stream=0),
             lambda: qmm.qmm_quant_matmul_prefill(0, w8, x.bfloat16(), 4, stream=0)]
    for call in calls:
        with pytest.raises(qmm.QmmError) as e:
            call()
        assert e.value.status == qmm.QMM_ERR_NULL
    empty = torch.zeros(0, 4)
    assert qmm.qmm_q8_gemv(w8, x[:0], 4, empty, stream=0) is empty


@pytest.mark.parametrize("spoil", ["sys.modules['decode_gemv_qmm_b200._qmm_bind'] = None", "torch.__version__ = '1.0'"])
def test_package_without_a_usable_binding(spoil):
    """The native entry missing, or built against another torch: the other calls work, the cache's say what to do."""
    import os
    import subprocess
    import sys
    code = f"""
import sys, torch
{spoil}
import decode_gemv_qmm_b200 as qmm
assert qmm.version() and qmm.qmm_kv_page_bytes(2, 64, page=16) == 2 * 64 * 18
try:
    qmm.qmm_q8_gemv(torch.zeros(8, dtype=torch.uint8), torch.zeros(1, 33), 4, stream=0)
except qmm.QmmError as e:
    assert e.status == qmm.QMM_ERR_SHAPE
x = torch.zeros(1, 2, 64)
for call in (lambda: qmm.qmm_kv_write(x, x, x, x, page=16), lambda: qmm.qmm_kv_read(x, x, 2, 64, page=16),
             lambda: qmm.qmm_kv_attn(x, x, x, x, 2, page=16)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e)
    else:
        raise AssertionError("no ImportError")
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
