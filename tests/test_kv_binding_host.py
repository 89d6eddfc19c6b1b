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
