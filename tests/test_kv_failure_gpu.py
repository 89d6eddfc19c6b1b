"""qmm_kv_attn's bounded wait, made to run out without a fault: one copy is never issued
(qmm_test_kv_withheld_copy), with a limit of 2 ms. The call returns, the failure is recorded and cleared, what
the starved block does not work on is right, and so is the next call, with the same scratch."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_kv_attn_gpu import Case
from parity import dev, host

pytestmark = pytest.mark.gpu

qmm = pytest.importorskip("decode_gemv_qmm_b200")

WAIT_NS, FULL, DRAIN = 2_000_000, 1, 2


@pytest.mark.parametrize("lens", [[3000, 700, 50], [5, 40, 900]])
def test_wait_runs_out(lens):
    c = Case(lens, 1, 10, 2, 128, 1, 1, page=64, seed=31)
    table, ln = dev(c.table), dev(np.array(lens, np.int32))
    Y = torch.full((3, 1, 10, 128), float("nan"), device="cuda")
    ws = torch.empty(qmm.qmm_kv_attn_workspace(3, 1, 10, 2, 128), dtype=torch.uint8, device="cuda")
    assert qmm.device_status() == 0
    st = qmm.lib.qmm_test_kv_withheld_copy(
        1, 1, qmm.QMM_F32, 3, 1, 10, 2, 128, 32, c.cache.shape[0], 64, c.qd.data_ptr(), 10 * 128, 0, 128,
        c.cache.data_ptr(), table.data_ptr(), table.stride(0), table.shape[1], ln.data_ptr(), c.scale, 0, Y.data_ptr(),
        ws.data_ptr(), ws.numel(), WAIT_NS, torch.cuda.current_stream().cuda_stream)
    assert st == qmm.QMM_OK
    bits = qmm.device_status()
    assert bits & FULL and bits & DRAIN, bits
    assert qmm.device_status() == 0
    # the last key/value head of the last sequence lies behind the starved block's run of the work
    last = ref.attention(c.q[2][:, 5:], *(x[:, 1:] for x in c.kv[2]), lens[2], c.scale)
    ref.assert_attention(host(Y)[2][:, 5:], last)
    c.check(c.run(ws=ws), "the next call")
    c.check(c.run(), "and another")
