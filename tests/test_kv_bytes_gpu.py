"""The bytes that qmm_kv_write stores for blocks at the ends of the number range."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from parity import dev, host

pytestmark = pytest.mark.gpu

qmm = pytest.importorskip("decode_gemv_qmm_b200")


def write(x, kt, vt, dtype=torch.float32):
    """The cache's bytes after x [t, hkv, d] was written as keys and values, and what the plain cache holds then."""
    t, hkv, d = x.shape
    xt = torch.from_numpy(x).to(dtype)
    x = xt.float().numpy()
    pages = -(-t // 16)
    plain = ref.Cache(pages, hkv, d, 16, kt, vt, fill=0x5A)
    cache = dev(plain.bytes)
    qmm.qmm_kv_write(cache, xt.cuda(), (-xt).cuda(), dev(np.arange(t)), page=16, ktype=kt, vtype=vt)
    return host(cache), plain, x


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("beside", ["ties", "no ties", "zeros"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_of_either_sign(d, beside, dtype):
    """Q4_0's scale takes its sign from the first of the largest, of zeros too, whatever is written beside the block."""
    g = np.random.default_rng(d)
    t, hkv, nb = 40, 3, d // 32
    x = g.standard_normal((t, hkv, nb, 32)).astype(np.float32)
    if beside == "ties":
        x[..., 5], x[..., 9] = 9.0, -9.0
    if beside == "zeros":
        x[:] = 0.0
    signs = g.integers(0, 6, (t, hkv, nb))
    for kind, zeros in enumerate((np.zeros(32), -np.zeros(32), np.where(np.arange(32) % 2, 0.0, -0.0),
                                  np.where(np.arange(32) % 2, -0.0, 0.0), np.where(np.arange(32) > 20, -0.0, 0.0))):
        x[signs == kind] = zeros
    got, plain, x = write(x.reshape(t, hkv, d), 1, 1, dtype)
    plain.write(np.arange(t), x, -x)
    assert np.array_equal(got, plain.bytes)
