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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kt,vt", [(0, 1), (1, 0)])
def test_blocks_whose_inverse_scale_overflows(kt, vt, dtype):
    """|x| from 2^-149 to 2^-110, either side of where 1 / d is infinite: codes as the rule's clamps give them."""
    g = np.random.default_rng(7)
    t, hkv, d = 64, 2, 128
    size = 2.0 ** g.uniform(-149, -110, (t, hkv, 4, 1))
    x = (np.sign(g.standard_normal((t, hkv, 4, 32))) * np.maximum(size * g.uniform(0.05, 1, (t, hkv, 4, 32)), 2.0 ** -132
                                                                  if dtype == torch.bfloat16 else 2.0 ** -149))
    x[::3, :, 1] = g.standard_normal((len(x[::3]), hkv, 32))
    got, plain, x = write(x.astype(np.float32).reshape(t, hkv, d), kt, vt, dtype)
    assert (x != 0).all()
    plain.write(np.arange(t), x, -x)
    assert np.array_equal(got, plain.bytes)


def test_q8_blocks_are_those_of_the_activations():
    """The same codes and scales as qmm_quantize_act_q8_0 gives, zeros in blocks of tiny values and infinities among them."""
    g = np.random.default_rng(8)
    t, hkv, d = 64, 2, 128
    x = (g.standard_normal((t, hkv, 4, 32)) * 2.0 ** g.uniform(-149, 20, (t, hkv, 4, 1))).astype(np.float32)
    x[g.random(x.shape) < 0.1] = 0.0
    x[5, 0, 2, 7], x[6, 1, 0, :3] = np.inf, (-np.inf, 1.0, np.inf)     # d is infinite, 1 / d is 0
    x = x.reshape(t, hkv, d)
    got, plain, _ = write(x, 0, 0)
    for part, rows in enumerate((x, -x)):
        blocks = host(qmm.qmm_quantize_act_q8_0(dev(rows.reshape(t * hkv, d)))).reshape(t, hkv, 4, 34)
        _, code, scale = plain.at[part]
        for i in range(t):
            for h in range(hkv):
                pg, base, tok = plain._base(i, h)
                assert np.array_equal(got[pg, base + scale[tok]], blocks[i, h, :, :2]), (part, i, h)
                assert np.array_equal(got[pg, base + code[tok]], blocks[i, h, :, 2:]), (part, i, h)
