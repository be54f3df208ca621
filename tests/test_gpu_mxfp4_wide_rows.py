"""The quantiser and its inverse on rows of nearly 2^31 columns, the longest they take."""

import gc

import numpy as np
import pytest
import torch

from moe_grouped_matmul_amd import dg
from oracle import mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("K", [2147483136, 2147483264, 2147483520])
@pytest.mark.parametrize("R,dtype", [(3, torch.bfloat16), (1, torch.float32)])
def test_longest_rows(R, dtype, K):
    """Zeros but for runs of values at both ends and where a byte offset of a row passes 2^31."""
    assert K % 128 == 0 and K < 2 ** 31
    rng = np.random.default_rng(K % 1000 + R)
    at = sorted({0, 2 ** 29 - 512, 2 ** 30 - 512, K - 1024})
    x = torch.zeros(R, K, dtype=dtype, device=DEV)
    for c in at:
        x[:, c:c + 1024] = torch.from_numpy(rng.standard_normal((R, 1024)).astype(np.float32)).to(DEV).to(dtype)
    q = torch.full((R, K // 2), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((K // 128, R), 0x5A5A5A5A, dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(x, q, s)
    want = {}
    for c in at:
        codes, words = mxfp4.quant_mxfp4(x[:, c:c + 1024].float().cpu().numpy())
        want[c] = mxfp4.values_mxfp4(codes, words)
        assert np.array_equal(q[:, c // 2:c // 2 + 512].cpu().numpy(), codes), c
        assert np.array_equal(s[c // 128:c // 128 + 8].cpu().numpy(), words), c
    x.fill_(7.0)
    dg.dg_dequant_mxfp4(q, s, x)
    for c in at:
        assert np.array_equal(x[:, c:c + 1024].double().cpu().numpy(), want[c]), c
        x[:, c:c + 1024] = 0
        q[:, c // 2:c // 2 + 512] = 0
        s[c // 128:c // 128 + 8] = 0x7F7F7F7F
    for r in range(R):  # every other element is zero, every other scale 1
        assert not bool(q[r].any()) and not bool(x[r].any())
    assert bool((s == 0x7F7F7F7F).all())
    del x, q, s
    gc.collect()
    torch.cuda.empty_cache()
