"""Combine and its gradient of many tokens: rows past the caches, narrow and wide, on either side of where the gradient takes a
workgroup per token.  Bounds as in test_gpu_moe.py: a rounding per term in fp32, one to bf16 (2^-8)."""

import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.mark.parametrize("k,N", [(1, 16), (2, 64), (8, 320), (3, 1360), (8, 512), (3, 1376), (1, 4112), (16, 256), (9, 448)])
def test_combine_and_gradient(k, N):
    T = (50 << 20) // (2 * k * N) + 3  # just past 48 MB of rows
    R = T * k + 5
    g = torch.Generator(device=DEV).manual_seed(N)
    rows = torch.randn(R, N, device=DEV, generator=g).to(torch.bfloat16)
    ro = torch.randperm(R, device=DEV, generator=g)[: T * k].reshape(T, k).int()
    ro[torch.rand(T, k, device=DEV, generator=g) < 0.03] = -1
    ro[1], ro[T - 1, 0] = -1, R
    w = torch.randn(T, k, device=DEV, generator=g)
    dy = torch.randn(T, N, device=DEV, generator=g).to(torch.bfloat16)
    y, drows, dw = torch.full_like(dy, 7.0), torch.full_like(rows, 7.0), torch.full_like(w, 7.0)
    dg.dg_moe_combine(rows, ro, w, y)
    dg.dg_moe_combine_bwd(dy, rows, ro, w, drows, dw)
    there = (ro >= 0) & (ro < R)
    want, mag = torch.zeros(T, N, dtype=torch.float64, device=DEV), torch.zeros(T, N, dtype=torch.float64, device=DEV)
    used = torch.zeros(R, dtype=torch.bool, device=DEV)
    d = dy.double()
    for j in range(k):
        t = torch.nonzero(there[:, j])[:, 0]
        r = ro[t, j].long()
        x, wj = rows[r].double(), w[t, j].double()[:, None]
        want[t] += wj * x
        mag[t] += (wj * x).abs()
        used[r] = True
        assert bool(((drows[r].double() - wj * d[t]).abs() <= (2.0 ** -8 * 1.01 + U) * (wj * d[t]).abs()).all()), j
        assert bool(((dw[t, j].double() - (x * d[t]).sum(1)).abs() <= (N / 256 + 20) * U * (x * d[t]).abs().sum(1)).all()), j
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + (k + 1) * U * mag).all())
    assert bool((drows[~used] == 7).all()) and not bool(dw[~there].any())
