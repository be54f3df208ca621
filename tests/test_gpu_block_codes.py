"""Codes and scales of the epilogue's gradient and of the norm, bit for bit those of the quantisers where the values are the
same: rows with many zeros, groups of zeros and NaN, small quotients, scales at both ends of fp32."""

import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gradient_codes(dy):
    M, N = dy.shape
    q, sf = torch.empty(M, N, dtype=torch.uint8, device=DEV), torch.empty(N // 128, M, device=DEV)
    dg.dg_epilogue_bwd(dy, act="none", q=q, sf=sf)
    q2, sf2 = torch.empty_like(q), torch.empty_like(sf)
    dg.dg_quant_1x128(dy.float(), q2, sf2)
    return q, sf, q2, sf2


def _same(q, sf, q2, sf2):
    assert torch.equal(q, q2)
    assert torch.equal(sf.isnan(), sf2.isnan()) and torch.equal(sf.nan_to_num(nan=0.0), sf2.nan_to_num(nan=0.0))


@pytest.mark.parametrize("scale", [1.0, 1e-36, 1e-30, 1e30, 3e36])
@pytest.mark.parametrize("zeros", [0.0, 0.01, 0.5, 0.99])
def test_codes_equal_the_quantisers(zeros, scale):
    g = torch.Generator(device=DEV).manual_seed(int(100 * zeros))
    dy = torch.randn(70, 1152, device=DEV, generator=g) * scale
    dy[3] *= torch.exp2(-torch.randint(0, 24, (1152,), device=DEV, generator=g).float())  # quotients below the normal codes
    dy[4, ::2] = -0.0
    dy = torch.where(torch.rand(dy.shape, device=DEV, generator=g) < zeros, torch.zeros_like(dy), dy).to(torch.bfloat16)
    _same(*_gradient_codes(dy))


def test_groups_of_zeros_nan_and_infinities():
    g = torch.Generator(device=DEV).manual_seed(5)
    dy = torch.randn(12, 640, device=DEV, generator=g)
    nan, inf = float("nan"), float("inf")
    dy[0, :128] = nan  # nothing else in the group
    dy[1, :128] = 0
    dy[2, :128] = 0
    dy[2, 5] = nan
    dy[3, :128] = nan
    dy[3, 64:72] = 0  # one lane of zeros
    dy[4, 130] = nan
    dy[5, 128:256] = nan
    dy[5, 200] = 2.0
    dy[6, 7] = inf
    dy[7, :128] = nan
    dy[7, 127] = -inf
    dy[8, :128] = -0.0
    q, sf, q2, sf2 = _gradient_codes(dy.to(torch.bfloat16))
    _same(q, sf, q2, sf2)
    assert sf[0, 0].isnan() and sf[0, 1] == 1 and sf[0, 2] == 1 and sf[0, 3] == 1 and sf[0, 8] == 1


@pytest.mark.parametrize("M,K", [(3, 640), (5, 7168), (2000, 1152)])
def test_a_row_with_nan_shows_in_its_scales(M, K):
    # (a finite scale beside codes that hold no NaN would hide it from the product)
    x, w = torch.randn(M, K, device=DEV).to(torch.bfloat16), torch.ones(K, device=DEV)
    x[1, 7] = float("nan")
    q, sf = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(K // 128, M, device=DEV)
    dg.dg_rms_norm(x, w, q=q, sf=sf)
    assert sf[:, 1].isnan().all() and not sf[:, 0].isnan().any() and not sf[:, 2].isnan().any()


@pytest.mark.parametrize("kind", ["f32", "ue8m0"])
def test_sums_that_cancel(kind):
    # bf16 sums of like values are zeros: a fifth of the row
    M, K = 300, 1536
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn(M, K, device=DEV, generator=g)
    res = torch.where(torch.rand(M, K, device=DEV, generator=g) < 0.2, -x, torch.randn(M, K, device=DEV, generator=g))
    w = 1 + 0.2 * torch.randn(K, device=DEV, generator=g)
    shape, t, quant = ((K // 128, M), torch.float32, dg.dg_quant_1x128) if kind == "f32" else ((K // 512, M), torch.int32, dg.dg_quant_1x128_ue8m0)
    h, y, q, sf = torch.empty_like(x), torch.empty_like(x), torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(shape, dtype=t, device=DEV)
    dg.dg_rms_norm(x, w, residual=res, h=h, y=y, q=q, sf=sf)
    assert (h == 0).float().mean() > 0.15
    q2, sf2 = torch.empty_like(q), torch.empty_like(sf)
    quant(y, q2, sf2)  # in fp32, y is what was quantised
    assert torch.equal(q, q2) and torch.equal(sf, sf2)
