"""The 4-bit quantiser and products where they stream past the caches (wide arrays of 16 MB on, one row tile against 256 MB of
weights on), and the quantiser's gather from fp32."""

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_matmul_amd import dg
from oracle import mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _values(D):
    return oracle.bf16_bits_to_f64(D.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


@pytest.mark.parametrize("shape", [(1031, 4480), (3, 347, 4224), (2, 32771, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantiser_and_back(shape, dtype):
    """Just past the threshold in fp32; the bf16 arrays are doubled in rows to pass it too."""
    if dtype is torch.bfloat16:
        shape = shape[:-2] + (2 * shape[-2] + 1, shape[-1])
    K = shape[-1]
    g = torch.Generator(device=DEV).manual_seed(K)
    x = torch.randn(shape, device=DEV, generator=g) * torch.exp2(torch.randint(-20, 20, shape[:-1] + (1,), device=DEV, generator=g).float())
    x.view(-1, 32)[::11] = 0
    x.view(-1, K)[5, 40] = float("inf")
    x = x.to(dtype)
    assert x.nbytes >= 16 << 20
    q = torch.full(shape[:-1] + (K // 2,), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full(shape[:-2] + (K // 128, shape[-2]), 0x5A5A5A5A, dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(x, q, s)
    rows = x.view(-1, K).shape[0]
    at = np.unique(np.concatenate((np.arange(9), np.arange(rows - 9, rows), np.random.default_rng(1).integers(0, rows, 200))))
    codes, words = mxfp4.quant_mxfp4(x.view(-1, K)[_t(at)].float().cpu().numpy())
    flat_s = s.transpose(-1, -2).reshape(rows, K // 128)
    assert np.array_equal(q.view(rows, -1)[_t(at)].cpu().numpy(), codes)
    assert np.array_equal(flat_s[_t(at)].cpu().numpy(), words.T)
    want = mxfp4.values_mxfp4(codes, words)
    for out in (torch.float32, torch.bfloat16):
        y = torch.full(shape, 7.0, dtype=out, device=DEV)
        dg.dg_dequant_mxfp4(q, s, y)
        assert np.array_equal(y.view(rows, K)[_t(at)].double().cpu().numpy(), want, equal_nan=True)
    # every element is one of its code's: within half a step of x, 2^-2 of the block's scale's largest value (or zero blocks exactly)
    y = torch.empty(shape, device=DEV)
    dg.dg_dequant_mxfp4(q, s, y)
    xb, yb = x.float().view(-1, 32), y.view(-1, 32)
    good = torch.isfinite(xb).all(1)
    top = xb.abs().amax(1, keepdim=True)
    assert int((~good).sum()) == 1 and bool(yb[~good].isnan().all())
    assert bool(((xb - yb).abs() <= top / 3)[good].all())  # the widest step is 2 of 6, top > 3 scales: half of it at most top / 3


@pytest.mark.parametrize("lead", [(700,), (5, 90)])
def test_gather_from_fp32(lead):
    rng = np.random.default_rng(4)
    T, K = 61, 1408
    x = (rng.standard_normal((T, K)) * 2.0 ** rng.integers(-9, 9, (T, 1))).astype(np.float32)
    rt = rng.integers(-2, T + 3, lead).astype(np.int32)
    q = torch.full(lead + (K // 2,), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full(lead[:-1] + (K // 128, lead[-1]), 0x5A5A5A5A, dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(_t(x), q, s, row_token=_t(rt))
    codes, words = mxfp4.quant_mxfp4(x[np.clip(rt, 0, T - 1)])
    ok = (rt >= 0) & (rt < T)
    assert np.array_equal(q.cpu().numpy(), np.where(ok[..., None], codes, 0xA5))
    assert np.array_equal(s.cpu().numpy(), np.where(ok[..., None, :], words, 0x5A5A5A5A))


@pytest.mark.parametrize("max_m,tile", [(128, "128x256"), (100, None), (64, "64x64"), (33, None), (1, None)])
def test_masked_product_against_large_weights(monkeypatch, max_m, tile):
    """One row tile an expert against 271 MB of weights; scales 1, so sums are exact."""
    if tile:
        monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
    G, N, K = 17, 4368, 7296
    assert G * N * K // 2 >= 256 << 20
    g = torch.Generator(device=DEV).manual_seed(max_m)
    A = torch.randint(0, 256, (G, max_m, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    B = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    SA = torch.full((G, K // 128, max_m), 0x7F7F7F7F, dtype=torch.int32, device=DEV)
    SB = torch.full((G, K // 128, N), 0x7F7F7F7F, dtype=torch.int32, device=DEV)
    m = torch.randint(0, max_m + 1, (G,), device=DEV, generator=g).int()
    m[0], m[3], m[G - 1] = max_m, 0, max_m
    D = torch.full((G, max_m, N), 7.0, dtype=torch.bfloat16, device=DEV)
    dg.dg_m_grouped_mxfp4_gemm_nt_masked(A, SA, B, SB, D, m)
    for e in (0, 3, 8, G - 1):
        n = int(m[e])
        if n:
            at = sorted({0, n // 2, n - 1})
            a = A[e, at].cpu().numpy()
            ref, _ = mxfp4.gemm_mxfp4(a, SA[e][:, at].cpu().numpy(), B[e].cpu().numpy(), SB[e].cpu().numpy())
            assert np.array_equal(_values(D[e, at]), oracle.bf16_bits_to_f64(oracle.bf16_rne_bits(ref.astype(np.float32)))), e
        assert bool((D[e, n:] == 7).all())


@pytest.mark.parametrize("M", [1, 64, 128])
def test_dense_product_against_large_weights(M):
    N, K = 32784, 16512
    assert N * K // 2 >= 256 << 20
    g = torch.Generator(device=DEV).manual_seed(M)
    A = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    B = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    SA, SB = (torch.full((K // 128, n), 0x7F7F7F7F, dtype=torch.int32, device=DEV) for n in (M, N))
    D = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    dg.dg_mxfp4_gemm_nt(A, SA, B, SB, D)
    cols = torch.cat((torch.arange(300), torch.arange(N - 300, N), torch.arange(16000, 16300))).to(DEV)
    ref, mag = mxfp4.gemm_mxfp4(A.cpu().numpy(), SA.cpu().numpy(), B[cols].cpu().numpy(), SB[:, cols].cpu().numpy())
    assert mag.max() < 2 ** 22  # multiples of 1/4: exact in fp32
    assert np.array_equal(_values(D[:, cols]), oracle.bf16_bits_to_f64(oracle.bf16_rne_bits(ref.astype(np.float32))))
    assert not bool((D == 7).all(0).any() and M > 8)
