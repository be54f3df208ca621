"""Sums over blocks of different scales on every tile shape of the 4-bit products.  Scales of 2^-2 to 2^2 on either side: a
product is a multiple of 2^-2 * 2^-4 and at most 36 * 2^4, so a sum over K = 256 takes at most 24 bits (2^-6 to 2^17.2) and
fp32 accumulation is exact in any order; the result is that sum rounded once to bf16.  In the cancelling cases the second 256
elements of a row take away what the first 256 added, up to one block, so an accumulator of fewer bits shows at once."""

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


def _operands(rng, M, N, cancel):
    K = 256
    a, b = rng.integers(0, 256, (M, K // 2)).astype(np.uint8), rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    ca, cb = 127 + rng.integers(-2, 3, (M, K // 32)), 127 + rng.integers(-2, 3, (N, K // 32))
    if cancel:
        less = a ^ 0x88                                                    # both signs flipped
        less[:, 48:64] = rng.integers(0, 256, (M, 16))                     # one block is its own
        a, ca = np.concatenate((a, less), 1), np.concatenate((ca, ca), 1)
        b, cb = np.concatenate((b, b), 1), np.concatenate((cb, cb), 1)
    return a, mxfp4.pack_words(ca), b, mxfp4.pack_words(cb)


def _want(a, sa, b, sb):
    ref, mag = mxfp4.gemm_mxfp4(a, sa, b, sb)
    assert mag.max() <= 2 * 36 * 16 * 256 and np.array_equal(ref * 64, np.round(ref * 64))
    return oracle.bf16_bits_to_f64(oracle.bf16_rne_bits(ref.astype(np.float32)))


def _values(D):
    return oracle.bf16_bits_to_f64(D.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


@pytest.mark.parametrize("cancel", [False, True])
@pytest.mark.parametrize("tile", ["64x64", "64x64x2", "128x256", "256x256"])
def test_dense(monkeypatch, tile, cancel):
    monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
    rng = np.random.default_rng(len(tile) + cancel)
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    for M, N in ((1, 16), (70, 144), (300, 528)):
        ops = _operands(rng, M, N, cancel)
        want = _want(*ops)
        for cus in (0, 3):  # few: a persistent workgroup walks whole tiles, halves and quarters
            dg.dg_set_num_cus(cus)
            try:
                D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
                dg.dg_mxfp4_gemm_nt(*map(_t, ops), D, workspace=ws)
            finally:
                dg.dg_set_num_cus(0)
            assert np.array_equal(_values(D), want), (M, N, cus)


@pytest.mark.parametrize("cancel", [False, True])
@pytest.mark.parametrize("tile", ["64x64", "128x256", "256x256"])
def test_contiguous_and_masked(monkeypatch, tile, cancel):
    monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
    rng = np.random.default_rng(7 + cancel)
    G, per, N = 3, 256, 272
    ops = [_operands(rng, per, N, cancel) for _ in range(G)]
    want = [_want(*o) for o in ops]
    B, SB = _t(np.stack([o[2] for o in ops])), _t(np.stack([o[3] for o in ops]))
    A = np.concatenate([o[0] for o in ops])
    idx = np.repeat(np.arange(G), per).astype(np.int32)
    D = torch.full((G * per, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(_t(A), _t(np.concatenate([o[1] for o in ops], 1)), B, SB, D, _t(idx))
    assert np.array_equal(_values(D), np.concatenate(want))
    D = torch.full((G, per, N), 7.0, dtype=torch.bfloat16, device=DEV)
    m = np.array([per, 0, 131], np.int32)
    dg.dg_m_grouped_mxfp4_gemm_nt_masked(_t(A.reshape(G, per, -1)), _t(np.stack([o[1] for o in ops])), B, SB, D, _t(m))
    got = _values(D)
    for g in range(G):
        assert np.array_equal(got[g, : m[g]], want[g][: m[g]]) and np.all(got[g, m[g]:] == 7.0)
