"""Contiguous 4-bit products past the layout's rule: of several experts in an aligned 128-row block the largest index is the
block's, as in the FP8 forms, and only its rows are written, whatever the tile shape."""

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_matmul_amd import dg
from oracle import mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
G, N, K = 7, 272, 384


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _layouts():
    rng = np.random.default_rng(1)
    largest_last = np.repeat([0, 1, 2], [70, 130, 100])          # rows 0-127: experts 0 then 1; a partial last block
    largest_first = np.repeat([5, 2, 3, 1], [64, 64, 90, 166])
    padding_first = np.full(4 * 128, -1)
    padding_first[30], padding_first[100] = 2, 4                 # in both halves, rising and falling
    padding_first[128 + 5], padding_first[128 + 127] = 6, 0
    padding_first[256:256 + 70] = G                              # outside [0, G) is padding
    padding_first[383] = 1
    tail = {}
    for extra in (1, 2, 3, 5):                                   # the largest among rows past the last four whole ones
        x = np.full(128 + extra, 1)
        x[-1] = 6
        tail[f"tail {extra}"] = x
    many = rng.integers(-2, G + 2, 70 * 128 + 33)
    return dict(tail, largest_last=largest_last, largest_first=largest_first, padding_first=padding_first, many=many)


@pytest.mark.parametrize("name", list(_layouts()))
def test_largest_index_of_a_block(monkeypatch, name):
    idx = _layouts()[name].astype(np.int32)
    M = len(idx)
    rng = np.random.default_rng(M)
    a, b = rng.integers(0, 256, (M, K // 2)).astype(np.uint8), rng.integers(0, 256, (G, N, K // 2)).astype(np.uint8)
    sa, sb = np.full((K // 128, M), 0x7F7F7F7F, np.int32), np.full((G, K // 128, N), 0x7F7F7F7F, np.int32)  # scales 1: exact sums
    seven = oracle.bf16_rne_bits(np.float32(7.0))
    want = np.full((M, N), seven)
    valid = np.where((idx >= 0) & (idx < G), idx, -1)
    for r0 in range(0, M, 128):
        at = np.arange(r0, min(M, r0 + 128))
        e = valid[at].max()
        r = at[valid[at] == e]
        if e >= 0:
            want[r] = oracle.bf16_rne_bits(mxfp4.gemm_mxfp4(a[r], sa[:, r], b[e], sb[e])[0].astype(np.float32))
    for tile in ("64x64", "128x256", "256x256", None):
        if tile:
            monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
        else:
            monkeypatch.delenv("DG_FORCE_CONFIG")
        for cus in (0, 5):
            dg.dg_set_num_cus(cus)
            try:
                D = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
                dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(*map(_t, (a, sa, b, sb)), D, _t(idx))
            finally:
                dg.dg_set_num_cus(0)
            got = D.view(torch.int16).cpu().numpy().view(np.uint16)
            assert np.array_equal(oracle.bf16_bits_to_f64(got), oracle.bf16_bits_to_f64(want)), (tile, cus)
