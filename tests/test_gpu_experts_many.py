"""Experts with many tokens each: whole 16-token products, passes of several groups, runs of neighbouring units and their odd
ends.  Bounds and helpers are those of test_gpu_experts.py."""

import pytest
import torch

from moe_grouped_matmul_amd import dg
from test_gpu_experts import DEV, _check, _layer, _run, _tokens

pytestmark = pytest.mark.gpu


def _counts(T, counts, G, H, seed=0):
    """One choice a token: counts[e] tokens choose expert e, in a random order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    idx = torch.cat([torch.full((n,), e, device=DEV) for e, n in enumerate(counts)])[:T]
    idx = idx[torch.randperm(T, device=DEV, generator=g)][:, None].int().contiguous()
    return torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16), idx, torch.rand(T, 1, device=DEV, generator=g) + 0.5


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("counts", [(64,), (40, 24), (33, 31), (9, 55), (17, 16, 15, 16), (8, 8, 48), (1, 63), (10, 9, 11, 1, 2, 31)])
def test_counts_of_tokens(counts, fmt):
    H, inner = 384, 256
    L = _layer(fmt, len(counts), H, inner)
    x, idx, w = _counts(64, counts, len(counts), H)
    y = _check(L, x, idx, w)
    for _ in range(3):  # which of an expert's tokens share a pass changes no bit
        assert torch.equal(_run(L, x, idx, w), y)


@pytest.mark.parametrize("cus", [1, 3, 7, 8])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,k,G,H,inner", [(64, 2, 3, 256, 384), (40, 4, 5, 128, 640), (17, 2, 2, 640, 128), (64, 16, 40, 256, 256), (64, 1, 40, 256, 256)])
def test_runs_of_units(T, k, G, H, inner, fmt, cus):
    L = _layer(fmt, G, H, inner)
    x, idx, w = _tokens(T, k, G, H, seed=cus)
    y = _check(L, x, idx, w)
    dg.dg_set_num_cus(cus)
    try:
        few = _check(L, x, idx, w)
    finally:
        dg.dg_set_num_cus(0)
    assert few.shape == y.shape


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_nan_among_many_tokens(fmt):
    H, inner = 256, 256
    L = _layer(fmt, 2, H, inner)
    x, idx, w = _counts(64, (40, 24), 2, H)
    y = _run(L, x, idx, w)
    bad = x.clone()
    bad[5, 3], bad[60, 100] = float("nan"), float("inf")
    got = _run(L, bad, idx, w)
    keep = torch.ones(64, dtype=torch.bool, device=DEV)
    keep[[5, 60]] = False
    assert torch.equal(got[keep], y[keep])
    assert got[5].isnan().all() and not got[60].isfinite().all()
    w2 = w.clone()
    w2[9] = float("inf")
    got = _run(L, x, idx, w2)
    keep[:] = True
    keep[9] = False
    assert torch.equal(got[keep], y[keep]) and not got[9].isfinite().any()


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_many_calls_with_splits(fmt):
    # two workgroups and more share every 32 columns of y: each call's partial sums reach the last of them whole
    H, inner, G = 4096, 512, 8
    L = _layer(fmt, G, H, inner)
    for seed in range(4):
        x, idx, w = _tokens(64, 2, G, H, seed=seed, drop=0)
        y = _run(L, x, idx, w)
        for _ in range(60):
            assert torch.equal(_run(L, x, idx, w), y)
