"""Every kernel of the router and of its gradient: both types, every number of lanes and of values a lane, up to 8 and up to 16
choices, several workgroups.  Bounds as in test_gpu_moe.py."""

import numpy as np
import pytest
import torch

from moe_grouped_matmul_amd import dg
from oracle import moe
from tests.test_gpu_moe import DEV, U, _check_gate, _close, _gate, _spread, _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 8, 9, 16])
@pytest.mark.parametrize("E", [16, 60, 64, 100, 128, 129, 160, 256, 257, 384, 512, 513, 1000, 1024])
def test_forward_and_gradient(E, k, dtype):
    T = 150
    rng = np.random.default_rng(E + k)
    x = rng.standard_normal((T, E)).astype(np.float32) * 2
    x[::4] = np.round(x[::4])                                  # equal logits
    x[1::4][rng.random(x[1::4].shape) < 0.7] = -np.inf         # expert masks
    x[2::8, : E - k // 2] = torch.finfo(dtype).min
    x[T - 1], x[T - 2, 1:] = -np.inf, -np.inf                  # no expert left, one left
    X = _t(x).to(dtype)
    x = X.double().cpu().numpy()
    valid = _t(rng.random(T) < 0.9)
    for renorm in (True, False):
        kw = dict(renorm=renorm, w_scale=1.75, loss_coef=0.03)
        o = _gate(X, k, valid, **kw)
        want = moe.gate(x, k, valid=valid.cpu().numpy(), **kw)
        _check_gate(o, want, x, T)
        dw = rng.standard_normal((T, k)).astype(np.float32)
        got = torch.full((T, E), 7.0, dtype=dtype, device=DEV)
        dg.dg_moe_gate_bwd(X, o["topk_idx"], o["topk_w"], o["counts"], _t(dw), torch.full((1,), 1.5, device=DEV), got, **kw)
        d, mag = moe.gate_grad(want, dw, 1.5, **kw)
        out = 2.0 ** -8 if dtype is torch.bfloat16 else U
        _close(got.double().cpu(), d, out * np.abs(d) * 1.01 + (4 * _spread(x) + 100) * U * mag + 1e-37, renorm)


def test_gradient_past_32_bit_offsets():
    """4.3e9 logits: rows at both ends and around the places where an offset would wrap, against the oracle with random dw."""
    T, E, k = (1 << 22) + 5, 1024, 2
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(T, E, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    counts, load, loss = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV), torch.empty(1, device=DEV)
    ws = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, T, E, k), dtype=torch.uint8, device=DEV)
    dw = torch.randn(T, k, device=DEV, generator=g)
    for renorm in (True, False):
        kw = dict(renorm=renorm, loss_coef=0.1)
        dg.dg_moe_gate(x, idx, w, counts, load, loss, workspace=ws, **kw)
        dl = torch.full_like(x, 7.0)
        dg.dg_moe_gate_bwd(x, idx, w, counts, dw, torch.ones(1, device=DEV), dl, **kw)
        assert not bool((dl == 7).any())  # every element is written
        at = {0, 1, T - 2, T - 1}
        for b in (2 ** 31, 2 ** 32, 2 ** 33):
            for row in (E, 2 * E):
                at |= {r for r in (b // row - 1, b // row, b // row + 1) if r < T}
        at = torch.tensor(sorted(at), device=DEV)
        h = x[at].double().cpu().numpy()
        want = dict(moe.gate(h, k, **kw), counts=counts.cpu().numpy())
        assert np.array_equal(idx[at].cpu().numpy(), want["topk_idx"])
        d, mag = moe.gate_grad(want, dw[at].double().cpu().numpy(), 1.0, **kw)
        tol = 2.0 ** -8 * np.abs(d) * 1.01 + (4 * _spread(h) + 100) * U * mag + 1e-37
        assert np.all(np.abs(d).max(1) > 50 * tol.max(1))  # zeros would not pass
        _close(dl[at].double().cpu(), d, tol, renorm)
    del x, dl
    torch.cuda.empty_cache()
