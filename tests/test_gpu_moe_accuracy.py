"""The router's probabilities far below a row's maximum (u = 2^-24), at distances d that fp32 holds exactly.

e^-d: the exponent's fraction is rounded twice (below 2^-25 each, 0.7 u in the result), the exponential is within one place
(2 u): 2.7 u.  A weight e / (1 + e): the sum u and at most half of e's own error, the division 2 u: 2.7 + 1 + 1.4 + 2 < 8 u.
A gradient p1 p0: p1 = e * (1 / s) and p0 likewise, a rounding more each, and their product's: below 16 u.  None of them
grows with d."""

import numpy as np
import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def _rows(E, at):
    """Distances of 0 to 85 in steps of 1/64, a row each: 0 at one expert, -d at another, nothing anywhere else."""
    d = np.arange(4096) / 64.0
    d = np.where(d > 63, 63 + 22 * (d - 63), d)  # the last ones up to 85
    x = np.full((4096, E), -np.inf, np.float32)
    x[:, at[0]] = 0.0
    x[:, at[1]] = -d
    assert np.array_equal(x[:, at[1]].astype(np.float64), -d)
    return d, torch.from_numpy(x).to(DEV)


@pytest.mark.parametrize("E,at", [(2, (0, 1)), (64, (40, 3)), (256, (17, 255)), (1024, (1000, 5))])
def test_weights_and_gradient_at_any_distance(E, at):
    d, x = _rows(E, at)
    T = len(d)
    e = np.exp(-d)
    o = dict(idx=torch.empty(T, 2, dtype=torch.int32, device=DEV), w=torch.empty(T, 2, device=DEV),
             counts=torch.empty(E + 1, dtype=torch.int32, device=DEV), load=torch.empty(E, device=DEV), loss=torch.empty(1, device=DEV))
    ws = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, T, E, 2), dtype=torch.uint8, device=DEV)
    for renorm in (False, True):
        dg.dg_moe_gate(x, *o.values(), renorm=renorm, workspace=ws)
        w = o["w"].double().cpu().numpy()
        err = np.abs(w - np.stack([1 / (1 + e), e / (1 + e)], 1)) / np.stack([1 / (1 + e), e / (1 + e)], 1)
        assert err.max() <= 8 * U, (renorm, err.max() / U, d[err.max(1).argmax()])
    # one choice a token, the balance loss alone: g is 1 at the expert that every token chooses and 0 elsewhere
    idx = torch.full((T, 1), at[0], dtype=torch.int32, device=DEV)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    counts[at[0]] = counts[E] = T
    got = torch.empty_like(x)
    dg.dg_moe_gate_bwd(x, idx, torch.ones(T, 1, device=DEV), counts, None, torch.full((1,), T / E, device=DEV), got, loss_coef=1.0)
    g = got.double().cpu().numpy()
    want = e / (1 + e) ** 2
    err = np.abs(g[:, at[1]] + want) / want
    assert err.max() <= 16 * U, (err.max() / U, d[err.argmax()])
