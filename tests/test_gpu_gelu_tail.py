"""The activations of the product's epilogue where they are small: relative to their own value, not to their argument.

z is the bias alone (A is zero), so it is exact.  The tail Phi(-a) e^(a^2 / 2) is fitted to 5.1e-5 of itself, the exponent
-a^2 / 2 log2 e, up to 121 in magnitude, has three roundings (121 * 3 * 2^-24 * ln 2 = 1.5e-5 of the value), and what is left is
some ten roundings: below 7e-5.  The exponents of the sigmoids of silu and gelu_tanh, up to 124, have 1.5 and 6.5 roundings: 8e-6
and 3.4e-5.  D is rounded once to bf16: (2^-8 + 1e-4) of the value.  The values are above 2^-126, the sigmoids too."""

import math

import numpy as np
import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M,force", [(3, None), (100, None), (300, "kernel=wide"), (300, "kernel=persistent")])
def test_gelu_is_right_relative_to_its_value(M, force, monkeypatch):
    if force:
        monkeypatch.setenv("DG_FORCE_CONFIG", force)
    z = np.concatenate([np.linspace(-12.9, 12.9, 3056), -np.logspace(-30, 0, 520), np.logspace(-30, 0, 520)]).astype(np.float32)
    N, K = len(z), 128
    A, B = (torch.zeros(n, K, dtype=torch.uint8, device=DEV) for n in (M, N))
    sa, sb = torch.ones(1, M, device=DEV), torch.ones((N + 127) // 128, 1, device=DEV)
    D = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=torch.from_numpy(z).to(DEV), act="gelu")
    want = np.array([0.5 * v * math.erfc(-v / math.sqrt(2.0)) for v in z.astype(np.float64).tolist()])
    bad = ~(np.abs(D.double().cpu().numpy() - want) <= (2.0**-8 + 1e-4) * np.abs(want))
    assert not bad.any(), (int(bad.sum()), z[np.argwhere(bad)[:, 1]].min(), z[np.argwhere(bad)[:, 1]].max())


@pytest.mark.parametrize("kind,low", [("silu", -86.0), ("gelu_tanh", -9.9)])
def test_the_sigmoids_are_right_relative_to_their_values(kind, low):
    z = np.concatenate([np.linspace(low, -low, 3056), -np.logspace(-30, 0, 520), np.logspace(-30, 0, 520)]).astype(np.float32)
    N, K = len(z), 128
    A, B = (torch.zeros(n, K, dtype=torch.uint8, device=DEV) for n in (3, N))
    sa, sb = torch.ones(1, 3, device=DEV), torch.ones((N + 127) // 128, 1, device=DEV)
    D = torch.empty(3, N, dtype=torch.bfloat16, device=DEV)
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=torch.from_numpy(z).to(DEV), act=kind)
    v = z.astype(np.float64)
    want = v / (1.0 + np.exp(-(v if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v**3))))
    bad = ~(np.abs(D.double().cpu().numpy() - want) <= (2.0**-8 + 1e-4) * np.abs(want))
    assert not bad.any(), (int(bad.sum()), z[np.argwhere(bad)[:, 1]].min(), z[np.argwhere(bad)[:, 1]].max())


def test_infinities():
    # the limit where the formula has one without inf * 0, else NaN
    inf = float("inf")
    z = torch.tensor([-inf, inf] * 8, device=DEV)
    A, B = (torch.zeros(n, 128, dtype=torch.uint8, device=DEV) for n in (1, 16))
    D, dz = (torch.empty(1, 16, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    one, pre = torch.ones(1, 1, device=DEV), z.to(torch.bfloat16)[None].contiguous()
    for kind, low, slopes in (("none", -inf, (1, 1)), ("relu", 0, (0, 1)), ("silu", None, None), ("gelu", 0, None), ("gelu_tanh", None, (0, 1))):
        dg.dg_fp8_gemm_nt_epilogue(A, one, B, one, D, bias=z, act=kind)
        got = D.float()[0].tolist()
        assert all(v == inf for v in got[1::2]) and all(v != v if low is None else v == low for v in got[::2]), kind
        dg.dg_epilogue_bwd(torch.ones_like(pre), dz, pre=pre, act=kind)
        got = dz.float()[0].tolist()
        assert all(v != v for v in got) if slopes is None else (got == list(slopes) * 8), kind
