"""The printed plan of the epilogue form is the one that runs: it has the ring of each tile shape's default depth only, whatever
depth DG_FORCE_CONFIG asks for, and splits K for that one."""

import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("cfg,depth", [("64x16x2x8", 4), ("64x16x3x8", 4), ("64x32x2x6", 4), ("128x16x2x6", 6), ("64x16x3x4", 4)])
def test_depth_of_the_epilogue_form(cfg, depth, monkeypatch, capfd):
    M, N, K = 100, 272, 1664
    g = torch.Generator(device=DEV).manual_seed(0)
    A, B = (torch.randn(n, K, device=DEV, generator=g).to(torch.float8_e4m3fn) for n in (M, N))
    sa, sb = torch.rand(K // 128, M, device=DEV, generator=g) + 0.5, torch.rand((N + 127) // 128, K // 128, device=DEV, generator=g) + 0.5
    D, want = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device=DEV)
    shape, _, asked = cfg.rpartition("x")
    monkeypatch.setenv("DG_PRINT_CONFIGS", "1")
    monkeypatch.setenv("DG_FORCE_CONFIG", f"skinny={cfg}")
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, act="relu", workspace=ws)
    line = [s for s in capfd.readouterr().err.splitlines() if "gemm_nt_epilogue" in s][-1]
    assert f" depth={depth} " in line, line
    dg.dg_fp8_gemm_nt(A, sa, B, sb, want, workspace=ws)  # the other forms have the deeper rings
    line = [s for s in capfd.readouterr().err.splitlines() if "gemm_nt " in s][-1]
    assert f" depth={asked} " in line, line
    # the same split as the plain form's at that depth, so the same sums
    monkeypatch.setenv("DG_FORCE_CONFIG", f"skinny={shape}x{depth}")
    dg.dg_fp8_gemm_nt(A, sa, B, sb, want, workspace=ws)
    assert torch.equal(D, torch.relu(want))
