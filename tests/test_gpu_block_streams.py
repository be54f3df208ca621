"""The operators between the products on a stream of the caller's, given as an argument and as torch's current stream, beside
other work; two calls at once on two streams, each with a workspace of its own."""

import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ws(op, *size):
    return torch.zeros(max(16, dg.dg_get_workspace_size(op, *size)), dtype=torch.uint8, device=DEV)


def _product(seed):
    M, N, K = 100, 528, 1024
    g = torch.Generator(device=DEV).manual_seed(seed)
    A, B = (torch.randn(n, K, device=DEV, generator=g).to(torch.float8_e4m3fn) for n in (M, N))
    sa, sb = torch.rand(K // 128, M, device=DEV, generator=g), torch.rand((N + 127) // 128, K // 128, device=DEV, generator=g)
    bias, res = torch.randn(N, device=DEV, generator=g), torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16)
    D, Z, dz = (torch.zeros(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    db, w1, w2 = torch.zeros(N, device=DEV), _ws(dg.DG_OP_GEMM_NT, M, N, K), _ws(dg.DG_OP_EPILOGUE_BWD, M, N, 0)

    def run(stream=None):
        dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=bias, act="gelu", residual=res, pre=Z, workspace=w1, stream=stream)
        dg.dg_epilogue_bwd(res, dz, pre=Z, act="gelu", dbias=db, workspace=w2, stream=stream)

    return run, (D, Z, dz, db)


def _norm(seed):
    M, K = 300, 2048
    g = torch.Generator(device=DEV).manual_seed(seed)
    x, dy = (torch.randn(M, K, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    w = 1 + 0.2 * torch.randn(K, device=DEV, generator=g)
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    rstd, dw, ws = torch.zeros(M, device=DEV), torch.zeros(K, device=DEV), _ws(dg.DG_OP_RMS_NORM_BWD, M, 0, K)

    def run(stream=None):
        dg.dg_rms_norm(x, w, y=y, rstd=rstd, stream=stream)
        dg.dg_rms_norm_bwd(dy, x, w, rstd, dx, dw, workspace=ws, stream=stream)

    return run, (y, rstd, dx, dw)


@pytest.mark.parametrize("make", [_product, _norm])
def test_streams(make):
    run, outs = make(0)
    run()
    want = [t.clone() for t in outs]
    for how in ("argument", "current"):
        for t in outs:
            t.zero_()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        if how == "argument":
            run(s)
        else:
            with torch.cuda.stream(s):
                run()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), how


@pytest.mark.parametrize("make", [_product, _norm])
def test_two_at_once(make):
    calls = [make(seed) for seed in (1, 2)]
    want = []
    for run, outs in calls:
        run()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for (run, _), s in zip(calls, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
