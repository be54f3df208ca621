"""The experts for a few tokens on streams of the caller's, and two calls at once on two streams: each with weights, tokens,
routing and a workspace of its own.  Bit for bit the results of the calls one after the other, counters at zero afterwards."""

import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _experts(fmt, T, k, E, H, inner, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def weight(N, K):
        w = torch.randn(E, N, K, device=DEV, generator=g) / K**0.5
        if fmt == "fp8":
            q, s = torch.empty(E, N, K, dtype=torch.uint8, device=DEV), torch.empty(E, N // 128, K // 128, device=DEV)
            dg.dg_quant_128x128(w, q, s)
        else:
            q, s = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV), torch.empty(E, K // 128, N, dtype=torch.int32, device=DEV)
            dg.dg_quant_mxfp4(w, q, s)
        return q, s

    w1, w2 = weight(2 * inner, H), weight(H, inner)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    top = torch.topk(torch.randn(T, E, device=DEV, generator=g), k, dim=1)
    idx, w = top.indices.int(), torch.softmax(top.values, 1)
    idx[T // 2, 0] = -1
    y = torch.zeros_like(x)
    ws = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_EXPERTS, T * k, H, inner), dtype=torch.uint8, device=DEV)
    call = dg.dg_moe_experts_fp8 if fmt == "fp8" else dg.dg_moe_experts_mxfp4

    def run(stream=None):
        call(x, idx, w, *w1, *w2, y, workspace=ws, stream=stream)

    return run, y, ws


# few tokens, more than 16, many of an expert; columns that several workgroups share
CASES = [(1, 4, 16, 512, 512), (8, 4, 16, 512, 1024), (48, 4, 16, 512, 512), (64, 4, 8, 512, 1024)]


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("size", CASES)
def test_streams(size, fmt):
    run, y, ws = _experts(fmt, *size, 0)
    run()
    want = y.clone()
    assert want.any()
    for how in ("argument", "current"):
        y.zero_()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        if how == "argument":
            run(s)
        else:
            with torch.cuda.stream(s):
                run()
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want) and not ws[:4096].any(), how


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("sizes", [(CASES[0], CASES[0]), (CASES[1], CASES[3]), (CASES[3], CASES[3]), (CASES[2], CASES[1])])
def test_two_at_once(sizes, fmt):
    calls = [_experts(fmt, *size, 1 + i) for i, size in enumerate(sizes)]
    want = []
    for run, y, _ in calls:
        run()
        want.append(y.clone())
        y.zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for (run, _, _), s in zip(calls, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, y, ws), w in zip(calls, want):
        assert torch.equal(y, w) and not ws[:4096].any()


def test_two_formats_at_once():
    calls = [_experts("fp8", *CASES[3], 3), _experts("mxfp4", *CASES[2], 4)]
    want = []
    for run, y, _ in calls:
        run()
        want.append(y.clone())
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for (run, _, _), s in zip(calls, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, y, ws), w in zip(calls, want):
        assert torch.equal(y, w) and not ws[:4096].any()
