"""One workspace buffer handed from operator to operator: the first 4 KiB of every operator's workspace are counters that are
zero between calls, so whatever ran before on the buffer, each call gives what it gives on a buffer of its own."""

import itertools

import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _gate(T, E, k):
    x = torch.randn(T, E, device=DEV, generator=_gen(T))

    def call(ws):
        o = [torch.full((T, k), 77, **I32), torch.full((T, k), 7.0, device=DEV), torch.full((E + 1,), 7, **I32),
             torch.full((E,), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)]
        dg.dg_moe_gate(x, *o, loss_coef=0.5, workspace=ws)
        return o

    return call, dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, T, E, k)


def _layout(T, k, G, max_m=0):
    idx = torch.randint(0, G, (T, k), generator=_gen(G), **I32)
    M = (T * k + 127 * G + 127) // 128 * 128

    def call(ws):
        shapes = ((G,), (G, max_m), (T, k)) if max_m else ((G,), (M,), (M,), (T, k))
        o = [torch.full(s, 77, **I32) for s in shapes]
        (dg.dg_moe_layout_masked if max_m else dg.dg_moe_layout_contiguous)(idx, *o, workspace=ws)
        return o

    return call, dg.dg_get_workspace_size(dg.DG_OP_MOE_LAYOUT, T, 0, k, G)


def _mxfp4(M, N, K):
    g = _gen(K)
    a, b = (torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, device=DEV, generator=g) for n in (M, N))
    sa, sb = (torch.full((K // 128, n), 0x7F7F7F7F, **I32) for n in (M, N))

    def call(ws):
        d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
        dg.dg_mxfp4_gemm_nt(a, sa, b, sb, d, workspace=ws)
        return [d]

    return call, dg.dg_get_workspace_size(dg.DG_OP_MXFP4_GEMM_NT, M, N, K)


def _fp8(M, N, K):
    g = _gen(N)
    a, b = (torch.randn(n, K, device=DEV, generator=g).to(torch.float8_e4m3fn) for n in (M, N))
    sa, sb = torch.ones(K // 128, M, device=DEV), torch.ones((N + 127) // 128, K // 128, device=DEV)

    def call(ws):
        d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
        dg.dg_fp8_gemm_nt(a, sa, b, sb, d, workspace=ws)
        return [d]

    return call, dg.dg_get_workspace_size(dg.DG_OP_GEMM_NT, M, N, K)


def _bf16(M, N, K):
    g = _gen(M)
    a, b = (torch.randn(n, K, device=DEV, generator=g).to(torch.bfloat16) for n in (M, N))

    def call(ws):
        d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
        dg.dg_bf16_gemm_nt(a, b, d, workspace=ws)
        return [d]

    return call, dg.dg_get_workspace_size(dg.DG_OP_BF16_GEMM_NT, M, N, K)


# the gate of one group of workgroups and of several; row orders of one launch, of 16-bit and of 32-bit counts; products that split K
CALLS = {"gate": lambda: _gate(700, 256, 8), "gate_groups": lambda: _gate(5000, 60, 4), "layout": lambda: _layout(5000, 8, 64),
         "layout_masked": lambda: _layout(3000, 4, 256, 32), "layout_many": lambda: _layout(70000, 4, 1024),
         "layout_one": lambda: _layout(100, 8, 64), "mxfp4": lambda: _mxfp4(64, 4112, 7168), "fp8": lambda: _fp8(64, 4608, 7168),
         "bf16": lambda: _bf16(64, 2112, 7168)}


def test_every_operator_after_every_other():
    calls = {n: make() for n, make in CALLS.items()}
    for n in ("mxfp4", "fp8", "bf16"):
        assert calls[n][1] > 4096, n  # K is split
    alone = {n: call(torch.zeros(size, dtype=torch.uint8, device=DEV)) for n, (call, size) in calls.items()}
    size = max(size for _, size in calls.values())
    for a, b in itertools.permutations(calls, 2):
        ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
        for n in (a, b, a, b):
            got = calls[n][0](ws)
            assert all(torch.equal(x, y) for x, y in zip(got, alone[n])), (a, b, n)
        assert not bool(ws[:4096].any()), (a, b)


def test_gate_and_layout_leave_counters_alone_at_their_own_size():
    """A buffer of exactly the queried size, which a split product with a small plan then takes."""
    for n in ("gate", "gate_groups", "layout", "layout_masked", "layout_many"):
        call, size = CALLS[n]()
        ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
        guard = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device=DEV)
        guard[:size] = 0
        first = call(ws)
        again = call(guard[:size])
        assert all(torch.equal(x, y) for x, y in zip(first, again)), n
        assert bool((guard[size:] == 0xA5).all()), n
        assert not bool(ws[: min(size, 4096)].any()), n


def test_row_order_in_a_buffer_for_more_choices():
    G = 64
    size = dg.dg_get_workspace_size(dg.DG_OP_MOE_LAYOUT, 400000, 0, 1, G)
    guard = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    for T, k in ((400000, 1), (16384, 8), (131073, 1), (2049, 1), (32768, 8), (300, 2)):
        call, own = _layout(T, k, G)
        alone = call(torch.zeros(own, dtype=torch.uint8, device=DEV))
        assert all(torch.equal(x, y) for x, y in zip(call(guard[:size]), alone)), (T, k)
        assert bool((guard[size:] == 0xA5).all()) and bool((guard[:4096] == 0xA5).all())
