"""Norm, epilogue and their gradients past 32-bit offsets and at the largest counts: parts of a large call against the same rows
in a small one, whose bits must be the same, except where the order of a sum depends on the number of rows (a row of the norm is
summed by one to sixteen waves, fewer the more rows there are): those parts against the 64-bit oracle, within the bounds of
test_gpu_norm.py."""

import pytest
import torch

from moe_grouped_matmul_amd import dg
from oracle import block
from test_gpu_norm import U, _check_codes, _near, _np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _fill(t, seed):
    """Normal values in pieces (no fp32 copy of the whole)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    for i in range(0, t.shape[0], 1 << 14):
        t[i:i + (1 << 14)] = torch.randn(t[i:i + (1 << 14)].shape, device=DEV, generator=g).to(t.dtype)
    return t


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_norm_past_32_bit_offsets():
    M, K = 270001, 16384  # 4.4e9 elements
    x, res = (_fill(torch.empty(M, K, dtype=torch.bfloat16, device=DEV), i) for i in range(2))
    w = 1 + 0.1 * torch.randn(K, device=DEV)
    q, sf, rstd = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(K // 128, M, device=DEV), torch.empty(M, device=DEV)
    parts = [slice(0, 3), slice(131070, 131075), slice(262142, 262147), slice(M - 3, M)]  # about 2^31 and 2^32 elements, the ends
    want = [(x[p].double() + res[p].double()).to(torch.bfloat16) for p in parts]
    dg.dg_rms_norm(x, w, residual=res, h=res, q=q, sf=sf, rstd=rstd)  # the stream in place
    for p, h in zip(parts, want):
        assert torch.equal(res[p], h)
        v, r = block.rms_norm(_np(h), _np(w), 1e-6)
        _near(rstd[p], r, 80 * U * r, "rstd")
        _check_codes(q[p], sf[:, p].contiguous(), v, p.stop - p.start, K)
    # the gradient over x (its result goes there)
    dy = _fill(torch.empty(M, K, dtype=torch.bfloat16, device=DEV), 5)
    dw, ws = torch.empty(K, device=DEV), torch.empty(dg.dg_get_workspace_size(dg.DG_OP_RMS_NORM_BWD, M, 0, K), dtype=torch.uint8, device=DEV)
    dg.dg_rms_norm_bwd(dy, res, w, rstd, x, dw, workspace=ws)
    for p in parts:
        small = torch.empty(p.stop - p.start, K, dtype=torch.bfloat16, device=DEV)
        dg.dg_rms_norm_bwd(dy[p].contiguous(), res[p].contiguous(), w, rstd[p].contiguous(), small, torch.empty(K, device=DEV), workspace=ws)
        assert torch.equal(x[p], small)


def test_norm_of_the_most_rows():
    M, K = (1 << 23) - 1, 8
    x, y = _fill(torch.empty(M, K, dtype=torch.bfloat16, device=DEV), 0), torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    w, rstd = torch.rand(K, device=DEV) + 0.5, torch.empty(M, device=DEV)
    dg.dg_rms_norm(x, w, y=y, rstd=rstd)
    want = torch.rsqrt(x.float().square().mean(1) + 1e-6)
    assert (rstd - want).abs().max() <= 1e-6 * want.max() and torch.equal((rstd == 0), torch.zeros_like(rstd, dtype=torch.bool))
    for p in (slice(0, 5), slice(M - 5, M)):
        small = torch.empty(5, K, dtype=torch.bfloat16, device=DEV)
        dg.dg_rms_norm(x[p].contiguous(), w, y=small)
        assert torch.equal(y[p], small)
    dx, dw = torch.empty_like(x), torch.empty(K, device=DEV)
    ws = torch.empty(dg.dg_get_workspace_size(dg.DG_OP_RMS_NORM_BWD, M, 0, K), dtype=torch.uint8, device=DEV)
    dg.dg_rms_norm_bwd(y, x, w, rstd, dx, dw, workspace=ws)
    want = (y.double() * x.double() * rstd.double()[:, None]).sum(0)
    assert ((dw.double() - want).abs() <= 1e-4 * (y.double() * x.double() * rstd.double()[:, None]).abs().sum(0)).all()


def test_epilogue_gradient_past_32_bit_offsets():
    M, N = 1100001, 4096  # 4.5e9 elements
    dy, z = (_fill(torch.empty(M, N, dtype=torch.bfloat16, device=DEV), i) for i in range(2))
    q, sf, db = torch.empty(M, N, dtype=torch.uint8, device=DEV), torch.empty(N // 128, M, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(dg.dg_get_workspace_size(dg.DG_OP_EPILOGUE_BWD, M, N, 0), dtype=torch.uint8, device=DEV)
    parts = [slice(0, 3), slice(524286, 524291), slice(1048574, 1048579), slice(M - 3, M)]
    want = []
    for p in parts:
        n = p.stop - p.start
        o = [torch.empty(n, N, dtype=torch.bfloat16, device=DEV), torch.empty(n, N, dtype=torch.uint8, device=DEV), torch.empty(N // 128, n, device=DEV)]
        dg.dg_epilogue_bwd(dy[p].contiguous(), o[0], pre=z[p].contiguous(), act="silu", q=o[1], sf=o[2])
        want.append(o)
    dg.dg_epilogue_bwd(dy, z, pre=z, act="silu", q=q, sf=sf, dbias=db, workspace=ws)  # over what the forward pass kept
    for p, o in zip(parts, want):
        assert torch.equal(z[p], o[0]) and torch.equal(q[p], o[1]) and torch.equal(sf[:, p], o[2])
    total = sum(z[i:i + (1 << 16)].double().sum(0) for i in range(0, M, 1 << 16))
    mag = sum(z[i:i + (1 << 16)].double().abs().sum(0) for i in range(0, M, 1 << 16))
    # dbias sums before the rounding to bf16: half a step each of the stored values, and the fp32 sums of 1100001 / 1024 rows and 1024 parts
    assert ((db.double() - total).abs() <= (2.0**-8 + 2400 * 2.0**-24) * mag).all()


def test_epilogue_in_row_chunks_of_32_bit_offsets():
    M, N, K = 400000, 8192, 128  # 6.6 GB of output: more than one launch addresses
    g = torch.Generator(device=DEV).manual_seed(0)
    A = torch.randn(M, K, device=DEV, generator=g).to(torch.float8_e4m3fn)
    B = torch.randn(N, K, device=DEV, generator=g).to(torch.float8_e4m3fn)
    sa, sb = torch.rand(1, M, device=DEV, generator=g) + 0.5, torch.rand(N // 128, 1, device=DEV, generator=g) + 0.5
    bias = torch.randn(N, device=DEV, generator=g)
    D = _fill(torch.empty(M, N, dtype=torch.bfloat16, device=DEV), 3)
    pre = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(max(16, dg.dg_get_workspace_size(dg.DG_OP_GEMM_NT, M, N, K)), dtype=torch.uint8, device=DEV)
    rows = [0, 100000, 262143, 262144, 299999, M - 300]
    want = []
    for r in rows:
        p = slice(r, r + 300)
        d, z = torch.empty(300, N, dtype=torch.bfloat16, device=DEV), torch.empty(300, N, dtype=torch.bfloat16, device=DEV)
        dg.dg_fp8_gemm_nt_epilogue(A[p].contiguous(), sa[:, p].contiguous(), B, sb, d, bias=bias, act="gelu", residual=D[p].contiguous(), pre=z, workspace=ws)
        want.append((d, z))
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=bias, act="gelu", residual=D, pre=pre, workspace=ws)
    for r, (d, z) in zip(rows, want):
        assert torch.equal(D[r:r + 300], d) and torch.equal(pre[r:r + 300], z)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_experts_past_32_bit_offsets(fmt):
    G, H, inner, T = 400, 4096, 2048, 5  # 6.7 GB of gate and up weights in fp8
    g = torch.Generator(device=DEV).manual_seed(0)
    per = 1 if fmt == "fp8" else 2

    def codes(*shape):
        q = torch.empty(shape, dtype=torch.uint8, device=DEV)
        for i in range(shape[0]):
            q[i] = torch.randint(0, 112, shape[1:], dtype=torch.uint8, device=DEV, generator=g) | (torch.randint(0, 2, shape[1:], dtype=torch.uint8, device=DEV, generator=g) << 7)
        return q

    q1, q2 = codes(G, 2 * inner, H // per), codes(G, H, inner // per)
    if fmt == "fp8":
        s1, s2 = (torch.rand(G, n // 128, k // 128, device=DEV, generator=g) * 1e-3 for n, k in ((2 * inner, H), (H, inner)))
        call = dg.dg_moe_experts_fp8
    else:  # codes 116..119 in each byte: 2^-11 .. 2^-8
        s1, s2 = (torch.randint(116, 120, (G, k // 128, n, 4), dtype=torch.uint8, device=DEV, generator=g).view(torch.int32)[..., 0].contiguous()
                  for n, k in ((2 * inner, H), (H, inner)))
        call = dg.dg_moe_experts_mxfp4
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    w = torch.rand(T, 1, device=DEV, generator=g) + 0.5
    ws = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_EXPERTS, T, H, inner), dtype=torch.uint8, device=DEV)
    one = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    for e in (0, 127, 128, 255, 256, 399):
        y, alone = torch.empty_like(x), torch.empty_like(x)
        call(x, one + e, w, q1, s1, q2, s2, y, workspace=ws)
        call(x, one, w, q1[e:e + 1], s1[e:e + 1], q2[e:e + 1], s2[e:e + 1], alone, workspace=ws)
        assert y.isfinite().all() and y.abs().max() > 0 and torch.equal(y, alone)
