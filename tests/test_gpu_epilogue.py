"""The FP8 product's epilogue form and its gradient on the GPU against the 64-bit oracle.

Bounds (u = 2^-24).  z: helpers.acc_tolerance, t (the matrix cores' truncation and the fp32 sums), with the bias in place of
C.  An activation's slope is below 1.2, its own fp32 error at most (16 + 8 |z|) u of max(|z|, 1) (sigmoid: the exponent's
rounding, 2 |z| u relative of e^-z, weighs p (1 - p); gelu: 7.5e-8 of the normal distribution's table formula and a few
roundings).  D: 1.2 t, that, a rounding of the sum with the residual and half a step of bf16 (2^-8).  dz: (32 + 8 |z|) u |dy|
and 2^-8 |dz|; dbias: that and (M + 40) u of the sum of |dz|; codes and scales as in test_gpu_norm.py, E = that of dz."""

import numpy as np
import pytest
import torch

import oracle
from helpers import acc_tolerance
from moe_grouped_matmul_amd import dg
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0**-24
STEP = 2.0**-8


def _np(t):
    return t.double().cpu().numpy()


def _operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    qa, sa = oracle.quant_1x128(rng.normal(size=(M, K)).astype(np.float32))
    qb, sb = oracle.quant_128x128((rng.normal(size=(N, K)) / np.sqrt(K)).astype(np.float32))
    bias = rng.normal(size=N).astype(np.float32)
    res = torch.from_numpy(rng.normal(size=(M, N)).astype(np.float32)).to(torch.bfloat16)
    return qa, sa, qb, sb, bias, res


def _dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in arrays]


def _ws(M, N, K):
    return torch.zeros(max(16, dg.dg_get_workspace_size(dg.DG_OP_GEMM_NT, M, N, K)), dtype=torch.uint8, device=DEV)


def _z(qa, sa, qb, sb):
    K = qa.shape[1]
    a = oracle.decode_e4m3(qa) * np.repeat(sa.T.astype(np.float64), 128, 1)
    b = oracle.decode_e4m3(qb) * np.repeat(np.repeat(sb.astype(np.float64), 128, 0)[: qb.shape[0]], 128, 1)[:, :K]
    return a @ b.T


def _check(M, N, K, kind, bias, residual, pre, seed=0):
    qa, sa, qb, sb, b, r = _operands(M, N, K, seed)
    dA, dsa, dB, dsb, db = _dev(qa, sa, qb, sb, b)
    D = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    Z = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _ws(M, N, K)
    dg.dg_fp8_gemm_nt_epilogue(dA, dsa, dB, dsb, D[:M], bias=db if bias else None, act=kind, residual=r.to(DEV) if residual else None,
                               pre=Z[:M] if pre else None, workspace=ws)
    assert (D[M] == 7).all() and (Z[M] == 7).all() and (pre or (Z == 7).all())  # nothing past the rows
    assert not ws[:4096].any()  # counters back at zero
    z = _z(qa, sa, qb, sb) + (b.astype(np.float64) if bias else 0.0)
    t = acc_tolerance(qa, sa, qb, sb, np.broadcast_to(b, z.shape) if bias else None)
    want = block.act(z, kind) + (_np(r) if residual else 0.0)
    mag = np.abs(block.act(z, kind)) + (np.abs(_np(r)) if residual else 0.0)
    tol = 1.2 * t + (16 + 8 * np.abs(z)) * U * np.maximum(np.abs(z), 1) + U * mag
    bad = ~(np.abs(_np(D[:M]) - want) <= tol + STEP * (np.abs(want) + tol))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())
    if pre:
        bad = ~(np.abs(_np(Z[:M]) - z) <= t + STEP * (np.abs(z) + t))
        assert not bad.any(), ("pre", int(bad.sum()), np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("kind", block.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (5, 144, 256), (64, 272, 1024), (65, 2112, 384), (128, 528, 896), (200, 400, 512)])
def test_few_rows(M, N, K, kind):
    i = block.ACTS.index(kind) + M
    _check(M, N, K, kind, i % 2 == 0, i % 3 != 0, i % 2 == 1 or M == 65)


@pytest.mark.parametrize("kind", block.ACTS)
@pytest.mark.parametrize("tile", ["wide", "persistent"])
@pytest.mark.parametrize("M,N,K", [(257, 272, 256), (300, 528, 640), (513, 784, 384)])
def test_tile_kernels(M, N, K, tile, kind, monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", f"kernel={tile}")
    i = block.ACTS.index(kind) + M
    for residual in (True, False):
        _check(M, N, K, kind, (i + residual) % 2 == 0, residual, i % 3 != 0)


@pytest.mark.parametrize("cfg", ["64x16x1x4", "64x16x3x4", "64x32x2x4", "128x16x2x6", "128x32x1x4", "64x16x2x8"])
def test_decode_configurations(cfg, monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", f"skinny={cfg}")
    for kind, residual in (("silu", True), ("gelu", False)):
        _check(100, 272, 1024, kind, True, residual, True)


def test_row_chunks(monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", "chunk_rows=256")
    _check(700, 272, 256, "gelu_tanh", True, True, True)


@pytest.mark.parametrize("M,N,K", [(64, 2112, 7168), (100, 272, 1024), (640, 1024, 512), (1024, 4096, 1024), (4096, 4096, 512), (2100, 2112, 512)])
def test_without_an_epilogue_it_is_the_plain_product(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(0)
    A, B = (torch.randn(n, K, device=DEV, generator=g).to(torch.float8_e4m3fn) for n in (M, N))
    sa, sb = torch.rand(K // 128, M, device=DEV, generator=g) + 0.5, torch.rand((N + 127) // 128, K // 128, device=DEV, generator=g) + 0.5
    plain, D, Z = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    ws = _ws(M, N, K)
    dg.dg_fp8_gemm_nt(A, sa, B, sb, plain, workspace=ws)
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, workspace=ws)
    assert torch.equal(D, plain)
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, act="relu", pre=Z, workspace=ws)
    assert torch.equal(Z, plain) and torch.equal(D, torch.relu(plain))
    # the residual in place
    res = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16)
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, residual=res, workspace=ws)
    over = res.clone()
    dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, over, residual=over, workspace=ws)
    assert torch.equal(over, D)


def test_large_arguments_of_the_activations():
    # z = bias alone (A is zero): far tails, infinities, NaN
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 11.0, -11.0, 40.0, -40.0, 3e4, -3e4, 1e30, -1e30, float("inf"), float("nan"), 0.5, -0.5], device=DEV)
    N, K = 16, 128
    A, B = torch.zeros(3, K, dtype=torch.uint8, device=DEV), torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    sa, sb = torch.ones(1, 3, device=DEV), torch.ones(1, 1, device=DEV)
    for kind in block.ACTS:
        D = torch.empty(3, N, dtype=torch.bfloat16, device=DEV)
        dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=z, act=kind)
        got = _np(D)
        assert (got[:, 13] != got[:, 13]).all() and (got[:, 12] == np.inf).all()
        with np.errstate(over="ignore", invalid="ignore"):
            want = block.act(_np(z), kind)
        if kind == "gelu_tanh":
            want[10], want[11] = 1e30, 0.0  # (the oracle's cube stays finite; its tanh is 1)
        ok = [i for i in range(16) if i not in (12, 13)]
        assert (np.abs(got[:, ok] - want[ok]) <= STEP * np.abs(want[ok]) + 1e-6).all(), kind


def _bwd_ws(M, N):
    return torch.full((dg.dg_get_workspace_size(dg.DG_OP_EPILOGUE_BWD, M, N, 0),), 0x7F, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("kind", block.ACTS)
@pytest.mark.parametrize("M,N", [(1, 16), (3, 128), (17, 640), (64, 144), (100, 1024), (1000, 2048), (5000, 384), (33, 16384)])
def test_gradient(M, N, kind):
    g = torch.Generator(device=DEV).manual_seed(M)
    dy, z = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16), (2 * torch.randn(M, N, device=DEV, generator=g)).to(torch.bfloat16)
    quant = N % 128 == 0
    dz = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    q = torch.full((M, N), 0x55, dtype=torch.uint8, device=DEV) if quant else None
    sf = torch.full((N // 128, M), 7.0, device=DEV) if quant else None
    db, ws = torch.full((N,), 7.0, device=DEV), _bwd_ws(M, N)
    before = ws[:4096].clone()
    dg.dg_epilogue_bwd(dy, dz, pre=None if kind == "none" else z, act=kind, q=q, sf=sf, dbias=db, workspace=ws)
    assert torch.equal(ws[:4096], before)
    zn, dyn = _np(z), _np(dy)
    want = dyn * block.act_slope(zn, kind)
    err = (32 + 8 * np.abs(zn)) * U * np.abs(dyn)
    assert (np.abs(_np(dz) - want) <= err + STEP * (np.abs(want) + err)).all()
    assert (np.abs(_np(db) - want.sum(0)) <= err.sum(0) + (M + 40) * U * np.abs(want).sum(0)).all()
    if quant:
        amax, e = np.abs(want).reshape(M, N // 128, 128).max(2), err.reshape(M, N // 128, 128).max(2)
        s = _np(sf).T
        assert (np.abs(s * 448 - amax)[amax > 0] <= (e + 2 * U * amax)[amax > 0]).all() and (s[amax == 0] == 1).all()
        s = np.repeat(s, 128, 1)
        back = oracle.decode_e4m3(q.cpu().numpy()) * s
        assert (np.abs(back - want) <= np.maximum(2.0**-4 * np.abs(want), 2.0**-10 * s) * (1 + 8 * U) + 2 * err + 8 * U * np.abs(want)).all()
    # outputs on their own and in place are the same bits
    dz2, db2 = dy.clone(), torch.empty_like(db)
    dg.dg_epilogue_bwd(dz2, dz2, pre=None if kind == "none" else z, act=kind)
    assert torch.equal(dz2, dz)
    dg.dg_epilogue_bwd(dy, pre=None if kind == "none" else z, act=kind, dbias=db2, workspace=ws)
    assert torch.equal(db2, db)
    if quant:
        q2, sf2 = torch.empty_like(q), torch.empty_like(sf)
        dg.dg_epilogue_bwd(dy, pre=None if kind == "none" else z, act=kind, q=q2, sf=sf2)
        assert torch.equal(q2, q) and torch.equal(sf2, sf)


def test_gradient_against_differences():
    # the product's own forward, moved by a step of the bias: sum(dy * D) / 2 t against dbias
    M, N, K, t = 6, 128, 256, 2.0**-5
    g = torch.Generator(device=DEV).manual_seed(3)
    A, B = (torch.randn(n, K, device=DEV, generator=g).to(torch.float8_e4m3fn) for n in (M, N))
    sa, sb = torch.full((K // 128, M), 0.25, device=DEV), torch.full((1, K // 128), 0.25, device=DEV)
    bias, dy = torch.randn(N, device=DEV, generator=g), torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16)
    D, Z = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for kind in block.ACTS[2:]:
        f = []
        for sign in (-1, 1):
            dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=bias + sign * t, act=kind)
            f.append(D.double().clone())
        dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=bias, act=kind, pre=Z)
        db = torch.empty(N, device=DEV)
        dg.dg_epilogue_bwd(dy, pre=Z, act=kind, dbias=db, workspace=_bwd_ws(M, N))
        diff = ((f[1] - f[0]) * dy.double()).sum(0) / (2 * t)
        # bf16 roundings of the two D over 2 t, curvature t^2 (third derivatives below 1), the rounding of pre (slopes of the slope below 1)
        tol = (dy.double().abs() * (STEP * D.double().abs() * 1.2 / t + t * t + STEP * Z.double().abs() + STEP * 2 / t * t)).sum(0)
        assert ((diff - db.double()).abs() <= tol).all()


def test_gradient_of_far_arguments():
    z = torch.tensor([3e38, -3e38, 1e20, -1e20, 50.0, -50.0, 12.0, -12.0, 0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 2.0, -2.0], device=DEV).to(torch.bfloat16)[None].contiguous()
    dy = torch.ones_like(z)
    for kind in block.ACTS[1:]:
        dz = torch.empty_like(z)
        dg.dg_epilogue_bwd(dy, dz, pre=z, act=kind)
        with np.errstate(over="ignore", invalid="ignore"):
            want = block.act_slope(np.clip(_np(z), -100, 100), kind)
        assert (np.abs(_np(dz) - want) <= STEP * np.abs(want) + 1e-6).all(), kind


def test_without_rows():
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    db = torch.full((256,), 7.0, device=DEV)
    dg.dg_epilogue_bwd(e, e, pre=e, act="gelu", dbias=db, workspace=_bwd_ws(0, 256))
    assert (db == 0).all()


def test_graph_replays():
    M, N, K = 96, 512, 1024
    g0 = torch.Generator(device=DEV).manual_seed(0)
    A, B = (torch.randn(n, K, device=DEV, generator=g0).to(torch.float8_e4m3fn).view(torch.uint8) for n in (M, N))
    sa, sb = torch.full((K // 128, M), 0.1, device=DEV), torch.full((N // 128, K // 128), 0.1, device=DEV)
    bias, dy = torch.randn(N, device=DEV, generator=g0), torch.randn(M, N, device=DEV, generator=g0).to(torch.bfloat16)
    D, Z, dz = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    q, sf, db = torch.empty(M, N, dtype=torch.uint8, device=DEV), torch.empty(N // 128, M, device=DEV), torch.empty(N, device=DEV)
    ws = torch.zeros(max(dg.dg_get_workspace_size(dg.DG_OP_GEMM_NT, M, N, K), dg.dg_get_workspace_size(dg.DG_OP_EPILOGUE_BWD, M, N, 0)),
                     dtype=torch.uint8, device=DEV)  # one for both

    def calls():
        dg.dg_fp8_gemm_nt_epilogue(A, sa, B, sb, D, bias=bias, act="gelu", pre=Z, workspace=ws)
        dg.dg_epilogue_bwd(dy, dz, pre=Z, act="gelu", q=q, sf=sf, dbias=db, workspace=ws)

    outs = (D, Z, dz, q, sf, db)
    calls()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for i in range(3):
        A.copy_(torch.randn(M, K, device=DEV, generator=g0).to(torch.float8_e4m3fn).view(torch.uint8))
        calls()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_binding_refusals():
    z = torch.zeros(8, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="act"):
        dg.dg_epilogue_bwd(z, z.clone(), pre=z, act="tanh")
    with pytest.raises(ValueError, match="pre"):
        dg.dg_epilogue_bwd(z, z.clone(), pre=z[:4], act="relu")
    with pytest.raises(TypeError, match="dy"):
        dg.dg_epilogue_bwd(z.float(), z, pre=z, act="relu")
    with pytest.raises(dg.DGError, match="workspace"):
        dg.dg_epilogue_bwd(z, pre=z, act="relu", dbias=torch.empty(128, device=DEV))
    A, sa, sb = torch.zeros(8, 128, dtype=torch.uint8, device=DEV), torch.ones(1, 8, device=DEV), torch.ones(1, 1, device=DEV)
    with pytest.raises(ValueError, match="bias"):
        dg.dg_fp8_gemm_nt_epilogue(A, sa, A, sb, torch.empty(8, 8, dtype=torch.bfloat16, device=DEV), bias=torch.ones(128, device=DEV))
    with pytest.raises(dg.DGError, match="multiple of 16"):
        dg.dg_fp8_gemm_nt_epilogue(A, sa, A, sb, torch.empty(8, 8, dtype=torch.bfloat16, device=DEV))
