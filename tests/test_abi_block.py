"""Host-side refusals of the norm, of the epilogue form and of their gradients (no GPU needed): every status code from
arguments that fail before any device work, sizes of the workspaces, and what calls with nothing to do return."""

import ctypes
import os

import pytest

from moe_grouped_matmul_amd import dg

P = 0x10000      # fake, never dereferenced
S, A, V, W, OK = dg.DG_ERR_SHAPE, dg.DG_ERR_ALIGN, dg.DG_ERR_INVALID_ARG, dg.DG_ERR_WORKSPACE, dg.DG_OK
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.LIB_PATH):
        from moe_grouped_matmul_amd import build

        build.build()
    return dg.load_library()


def _expect(lib, rc, want, text=""):
    msg = lib.dg_get_last_error().decode()
    assert rc == want, (rc, msg)
    assert (msg == "") == (want == OK) and text in msg


def _norm(lib, x=P, residual=P, weight=P, dtype=1, wt=1, h=P, y=None, q=P, sf=P, kind=0, rstd=P, M=4, K=256, eps=1e-6):
    return lib.dg_rms_norm(x, residual, weight, dtype, wt, h, y, q, sf, kind, rstd, M, K, eps, NULL)


def test_norm(lib):
    for kw, want, text in [
        (dict(dtype=2), V, "dtypes"), (dict(wt=-1), V, "dtypes"), (dict(kind=2), V, "scale_kind"),
        (dict(eps=0.0), V, "eps"), (dict(eps=-1.0), V, "eps"), (dict(eps=float("nan")), V, "eps"), (dict(eps=float("inf")), V, "eps"),
        (dict(K=0), S, "K"), (dict(K=12), S, "K"), (dict(K=16392), S, "K"), (dict(M=-1), S, "M"), (dict(M=1 << 23), S, "M"),
        (dict(K=136), S, "128"), (dict(x=None), V, "null"), (dict(weight=None), V, "null"), (dict(h=None), V, "null"),
        (dict(q=None, sf=None), V, "null"), (dict(sf=None), V, "null"), (dict(q=None, y=P), V, "null"), (dict(y=P), V, "different"),
        (dict(x=P + 8), A, "16"), (dict(residual=P + 4), A, "16"), (dict(weight=P + 2), A, "16"), (dict(h=P + 8), A, "16"),
        (dict(y=P + 8), A, "16"), (dict(q=P + 8), A, "16"), (dict(sf=P + 2), A, "4"), (dict(rstd=P + 1), A, "4"),
    ]:
        _expect(lib, _norm(lib, **kw), want, text)
    _expect(lib, _norm(lib, x=None, weight=None, M=0), OK)  # nothing to do


def _norm_bwd(lib, dy=P, h=P, weight=P, rstd=P, dtype=1, wt=1, dh=None, dx=P, dw=P, M=4, K=256, ws=None, n=0):
    return lib.dg_rms_norm_bwd(dy, h, weight, rstd, dtype, wt, dh, dx, dw, M, K, ws, n, NULL)


def test_norm_bwd(lib):
    for kw, want, text in [
        (dict(dtype=2), V, "dtypes"), (dict(K=4), S, "K"), (dict(K=16392), S, "K"), (dict(M=-1), S, "M"), (dict(dy=None), V, "null"),
        (dict(h=None), V, "null"), (dict(rstd=None), V, "null"), (dict(dx=None), V, "null"), (dict(weight=None), V, "null"),
        (dict(dw=None, M=0), V, "null"), (dict(dy=P + 8), A, "16"), (dict(dh=P + 8), A, "16"), (dict(dx=P + 8), A, "16"),
        (dict(rstd=P + 2), A, "4"), (dict(dw=P + 2), A, "4"),
    ]:
        _expect(lib, _norm_bwd(lib, **kw), want, text)


def _epi(lib, A=P, sfa=P, B=P, sfb=P, bias=P, act=2, residual=P, pre=2 * P, D=P, M=4, N=32, K=256, ws=None, n=0):
    return lib.dg_fp8_gemm_nt_epilogue(A, sfa, B, sfb, bias, act, residual, pre, D, M, N, K, ws, n, NULL)


def test_epilogue(lib):
    for kw, want, text in [
        (dict(K=100), S, "K"), (dict(N=24), S, "N"), (dict(M=-1), S, "M"), (dict(act=5), V, "activation"), (dict(act=-1), V, "activation"),
        (dict(A=None), V, "null"), (dict(D=None), V, "null"), (dict(sfb=None), V, "null"), (dict(pre=P), V, "own"), (dict(pre=3 * P, residual=3 * P), V, "own"),
        (dict(A=P + 8), A, "16"), (dict(sfa=P + 2), A, "4"), (dict(bias=P + 4), A, "16"), (dict(residual=P + 8), A, "16"),
        (dict(pre=P + 8), A, "16"), (dict(ws=P + 4, n=64), W, "16"), (dict(ws=P, n=3), W, "multiple of 4"),
        (dict(N=1 << 24, K=1 << 10), S, "4 GiB"),
    ]:
        _expect(lib, _epi(lib, **kw), want, text)
    _expect(lib, _epi(lib, M=0, A=None, D=None), OK)


def _epi_bwd(lib, dy=P, pre=P, act=3, dz=P, q=P, sf=P, dbias=None, M=4, N=256, ws=None, n=0):
    return lib.dg_epilogue_bwd(dy, pre, act, dz, q, sf, dbias, M, N, ws, n, NULL)


def test_epilogue_bwd(lib):
    for kw, want, text in [
        (dict(act=5), V, "activation"), (dict(N=24), S, "N"), (dict(N=0), S, "N"), (dict(M=-1), S, "M"), (dict(N=144), S, "128"),
        (dict(dy=None), V, "null"), (dict(pre=None), V, "null"), (dict(dz=None, q=None, sf=None), V, "null"), (dict(sf=None), V, "null"),
        (dict(q=None), V, "null"), (dict(dy=P + 8), A, "16"), (dict(pre=P + 8), A, "16"), (dict(dz=P + 8), A, "16"),
        (dict(q=P + 8), A, "16"), (dict(sf=P + 2), A, "4"), (dict(dbias=P + 2), A, "4"),
    ]:
        _expect(lib, _epi_bwd(lib, **kw), want, text)
    _expect(lib, _epi_bwd(lib, M=0, dy=None), OK)


def test_workspace_sizes(lib):
    size = dg.dg_get_workspace_size
    for K in (8, 2048, 4096, 16384):
        assert size(dg.DG_OP_RMS_NORM_BWD, 100, 0, K) >= 4096 + 4 * K
        # more rows never ask for less
        assert size(dg.DG_OP_RMS_NORM_BWD, 10**6, 0, K) >= size(dg.DG_OP_RMS_NORM_BWD, 1000, 0, K)
    assert size(dg.DG_OP_RMS_NORM_BWD, 100, 0, 12) == 0 and size(dg.DG_OP_RMS_NORM_BWD, -1, 0, 64) == 0
    assert size(dg.DG_OP_EPILOGUE_BWD, 1, 16, 0) == 4096 + 64
    assert size(dg.DG_OP_EPILOGUE_BWD, 4096, 4096, 0) >= 4096 + 4 * 4096
    assert size(dg.DG_OP_EPILOGUE_BWD, 4096, 24, 0) == 0
    assert dg.dg_describe_plan(dg.DG_OP_RMS_NORM_BWD, 4, 4, 128) == ""


def test_activation_names():
    assert [dg._act_arg(a) for a in ("none", "relu", "silu", "gelu", "gelu_tanh")] == [0, 1, 2, 3, 4] and dg._act_arg(dg.DG_ACT_GELU) == 3
    with pytest.raises(ValueError, match="gelu_tanh"):
        dg._act_arg("swish")


def _experts(lib, name, x=P, idx=P, w=P, w1=P, s1=P, w2=P, s2=P, y=P, T=4, k=2, first=0, G=8, H=256, I=128, ws=None, n=0):
    return getattr(lib, name)(x, idx, w, w1, s1, w2, s2, y, T, k, first, G, H, I, ws, n, NULL)


@pytest.mark.parametrize("name", ["dg_moe_experts_fp8", "dg_moe_experts_mxfp4"])
def test_experts(lib, name):
    for kw, want, text in [
        (dict(T=65), S, "T"), (dict(T=-1), S, "T"), (dict(k=0), S, "k"), (dict(k=17), S, "k"), (dict(G=0), S, "G"), (dict(G=1025), S, "G"),
        (dict(first=-1), S, "first_expert"), (dict(first=(1 << 31) - 4), S, "first_expert"), (dict(H=192), S, "H"), (dict(H=0), S, "H"),
        (dict(I=64), S, "I"), (dict(I=32896), S, "I"), (dict(x=None), V, "null"), (dict(idx=None), V, "null"), (dict(w=None), V, "null"),
        (dict(w1=None), V, "null"), (dict(s1=None), V, "null"), (dict(w2=None), V, "null"), (dict(s2=None), V, "null"), (dict(y=None), V, "null"),
        (dict(x=P + 8), A, "16"), (dict(w1=P + 4), A, "16"), (dict(w2=P + 8), A, "16"), (dict(y=P + 2), A, "16"), (dict(idx=P + 2), A, "4"),
        (dict(w=P + 1), A, "4"), (dict(s1=P + 2), A, "4"), (dict(s2=P + 2), A, "4"),
    ]:
        _expect(lib, _experts(lib, name, **kw), want, text)
    _expect(lib, _experts(lib, name, T=0, x=None, y=None), OK)


def test_experts_workspace(lib):
    size = dg.dg_get_workspace_size
    for H, inner in ((256, 128), (1024, 512), (7168, 2048), (32768, 128)):
        got = [size(dg.DG_OP_MOE_EXPERTS, n, H, inner) for n in (1, 2, 8, 64, 512, 1024)]
        assert got == sorted(got) and got[0] >= 4096 + 2 * inner and got[-1] >= 4096 + 2048 * inner
    for bad in ((1025, 256, 128), (-1, 256, 128), (8, 200, 128), (8, 256, 0)):
        assert size(dg.DG_OP_MOE_EXPERTS, *bad) == 0
