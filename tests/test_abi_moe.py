"""Host-side refusals of the mixture-of-experts operators and the microscaled
4-bit products (no GPU needed): every status code from arguments that fail
before any device work, sizes of the workspaces, plan texts, and what calls
with nothing to do return."""

import ctypes
import os

import pytest

from moe_grouped_matmul_amd import dg

P = 0x10000      # fake, never dereferenced
P4 = 0x10004
S, A, V, W, OK = dg.DG_ERR_SHAPE, dg.DG_ERR_ALIGN, dg.DG_ERR_INVALID_ARG, dg.DG_ERR_WORKSPACE, dg.DG_OK
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.LIB_PATH):
        from moe_grouped_matmul_amd import build

        build.build()
    return dg.load_library()


def _expect(lib, call, rc, text=""):
    assert call == rc
    msg = lib.dg_get_last_error().decode()
    assert (msg == "") == (rc == OK) and text in msg


def test_quantiser(lib):
    q, d = lib.dg_quant_mxfp4, lib.dg_dequant_mxfp4
    _expect(lib, q(P, 2, P, P, None, 1, 4, 4, 128, NULL), V, "dtype")
    _expect(lib, q(P, 0, P, P, None, 1, 4, 4, 100, NULL), S, "K")
    _expect(lib, q(P, 0, P, P, None, -1, 4, 4, 128, NULL), S)
    _expect(lib, q(P, 0, P, P, None, 65536, 4, 4, 128, NULL), S, "large")
    _expect(lib, q(P, 0, P, P, None, 1, 4, 1 << 31, 128, NULL), S)
    _expect(lib, q(P, 0, P, P, P, 1, 1 << 31, 4, 128, NULL), S)
    _expect(lib, q(None, 0, P, P, None, 1, 4, 4, 128, NULL), V)
    _expect(lib, q(P + 8, 0, P, P, None, 1, 4, 4, 128, NULL), A)
    _expect(lib, q(P, 0, P, P + 2, None, 1, 4, 4, 128, NULL), A)
    _expect(lib, q(P, 0, P, P, P + 1, 1, 4, 4, 128, NULL), A)
    _expect(lib, q(None, 0, None, None, None, 1, 4, 0, 128, NULL), OK)
    _expect(lib, d(P, P, P, 7, 1, 4, 128, NULL), V)
    _expect(lib, d(P, P, P4, 0, 1, 4, 128, NULL), A)
    _expect(lib, d(None, None, None, 0, 0, 4, 128, NULL), OK)


def test_products(lib):
    m = lib.dg_mxfp4_gemm_nt
    _expect(lib, m(P, P, P, P, P, 4, 16, 64, None, 0, NULL), S, "K")
    _expect(lib, m(P, P, P, P, P, 4, 24, 128, None, 0, NULL), S, "N")
    _expect(lib, m(P, P, P, P, P, 4, 16, 1 << 25, None, 0, NULL), S, "large")
    _expect(lib, m(P, P, P, P, P, -4, 16, 128, None, 0, NULL), S)
    _expect(lib, m(P, P, P, P, P, 1 << 31, 16, 128, None, 0, NULL), S)
    _expect(lib, m(P, P, P, P, P, 1 << 28, 16, 16384, None, 0, NULL), S, "scale")
    _expect(lib, m(P, None, P, P, P, 4, 16, 128, None, 0, NULL), V)
    _expect(lib, m(P4, P, P, P, P, 4, 16, 128, None, 0, NULL), A)
    _expect(lib, m(P, P + 2, P, P, P, 4, 16, 128, None, 0, NULL), A)
    _expect(lib, m(P, P, P, P, P, 4, 16, 128, P4, 64, NULL), W)
    _expect(lib, m(P, P, P, P, P, 4, 16, 128, P, 6, NULL), W)
    _expect(lib, m(None, None, None, None, None, 0, 16, 128, None, 0, NULL), OK)
    c, k = lib.dg_m_grouped_mxfp4_gemm_nt_contiguous, lib.dg_m_grouped_mxfp4_gemm_nt_masked
    _expect(lib, c(P, P, P, P, P, P, 128, 16, 128, 0, None, 0, NULL), S, "G")
    _expect(lib, c(P, P, P, P, P, P, 128, 16, 128, 1025, None, 0, NULL), S, "G")
    _expect(lib, c(P, P, P, P, P, None, 128, 16, 128, 2, None, 0, NULL), V, "m_indices")
    _expect(lib, c(P, P, P, P, P, P + 2, 128, 16, 128, 2, None, 0, NULL), A)
    _expect(lib, k(P, P, P, P, P, None, 2, 8, 16, 128, 0, None, 0, NULL), V, "masked_m")
    _expect(lib, k(P, P, P, P, P, P, 1025, 8, 16, 128, 0, None, 0, NULL), S)
    _expect(lib, k(None, None, None, None, None, None, 2, 0, 16, 128, 0, None, 0, NULL), OK)


def test_gate(lib):
    def g(logits=P, dtype=0, valid=None, idx=P, w=P, counts=P, load=P, loss=P, T=4, E=8, k=2, scale=1.0, ws=P, n=1 << 20):
        return lib.dg_moe_gate(logits, dtype, valid, idx, w, counts, load, loss, T, E, k, 1, scale, 0.0, ws, n, NULL)

    _expect(lib, g(dtype=5), V, "dtype")
    for kw in (dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025), dict(k=0), dict(k=17, E=32), dict(k=9)):
        _expect(lib, g(**kw), S)
    for s in (0.0, float("inf"), float("nan")):
        _expect(lib, g(scale=s), V, "w_scale")
    for n in ("logits", "idx", "w", "counts", "load", "loss"):
        _expect(lib, g(**{n: None}), V)
    _expect(lib, g(logits=P4), A)
    _expect(lib, g(idx=P + 2), A)
    _expect(lib, g(ws=None), W, "bytes")
    _expect(lib, g(n=16), W)
    _expect(lib, g(ws=P4), W)

    def b(logits=P, dtype=0, idx=P, w=P, counts=P, dw=P, dloss=P, dl=P, T=4, E=8, k=2):
        return lib.dg_moe_gate_bwd(logits, dtype, idx, w, counts, dw, dloss, dl, T, E, k, 1, 1.0, 0.0, NULL)

    _expect(lib, b(E=2000), S)
    _expect(lib, b(dl=None), V)
    _expect(lib, b(dl=P4), A)
    _expect(lib, b(dw=P + 1), A)
    _expect(lib, b(logits=None, idx=None, w=None, counts=None, dl=None, T=0), OK)


def test_layout_and_combine(lib):
    def c(idx=P, counts=P, m=P, rt=P, ro=P, T=4, k=2, first=0, G=2, M=256, ws=P, n=1 << 16):
        return lib.dg_moe_layout_contiguous(idx, counts, m, rt, ro, T, k, first, G, M, ws, n, NULL)

    for kw in (dict(T=-1), dict(k=0), dict(k=17), dict(G=0), dict(G=1025), dict(first=-1), dict(M=-1), dict(M=1 << 31), dict(T=1 << 28, k=8),
               dict(first=(1 << 31) - 2, G=2)):
        _expect(lib, c(**kw), S)
    for n in ("idx", "counts", "m", "rt", "ro"):
        _expect(lib, c(**{n: None}), V)
        _expect(lib, c(**{n: P + 2}), A)
    _expect(lib, c(ws=None), W)
    _expect(lib, c(n=4), W)
    m = lib.dg_moe_layout_masked
    _expect(lib, m(P, P, P, P, 4, 2, 0, 2, 0, P, 1 << 16, NULL), S)
    _expect(lib, m(P, P, P, P, 4, 2, 0, 1024, 1 << 22, P, 1 << 16, NULL), S)
    f, b = lib.dg_moe_combine, lib.dg_moe_combine_bwd
    _expect(lib, f(P, P, P, P, 3, 4, 2, 16, 9, NULL), V, "dtype")
    _expect(lib, f(P, P, P, P, 1, 4, 2, 24, 9, NULL), S, "N")
    _expect(lib, f(P, P, P, P, 1, 4, 17, 16, 9, NULL), S)
    _expect(lib, f(P, P, P, P, 1, 4, 2, 16, -1, NULL), S)
    _expect(lib, f(None, P, P, P, 1, 4, 2, 16, 9, NULL), V)
    _expect(lib, f(P4, P, P, P, 1, 4, 2, 16, 9, NULL), A)
    _expect(lib, f(None, None, None, None, 1, 0, 2, 16, 9, NULL), OK)
    _expect(lib, b(P, 1, P, P, P, None, P, 4, 2, 16, 9, NULL), V)
    _expect(lib, b(P, 1, P, P, P, P4, P, 4, 2, 16, 9, NULL), A)
    _expect(lib, b(None, 1, None, None, None, None, None, 0, 2, 16, 9, NULL), OK)


def test_argument_check(lib):
    """The native check of the binding's tensors: a host tensor is none of its, wrong arguments are errors."""
    import torch

    from moe_grouped_matmul_amd import _args

    t = torch.zeros(3, 4)
    assert dg._pointer is _args.pointer
    assert _args.pointer(t, torch.float32, (3, 4), 0) is None
    for bad in ((t, 1, (3, 4), 0), (1, torch.float32, (3, 4), 0), (t, torch.float32, [3, 4], 0), (t, torch.float32, (3, 4), "x"), (t,)):
        with pytest.raises(TypeError):
            _args.pointer(*bad)


def test_no_device(lib):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this checks the no-device path only")
    assert lib.dg_mxfp4_gemm_nt(P, P, P, P, P, 4, 16, 128, None, 0, NULL) == dg.DG_ERR_DEVICE
    assert lib.dg_moe_combine(P, P, P, P, 1, 4, 2, 16, 9, NULL) == dg.DG_ERR_DEVICE


def test_workspaces_and_plans(lib):
    try:
        dg.dg_set_num_cus(256)
        size, plan = dg.dg_get_workspace_size, dg.dg_describe_plan
        op = dg.DG_OP_MXFP4_GEMM_NT
        assert "tile=64x64 tiles=33 splits=4" in plan(op, 64, 2112, 7168)
        assert size(op, 64, 2112, 7168) == 4096 + 4 * 33 * 64 * 64 * 4
        assert "tile=64x64 tiles=112 splits=1" in plan(op, 64, 7168, 2048) and size(op, 64, 7168, 2048) == 0
        assert "tile=128x256" in plan(op, 1829, 3952, 640)
        assert "tile=256x256 tiles=256" in plan(op, 4096, 4096, 7168) and size(op, 4096, 4096, 7168) == 0
        assert plan(op, 64, 2110, 7168) == "" and plan(op, 64, 2112, 100) == "" and size(op, 0, 16, 128) == 0
        assert size(dg.DG_OP_MOE_GATE, 1, 8, 2) > 0 and size(dg.DG_OP_MOE_GATE, 1, 2000, 2) == 0
        assert size(dg.DG_OP_MOE_GATE, 1 << 20, 256, 8) == size(dg.DG_OP_MOE_GATE, 1 << 21, 256, 8)
        assert size(dg.DG_OP_MOE_LAYOUT, 16384, 0, 8, 64) == 128 * 64 * 4 and size(dg.DG_OP_MOE_LAYOUT, 4, 0, 17, 64) == 0
    finally:
        dg.dg_set_num_cus(0)
