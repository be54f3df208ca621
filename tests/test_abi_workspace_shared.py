"""Workspace sizes of the operators leave room for the 4 KiB of counters that all of them keep at the buffer's start (no GPU needed)."""

import os

import pytest

from moe_grouped_matmul_amd import dg


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(dg.LIB_PATH):
        from moe_grouped_matmul_amd import build

        build.build()
    return dg.load_library()


@pytest.mark.parametrize("T,E", [(1, 8), (700, 256), (5000, 60), (1 << 20, 1024)])
def test_gate(T, E):
    blocks = min(256, -(-T // (64 if E <= 256 else 16)))
    assert dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, T, E, 2) >= 4096 + blocks * (2 * E + 1) * 4


@pytest.mark.parametrize("T,k,G", [(2049, 1, 1), (300, 8, 3), (5000, 8, 64), (16384, 8, 64), (16384, 8, 1024), (1 << 17, 2, 5)])
def test_row_order_of_16_bit_counts(T, k, G):
    n = T * k
    blocks = -(-n // (1024 * -(-n // (1024 * 128))))
    size = dg.dg_get_workspace_size(dg.DG_OP_MOE_LAYOUT, T, 0, k, G)
    assert size >= 4096 + 2 * blocks * G and size >= 4 * blocks * G


def test_row_order_of_32_bit_counts():
    for G in (1, 1024):
        assert dg.dg_get_workspace_size(dg.DG_OP_MOE_LAYOUT, (1 << 18) + 1, 0, 1, G) >= 4096 + 4 * 86 * G


@pytest.mark.parametrize("G", [1, 7, 64, 1024])
def test_a_buffer_for_many_choices_serves_fewer(lib, G):
    """Of the router and the row order, whose calls refuse a buffer that is too small; without a device a call that accepts its
    arguments stops at the device check."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present; the pointers are not real")
    P = 0x10000
    for T, k in ((40000, 8), (200000, 1), (25000, 8), (400000, 1), (1 << 20, 2), (2049, 1), (140000, 1)):
        size = dg.dg_get_workspace_size(dg.DG_OP_MOE_LAYOUT, T, 0, k, G)
        for n in (1, 2048, 2049, 100000, 131072, 131073, 262144, 262145, 393216, T * k - 1):
            if n <= T * k:
                assert dg.dg_get_workspace_size(dg.DG_OP_MOE_LAYOUT, n, 0, 1, G) <= size
                assert lib.dg_moe_layout_contiguous(P, P, P, P, P, n, 1, 0, G, 256, P, size, None) == dg.DG_ERR_DEVICE, (T, k, n)
        full = dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, T, G, 1)
        for t in (1, 64, 65, 16384, T - 1):
            if t <= T:
                assert lib.dg_moe_gate(P, 0, None, P, P, P, P, P, t, G, 1, 1, 1.0, 0.0, P, full, None) == dg.DG_ERR_DEVICE
