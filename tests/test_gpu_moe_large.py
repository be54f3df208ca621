"""Arrays whose offsets pass 32 bits: more than 2^32 elements in one operand of
each operator, with the rows that are checked at both ends and around the
places where a 32-bit index or byte offset would wrap."""

import gc

import numpy as np
import pytest
import torch

from moe_grouped_matmul_amd import dg
from oracle import moe, mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _free():
    yield
    gc.collect()
    torch.cuda.empty_cache()


def _rand(shape, seed, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


def _ends(rows, row_bytes):
    """Rows at the ends and around the 2^31 and 2^32 byte and element offsets."""
    at = {0, 1, rows - 2, rows - 1}
    for b in (2 ** 31, 2 ** 32, 2 ** 33):
        at |= {r for r in (b // row_bytes - 1, b // row_bytes, b // row_bytes + 1) if 0 <= r < rows}
    return sorted(at)


def _sample(x, at):
    return x[torch.tensor(at, device=DEV)].float().cpu().numpy()


def test_quantiser():
    N, R = 16384, 540672  # 8.9e9 elements: 17.7 GB in, 4.4 GB of codes
    at = _ends(R, 2 * N) + _ends(R, N // 2)
    x = _rand((R, N), 0)
    q = torch.zeros(R, N // 2, dtype=torch.uint8, device=DEV)
    s = torch.zeros(N // 128, R, dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(x, q, s)
    want, words = mxfp4.quant_mxfp4(_sample(x, at))
    sel = torch.tensor(at, device=DEV)
    assert np.array_equal(q[sel].cpu().numpy(), want) and np.array_equal(s[:, sel].cpu().numpy(), words)
    rt = torch.tensor(at, dtype=torch.int32, device=DEV)
    q2 = torch.zeros(len(at), N // 2, dtype=torch.uint8, device=DEV)
    s2 = torch.zeros(N // 128, len(at), dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(x, q2, s2, row_token=rt)
    assert np.array_equal(q2.cpu().numpy(), want) and np.array_equal(s2.cpu().numpy(), words)
    x.zero_()
    dg.dg_dequant_mxfp4(q, s, x)
    assert np.array_equal(_sample(x, at).astype(np.float64), mxfp4.values_mxfp4(want, words))


@pytest.mark.parametrize("form", ["dense", "contiguous", "masked"])
def test_products(form):
    N, K, G = 16384, 128, 8
    R = 294912  # x N: 4.8e9 elements of D, 9.7 GB
    a, b = _rand((R, K), 1), _rand((G, N, K), 2)
    qa, sa = torch.zeros(R, K // 2, dtype=torch.uint8, device=DEV), torch.zeros(1, R, dtype=torch.int32, device=DEV)
    qb, sb = torch.zeros(G, N, K // 2, dtype=torch.uint8, device=DEV), torch.zeros(G, 1, N, dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(a, qa, sa)
    dg.dg_quant_mxfp4(b, qb, sb)
    d = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
    at = _ends(R, 2 * N) + _ends(R, N)
    m = R // G
    if form == "dense":
        dg.dg_mxfp4_gemm_nt(qa, sa, qb[0], sb[0], d)
        of = [0] * len(at)
    elif form == "contiguous":
        idx = torch.arange(R, device=DEV, dtype=torch.int32) // m
        dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(qa, sa, qb, sb, d, idx)
        of = [r // m for r in at]
    else:
        mm = torch.tensor([m if g % 2 else m - 1 for g in range(G)], dtype=torch.int32, device=DEV)
        sg = sa.reshape(G, 1, m)  # one word of K per row: group-major as it is
        dg.dg_m_grouped_mxfp4_gemm_nt_masked(qa.reshape(G, m, K // 2), sg, qb, sb, d.reshape(G, m, N), mm)
        of = [r // m if r % m < int(mm[r // m]) else -1 for r in at]
    got = _sample(d, at).astype(np.float64)
    ha, hsa = mxfp4.quant_mxfp4(_sample(a, at))
    for i, g in enumerate(of):
        if g < 0:
            assert not got[i].any()
            continue
        ref, mag = mxfp4.gemm_mxfp4(ha[i:i + 1], hsa[:, i:i + 1], qb[g].cpu().numpy(), sb[g].cpu().numpy())
        assert np.all(np.abs(got[i] - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -10 + (K / 32 + 2) * U) * mag[0])


def test_combine():
    N, R, k = 16384, 294912, 2
    rows = _rand((R, N), 3)
    at = (_ends(R, 2 * N) + _ends(R, N))[:18]
    T = len(at)
    ro = np.stack([np.array(at), np.array(at[::-1])], 1).astype(np.int32)
    keep = np.unique(ro[:, 0], return_index=True)[1]  # each row one owner in the gradient
    w = np.linspace(0.1, 0.9, T * k).reshape(T, k).astype(np.float32)
    y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    dg.dg_moe_combine(rows, torch.from_numpy(ro).to(DEV), torch.from_numpy(w).to(DEV), y)
    small = _sample(rows, at).astype(np.float64)
    local = np.stack([np.arange(T), np.arange(T)[::-1]], 1)
    want, mag = moe.combine(small, local, w)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + (k + 1) * U * mag)
    ro1, w1 = ro[keep, :1].copy(), w[keep, :1].copy()
    dy = _rand((len(keep), N), 4)
    drows = torch.zeros_like(rows)
    dw = torch.empty(len(keep), 1, device=DEV)
    dg.dg_moe_combine_bwd(dy, rows, torch.from_numpy(ro1).to(DEV), torch.from_numpy(w1).to(DEV), drows, dw)
    g, dwant, dmag = moe.combine_grad(dy.double().cpu().numpy(), small[keep], np.arange(len(keep))[:, None], w1)
    got = _sample(drows, ro1[:, 0].tolist()).astype(np.float64)
    assert np.all(np.abs(got - g) <= (2.0 ** -8 * 1.01 + U) * np.abs(g))
    assert np.all(np.abs(dw.double().cpu().numpy() - dwant) <= (N / 256 + 20) * U * dmag)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine_of_rows_past_the_cache(dtype):
    """Rows that are streamed; more choices than are in flight at once, tokens without rows, a last partial run of columns."""
    T, k, N = 1100, 9, 7184
    R = T * k
    rng = np.random.default_rng(8)
    ro = rng.permutation(R).reshape(T, k).astype(np.int32)
    ro[rng.random((T, k)) < 0.05] = -1
    ro[5], ro[T - 1, 0], ro[7, 8] = -1, R, R + 9
    w = rng.standard_normal((T, k)).astype(np.float32)
    rows, dy = _rand((R, N), 9), _rand((T, N), 10, dtype)
    y, drows, dw = torch.full((T, N), 7.0, dtype=dtype, device=DEV), torch.full_like(rows, 7.0), torch.full((T, k), 7.0, device=DEV)
    dro, dwt = torch.from_numpy(ro).to(DEV), torch.from_numpy(w).to(DEV)
    dg.dg_moe_combine(rows, dro, dwt, y)
    dg.dg_moe_combine_bwd(dy, rows, dro, dwt, drows, dw)
    h = rows.float().cpu().numpy()
    want, mag = moe.combine(h, ro, w.astype(np.float64))
    out = 2.0 ** -8 if dtype is torch.bfloat16 else 0.0
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= out * 1.01 * np.abs(want) + (k + 1) * U * mag)
    g, dwant, dmag = moe.combine_grad(dy.double().cpu().numpy(), h, ro, w.astype(np.float64))
    got = drows.float().cpu().numpy()
    free = np.isnan(g[:, 0])
    assert free.any() and np.all(got[free] == 7)
    assert np.all(np.abs(got[~free] - g[~free]) <= (2.0 ** -8 * 1.01 + U) * np.abs(g[~free]))
    assert np.all(np.abs(dw.double().cpu().numpy() - dwant) <= (N / 256 + 20) * U * dmag)


def test_combine_of_many_tokens():
    """More workgroups than one launch takes."""
    N, R = 16, 40
    rows = _rand((R, N), 6)
    h = rows.double().cpu().numpy()
    for T, k in (((1 << 23) + 7, 1), ((1 << 20) + 9, 8)):
        at = [0, 1, (1 << 20) - 1, 1 << 20, T - 1]
        ro = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
        ro[torch.tensor(at, device=DEV)] = torch.arange(len(at) * k, dtype=torch.int32, device=DEV).reshape(-1, k)
        w = torch.full((T, k), 0.75, device=DEV)
        y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV)
        dg.dg_moe_combine(rows, ro, w, y)
        idx, c = np.arange(len(at) * k).reshape(-1, k), np.full((len(at), k), 0.75, np.float32)
        want, mag = moe.combine(h, idx, c)
        assert np.all(np.abs(_sample(y, at) - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + (k + 1) * U * mag)
        assert int((y != 0).any(1).sum()) == len(at)
        drows, dw = torch.full_like(rows, 7.0), torch.full((T, k), 7.0, device=DEV)
        dg.dg_moe_combine_bwd(y, rows, ro, w, drows, dw)
        g, dwant, dmag = moe.combine_grad(_sample(y, at).astype(np.float64), h, idx, c)
        used = len(at) * k
        assert np.all(np.abs(drows[:used].double().cpu().numpy() - g[:used]) <= (2.0 ** -8 * 1.01 + U) * np.abs(g[:used]))
        assert bool((drows[used:] == 7).all())
        assert np.all(np.abs(_sample(dw, at) - dwant) <= (N / 256 + 20) * U * dmag)
        dw[torch.tensor(at, device=DEV)] = 0
        assert not bool(dw.any())


def test_gate():
    T, E, k = (1 << 22) + 5, 1024, 2  # 4.3e9 logits in bf16
    x = _rand((T, E), 5)
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    counts, load, loss = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV), torch.empty(1, device=DEV)
    ws = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, T, E, k), dtype=torch.uint8, device=DEV)
    dg.dg_moe_gate(x, idx, w, counts, load, loss, loss_coef=0.1, workspace=ws)
    at = _ends(T, 2 * E) + _ends(T, E)
    h = _sample(x, at).astype(np.float64)
    want = moe.gate(h, k)
    sel = torch.tensor(at, device=DEV)
    assert np.array_equal(idx[sel].cpu().numpy(), want["topk_idx"])
    spread = (h.max(1) - h.min(1)).max()
    assert np.all(np.abs(w[sel].double().cpu().numpy() - want["topk_w"]) <= (4 * spread + 100) * U * want["topk_w"])
    assert int(counts[E]) == T and int(counts[:E].sum()) == T * k
    assert np.array_equal(counts[:E].cpu().numpy(), torch.bincount(idx.reshape(-1), minlength=E).cpu().numpy())
    dw = torch.ones_like(w)
    dl = torch.empty_like(x)
    dg.dg_moe_gate_bwd(x, idx, w, counts, dw, torch.ones(1, device=DEV), dl, loss_coef=0.1)
    c = counts[:E].double().cpu().numpy()
    p, g = want["p"], 0.1 * E * c / (k * float(T) ** 2)  # equal gradients of renormalised weights cancel: the loss's share is left
    ref = p * (g - (p * g).sum(1, keepdims=True))
    mag = p * (g + (p * g).sum(1, keepdims=True) + 1)
    for i, t in enumerate(want["topk_idx"]):
        mag[i, t] += 2 * want["topk_w"][i]
    got = _sample(dl, at).astype(np.float64)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * 1.01 * np.abs(ref) + (4 * spread + 100) * U * mag + 1e-37)
