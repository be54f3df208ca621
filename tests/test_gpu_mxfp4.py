"""Microscaled 4-bit floats on the GPU: the quantiser bit-exact against the
64-bit oracle (extremes, midpoints, NaN blocks, gathered rows), the values
back, and the dense, contiguous and masked products on every tile shape: bit
for bit where fp32 sums are exact, within a derived bound elsewhere.

Bound of a product: one rounding to bf16 (8 significant bits: 2^-8 of the result); the matrix core's
sum of a block's terms keeps at least 13 bits below the largest term of a group
of 8 (2^-10 of the sum S of the magnitudes); one fp32 rounding of a partial sum
per 32 terms (2^-24 of S each)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_matmul_amd import dg
from oracle import mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _source(rng, shape):
    """Normal values over many magnitudes, zero blocks, signed zeros, midpoints of the grid."""
    x = rng.standard_normal(shape).astype(np.float32)
    x *= np.float32(2.0) ** rng.integers(-20, 20, shape[:-1] + (1,)).astype(np.float32)
    flat = x.reshape(-1, 32)
    flat[::7] = 0.0
    flat[1::7, :8] = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], np.float32)
    flat[1::7, 8:] = np.clip(flat[1::7, 8:], -6, 6)
    flat[2::7, 3] = -0.0
    return x


def _run_quant(x, bf16=False, row_token=None):
    X = _t(x).to(torch.bfloat16) if bf16 else _t(x)
    lead = x.shape[:-1] if row_token is None else row_token.shape
    K = x.shape[-1]
    q = torch.full(lead + (K // 2,), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full(lead[:-1] + (K // 128, lead[-1]), 0x5A5A5A5A, dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(X, q, s, row_token=None if row_token is None else _t(row_token))
    return X, q, s


QUANT = [((1, 128), False), ((17, 256), True), ((33, 384), False), ((3, 5, 640), True), ((2, 130, 128), False)]


@pytest.mark.parametrize("shape,bf16", QUANT)
def test_quantiser_bit_exact(shape, bf16):
    x = _source(np.random.default_rng(sum(shape)), shape)
    X, q, s = _run_quant(x, bf16)
    rq, rs = mxfp4.quant_mxfp4(X.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    want = mxfp4.values_mxfp4(rq, rs)
    for dt in (torch.bfloat16, torch.float32):
        y = torch.empty(shape, dtype=dt, device=DEV)
        dg.dg_dequant_mxfp4(q, s, y)
        assert np.array_equal(y.double().cpu().numpy(), want)


def _fp32(v):
    """The values as fp32 holds them: 4 * 2^126, the code of the largest fp32 numbers, is past its range."""
    with np.errstate(over="ignore"):
        return v.astype(np.float32).astype(np.float64)


def test_quantiser_extremes():
    f = np.finfo(np.float32)
    x = np.zeros((4, 256), np.float32)
    x[0, 0::32] = [f.max, f.tiny, 1e-45, 3.0, np.nan, np.inf, -np.inf, 6.000001]
    x[1] = np.float32(f.max)
    x[2] = np.float32(1e-45) * np.arange(256, dtype=np.float32)
    x[3] = np.float32(2.0 ** -127) * np.linspace(-8, 8, 256, dtype=np.float32)
    _, q, s = _run_quant(x)
    rq, rs = mxfp4.quant_mxfp4(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
    y = torch.empty(4, 256, device=DEV)
    dg.dg_dequant_mxfp4(q, s, y)
    assert np.array_equal(y.double().cpu().numpy(), _fp32(mxfp4.values_mxfp4(rq, rs)), equal_nan=True)
    yb = torch.empty(4, 256, dtype=torch.bfloat16, device=DEV)
    dg.dg_dequant_mxfp4(q, s, yb)
    assert np.array_equal(yb.double().cpu().numpy(), _fp32(mxfp4.values_mxfp4(rq, rs)), equal_nan=True)


@pytest.mark.parametrize("shape", [(40,), (3, 21)])
def test_quantiser_gathers_rows(shape):
    rng = np.random.default_rng(5)
    x = _source(rng, (9, 384))
    rows = rng.integers(-3, 12, shape).astype(np.int32)  # -1, -3 and 9..11 are outside
    _, q, s = _run_quant(x, True, rows)
    src = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    rq, rs = mxfp4.quant_mxfp4(src[np.clip(rows, 0, 8)])
    ok = (rows >= 0) & (rows < 9)
    want_q = np.where(ok[..., None], rq, 0xA5)
    want_s = np.where(ok[..., None, :], rs, 0x5A5A5A5A)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)


def _operand(rng, lead, rows, K, exact):
    """Random codes and scales: all scales 1 where sums have to be exact, else over +-6 octaves."""
    codes = rng.integers(0, 256, lead + (rows, K // 2)).astype(np.uint8)
    c = np.full(lead + (rows, K // 32), 127) if exact else 127 + rng.integers(-6, 7, lead + (rows, K // 32))
    return codes, mxfp4.pack_words(c)


def _check(got, ref, mag, K, exact, what):
    """got: bf16 bits; ref and mag from the oracle."""
    if exact:
        want = oracle.bf16_rne_bits(ref.astype(np.float32))
        v, w = oracle.bf16_bits_to_f64(got), oracle.bf16_bits_to_f64(want)
        assert np.array_equal(v, w), what
        return
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + (K / 32 + 2) * 2.0 ** -24) * mag
    err = np.abs(oracle.bf16_bits_to_f64(got) - ref)
    assert np.all(err <= tol), (what, float((err / tol).max()))
    assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(ref), what


# rows cover one token, partial tiles and every tile shape; K an odd and an even number of 128s; N partial tiles
DENSE = [(1, 16, 128), (1, 272, 1152), (3, 400, 256), (64, 2112, 896), (65, 144, 640), (130, 528, 1024), (200, 4112, 384),
         (300, 6160, 256), (700, 16384, 384), (2050, 4096, 640), (4096, 2048, 128)]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K, exact):
    rng = np.random.default_rng(M + N + K)
    a, sa = _operand(rng, (), M, K, exact)
    b, sb = _operand(rng, (), N, K, exact)
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    n = dg.dg_get_workspace_size(dg.DG_OP_MXFP4_GEMM_NT, M, N, K)
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device=DEV)
    A, SA, B, SB = map(_t, (a, sa, b, sb))
    ref, mag = mxfp4.gemm_mxfp4(a, sa, b, sb)
    for w in (ws, ws, None):  # the workspace is left reusable; none at all works too
        D.fill_(float("nan"))
        dg.dg_mxfp4_gemm_nt(A, SA, B, SB, D, workspace=w)
        _check(_bits(D), ref, mag, K, exact, (M, N, K, w is None))


TILES = ["64x64", "128x256", "256x256"]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (130, 272, 896), (600, 784, 1152), (257, 1040, 256), (1030, 2064, 2304)])
def test_dense_tile_shapes(monkeypatch, tile, M, N, K):
    """Every tile shape at sizes its rule would not give it: partial tiles, K an odd number of 128s, several tiles a workgroup."""
    monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
    rng = np.random.default_rng(M + N + K)
    for exact in (True, False):
        a, sa = _operand(rng, (), M, K, exact)
        b, sb = _operand(rng, (), N, K, exact)
        ref, mag = mxfp4.gemm_mxfp4(a, sa, b, sb)
        for cus in (0, 3, 7, 20, 45):  # few: a persistent workgroup walks many tiles, a partial last round is cut or spread
            dg.dg_set_num_cus(cus)
            try:
                D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
                ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
                dg.dg_mxfp4_gemm_nt(*map(_t, (a, sa, b, sb)), D, workspace=ws)
            finally:
                dg.dg_set_num_cus(0)
            _check(_bits(D), ref, mag, K, exact, (tile, M, N, K, cus))


def test_dense_long_k_and_shared_workspace_bit_identical():
    M, N, K = 17, 320, 16384
    rng = np.random.default_rng(0)
    a, sa = _operand(rng, (), M, K, False)
    b, sb = _operand(rng, (), N, K, False)
    A, SA, B, SB = map(_t, (a, sa, b, sb))
    ws = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MXFP4_GEMM_NT, M, N, K), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    outs = []
    for _ in range(3):
        D = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        dg.dg_mxfp4_gemm_nt(A, SA, B, SB, D, workspace=ws)
        outs.append(_bits(D))
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])
    ref, mag = mxfp4.gemm_mxfp4(a, sa, b, sb)
    _check(outs[0], ref, mag, K, False, "long K")


def test_nan_and_extreme_scales():
    M, N, K = 20, 48, 384
    rng = np.random.default_rng(9)
    a, _ = _operand(rng, (), M, K, True)
    b, _ = _operand(rng, (), N, K, True)
    ca, cb = np.full((M, K // 32), 127), np.full((N, K // 32), 127)
    ca[3, 5] = 255
    cb[7, 11] = 255
    ca[4] = 0      # 2^-127 on every block ...
    cb[9] = 250    # ... against large weights
    sa, sb = mxfp4.pack_words(ca), mxfp4.pack_words(cb)
    D = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    dg.dg_mxfp4_gemm_nt(_t(a), _t(sa), _t(b), _t(sb), D)
    got = oracle.bf16_bits_to_f64(_bits(D))
    ref, mag = mxfp4.gemm_mxfp4(a, sa, b, sb)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref) & (mag < 2.0 ** 127)  # column 9 elsewhere: a partial sum may pass fp32's range
    ok[4] = False
    assert np.array_equal(got[ok], oracle.bf16_bits_to_f64(oracle.bf16_rne_bits(ref.astype(np.float32)))[ok])
    # row 4: products of 2^-127 scales; those that fp32 holds as normal numbers are exact
    r = ref[4]
    big = ~np.isnan(r) & (np.abs(r) > 2.0 ** -100)
    assert np.array_equal(got[4][big], oracle.bf16_bits_to_f64(oracle.bf16_rne_bits(r.astype(np.float32)))[big])


CONTIG = [([5, 130, 1], 144, 256, 0), ([128, 256, 1, 300], 272, 640, 3), ([0, 0, 700, 0, 33], 528, 1152, 1), ([1], 16, 128, 0),
          ([1500, 2, 900, 1100], 4096, 384, 2)]


@pytest.mark.parametrize("tile", [None, "64x64", "128x256", "256x256"])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("counts,N,K,tail", CONTIG)
def test_contiguous(monkeypatch, counts, N, K, tail, exact, tile):
    """Segments padded to 128 rows, `tail` further padding blocks; padding rows are left untouched whatever they hold."""
    if tile:
        monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
    rng = np.random.default_rng(N + K)
    G = len(counts)
    idx = np.concatenate([np.concatenate((np.full(c, g), np.full(-c % 128, -1))) for g, c in enumerate(counts)] +
                         [np.full(128 * tail, -1)]).astype(np.int32)
    idx[idx < 0] = np.where(np.arange((idx < 0).sum()) % 2, -1, G + 3)  # any index outside [0, G) is padding
    M = len(idx)
    a, sa = _operand(rng, (), M, K, exact)
    b, sb = _operand(rng, (G,), N, K, exact)
    sa = sa.copy()
    sa[:, (idx < 0) | (idx >= G)] = -1  # NaN scales on padding rows
    A, SA, B, SB, I = map(_t, (a, sa, b, sb, idx))
    pad = (idx < 0) | (idx >= G)
    want = [mxfp4.gemm_mxfp4(a[idx == g], sa[:, idx == g], b[g], sb[g]) if (idx == g).any() else None for g in range(G)]
    for cus in (0, 2, 5, 9, 23, 60):
        dg.dg_set_num_cus(cus)
        try:
            D = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
            dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(A, SA, B, SB, D, I)
        finally:
            dg.dg_set_num_cus(0)
        got = _bits(D)
        for g in range(G):
            if want[g]:
                _check(got[idx == g], *want[g], K, exact, (g, counts[g], cus))
        assert np.all(got[pad] == oracle.bf16_rne_bits(np.float32(7.0)))


def test_contiguous_many_experts_and_long_layout(monkeypatch):
    """64 experts of 0-3 blocks each, rows tagged anywhere in their block; and a layout longer than one launch holds."""
    rng = np.random.default_rng(64)
    G, N, K = 64, 256, 256
    idx = np.full(128 * 2100, -1, np.int32)
    at = 0
    for g in rng.permutation(G):
        for _ in range(rng.integers(0, 4)):
            rows = rng.choice(128, rng.integers(1, 129), replace=False)
            idx[128 * at + rows] = g
            at += int(rng.integers(1, 3))  # blocks without a row in between
    idx[-128 * 3:] = 5   # past the first 2048 blocks
    idx[-1] = -1
    a, sa = _operand(rng, (), len(idx), K, True)
    b, sb = _operand(rng, (G,), N, K, True)
    for tile in TILES:
        monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
        D = torch.full((len(idx), N), 7.0, dtype=torch.bfloat16, device=DEV)
        dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(*map(_t, (a, sa, b, sb)), D, _t(idx))
        got = _bits(D)
        for g in range(G):
            r = idx == g
            if r.any():
                _check(got[r], *mxfp4.gemm_mxfp4(a[r], sa[:, r], b[g], sb[g]), K, True, (tile, g))
        assert np.all(got[idx < 0] == oracle.bf16_rne_bits(np.float32(7.0)))


@pytest.mark.parametrize("tile", TILES)
def test_contiguous_block_of_two_experts(monkeypatch, tile):
    """Past the layout's rule: rows of the block's one expert are right, others unwritten; refused when the check is on."""
    rng = np.random.default_rng(3)
    M, N, K, G = 300, 272, 384, 3
    idx = np.repeat([0, 1, 2], [70, 130, 100]).astype(np.int32)
    a, sa = _operand(rng, (), M, K, True)
    b, sb = _operand(rng, (G,), N, K, True)
    monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
    D = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    args = [*map(_t, (a, sa, b, sb)), D, _t(idx)]
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(*args)
    got = _bits(D)
    for r0 in range(0, M, 128):
        at = np.arange(r0, min(M, r0 + 128))
        wrote = {int(e) for e in set(idx[at]) if not np.all(got[at[idx[at] == e]] == oracle.bf16_rne_bits(np.float32(7.0)))}
        assert len(wrote) == 1, (tile, r0, wrote)
        e = wrote.pop()
        r = at[idx[at] == e]
        _check(got[r], *mxfp4.gemm_mxfp4(a[r], sa[:, r], b[e], sb[e]), K, True, (tile, r0))
        assert np.all(got[at[idx[at] != e]] == oracle.bf16_rne_bits(np.float32(7.0)))
    monkeypatch.setenv("DG_CHECK_LAYOUT", "1")
    with pytest.raises(dg.DGError, match="DG_CHECK_LAYOUT"):
        dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(*args)
    D.fill_(7.0)
    idx[:] = np.arange(M) // 128
    args[-1] = _t(idx)
    dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(*args)
    _check(_bits(D)[:128], *mxfp4.gemm_mxfp4(a[:128], sa[:, :128], b[0], sb[0]), K, True, tile)


MASKED = [(3, 16, [16, 0, 5], 144, 256), (4, 70, [70, 1, 64, 33], 272, 896), (2, 300, [300, 129], 528, 384), (5, 1, [1, 0, 1, 1, 0], 16, 128),
          (2, 40, [-3, 99], 400, 1152), (2, 600, [530, 257], 272, 640)]


@pytest.mark.parametrize("tile", [None, "64x64", "128x256"])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("G,max_m,m,N,K", MASKED)
def test_masked(monkeypatch, G, max_m, m, N, K, exact, tile):
    if tile:
        monkeypatch.setenv("DG_FORCE_CONFIG", f"mxfp4={tile}")
    rng = np.random.default_rng(N + K + G)
    a, sa = _operand(rng, (G,), max_m, K, exact)
    b, sb = _operand(rng, (G,), N, K, exact)
    D = torch.full((G, max_m, N), 7.0, dtype=torch.bfloat16, device=DEV)
    dg.dg_m_grouped_mxfp4_gemm_nt_masked(*map(_t, (a, sa, b, sb)), D, _t(np.array(m, np.int32)))
    got = _bits(D)
    for g in range(G):
        n = min(max(m[g], 0), max_m)
        if n:
            ref, mag = mxfp4.gemm_mxfp4(a[g, :n], sa[g][:, :n], b[g], sb[g])
            _check(got[g, :n], ref, mag, K, exact, (g, n))
        assert np.all(got[g, n:] == oracle.bf16_rne_bits(np.float32(7.0)))


def test_side_stream_and_graph_replay():
    """On a stream of their own, and captured: replays follow masked_m changed on the device."""
    G, max_m, N, K = 3, 32, 272, 512
    rng = np.random.default_rng(2)
    a, sa = _operand(rng, (G,), max_m, K, True)
    b, sb = _operand(rng, (G,), N, K, True)
    A, SA, B, SB = map(_t, (a, sa, b, sb))
    D = torch.zeros(G, max_m, N, dtype=torch.bfloat16, device=DEV)
    mm = torch.zeros(G, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        dg.dg_m_grouped_mxfp4_gemm_nt_masked(A, SA, B, SB, D, mm)
    s.synchronize()
    with torch.cuda.graph(graph, stream=s):
        dg.dg_m_grouped_mxfp4_gemm_nt_masked(A, SA, B, SB, D, mm)
    for m in ([3, 0, 32], [32, 32, 1], [0, 0, 0], [1, 2, 3]):
        mm.copy_(torch.tensor(m, dtype=torch.int32))
        D.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = _bits(D)
        for g in range(G):
            if m[g]:
                ref, mag = mxfp4.gemm_mxfp4(a[g, :m[g]], sa[g][:, :m[g]], b[g], sb[g])
                _check(got[g, :m[g]], ref, mag, K, True, m)
            assert np.all(got[g, m[g]:] == oracle.bf16_rne_bits(np.float32(7.0)))


def test_empty_calls_and_refusals():
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
    i32, bf = torch.int32, torch.bfloat16
    dg.dg_mxfp4_gemm_nt(z(0, 64), z(1, 0, dt=i32), z(16, 64), z(1, 16, dt=i32), z(0, 16, dt=bf))
    dg.dg_quant_mxfp4(z(0, 128, dt=torch.float32), z(0, 64), z(1, 0, dt=i32))
    good = (z(4, 64), z(1, 4, dt=i32), z(16, 64), z(1, 16, dt=i32), z(4, 16, dt=bf))
    for k, bad in ((0, z(4, 128)[:, :64]), (0, z(4, 128)), (1, z(4, 1, dt=i32)), (3, z(1, 17, dt=i32)), (4, z(4, 32, dt=bf)[:, ::2])):
        args = list(good)
        args[k] = bad
        with pytest.raises(ValueError):
            dg.dg_mxfp4_gemm_nt(*args)
    with pytest.raises(TypeError):
        dg.dg_mxfp4_gemm_nt(*good[:4], z(4, 16, dt=torch.float32))
    with pytest.raises(TypeError):
        dg.dg_quant_mxfp4(z(4, 128, dt=torch.float16), z(4, 64), z(1, 4, dt=i32))
    with pytest.raises(dg.DGError):  # K = 64
        dg.dg_mxfp4_gemm_nt(z(4, 32), z(0, 4, dt=i32), z(16, 32), z(0, 16, dt=i32), z(4, 16, dt=bf))
    with pytest.raises(ValueError):  # host tensors
        dg.dg_mxfp4_gemm_nt(*(t.cpu() for t in good))
    rc = dg.load_library().dg_mxfp4_gemm_nt(*(ctypes.c_void_p(t.data_ptr()) for t in good[:4]), ctypes.c_void_p(good[4].data_ptr() + 2),
                                            4, 16, 128, None, 0, None)
    assert rc == dg.DG_ERR_ALIGN
