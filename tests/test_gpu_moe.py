"""Router, row layout and combine on the GPU against the 64-bit oracle.

Bounds (u = 2^-24).  A probability: the difference l - m is rounded once (u |l - m|
in the exponent), exp and the division are within 2 ulp each, a row's sum adds
at most 30 roundings: (2 |l - m| + 40) u relative, D = largest |l - m| of the
finite logits that matter (beyond 110 the exponential is 0 in fp32).  prob_sum
adds one rounding per addition a term passes (at most min(T, 600) + 100).
A gradient: (4 D + 100) u of the sum of its terms' magnitudes, and its own
rounding (bf16: 8 significant bits, 2^-8).  combine: k roundings of the sum of the magnitudes."""

import numpy as np
import pytest
import torch

from moe_grouped_matmul_amd import dg
from oracle import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _ws(op, *shape):
    return torch.zeros(dg.dg_get_workspace_size(op, *shape), dtype=torch.uint8, device=DEV)


def _gate(x, k, valid=None, ws=None, **kw):
    T, E = x.shape
    i32 = dict(dtype=torch.int32, device=DEV)
    o = dict(topk_idx=torch.full((T, k), 77, **i32), topk_w=torch.full((T, k), 7.0, device=DEV), counts=torch.full((E + 1,), 7, **i32),
             prob_sum=torch.full((E,), 7.0, device=DEV), loss=torch.full((1,), 7.0, device=DEV))
    dg.dg_moe_gate(x, *o.values(), valid=valid, workspace=_ws(dg.DG_OP_MOE_GATE, T, E, k) if ws is None else ws, **kw)
    return o


def _spread(x):
    """Largest distance of a logit that matters from its row's maximum."""
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(x), x, -np.inf).max(1, keepdims=True) - x
    return float(np.max(np.where(np.isfinite(d) & (d < 110), d, 0.0), initial=0.0))


def _close(got, want, tol, what):
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    bad = ~(np.abs(got - want) <= tol) & ~np.isnan(want)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax((np.abs(got - want) - tol))))


def _check_gate(o, want, x, T):
    D = _spread(x)
    assert np.array_equal(o["topk_idx"].cpu().numpy(), want["topk_idx"])
    assert np.array_equal(o["counts"].cpu().numpy(), want["counts"])
    rel = (2 * D + 40) * U
    tiny = 1e-37  # fp32 exponentials below their normal range are coarse
    _close(o["topk_w"].cpu(), want["topk_w"], 2 * rel * np.abs(want["topk_w"]) + tiny, "weights")
    _close(o["prob_sum"].cpu(), want["prob_sum"], (rel + (min(T, 600) + 100) * U) * np.abs(want["prob_sum"]) + tiny * T, "prob_sum")
    _close(o["loss"].cpu(), [want["loss"]], (rel + (min(T, 600) + 1200) * U) * abs(want["loss"]) + tiny, "loss")


def _logits(rng, T, E, dtype, kind):
    x = rng.standard_normal((T, E)).astype(np.float32) * 2
    if kind == "ties":
        x = np.round(x)
    if kind == "masked":  # expert masks: -inf or the type's lowest value, some rows with few or no experts left
        drop = rng.random((T, E)) < 0.6
        x[drop] = -np.inf
        x[::5] = -np.inf
        x[1::5, : E // 2] = torch.finfo(dtype).min
        x[2::5] = torch.finfo(dtype).min
        x[3::5, 1:] = -np.inf
    if kind == "wide":
        x *= 40
    X = _t(x).to(dtype)
    return X, X.double().cpu().numpy()


GATE = [(1, 1, 1), (1, 8, 2), (3, 60, 4), (64, 256, 8), (37, 64, 6), (130, 97, 16), (300, 128, 1), (5, 1024, 16), (70, 512, 8),
        (33, 257, 3), (2500, 16, 2), (5000, 256, 8)]


@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "wide"])
@pytest.mark.parametrize("T,E,k", GATE)
def test_gate_and_gradient(T, E, k, kind):
    rng = np.random.default_rng(T + E + k)
    dtype = torch.bfloat16 if (T + E) % 2 else torch.float32
    X, x = _logits(rng, T, E, dtype, kind)
    renorm = bool(k % 3)
    valid = _t(rng.random(T) < 0.8) if T % 3 == 0 else None
    kw = dict(renorm=renorm, w_scale=2.5 if T % 2 else 1.0, loss_coef=0.02)
    o = _gate(X, k, valid, **kw)
    want = moe.gate(x, k, valid=None if valid is None else valid.cpu().numpy(), **kw)
    _check_gate(o, want, x, T)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for use_dw, dl in ((True, 1.5), (False, 1.5), (True, None)):
        got = torch.full((T, E), 7.0, dtype=dtype, device=DEV)
        dg.dg_moe_gate_bwd(X, o["topk_idx"], o["topk_w"], o["counts"], _t(dw) if use_dw else None,
                           None if dl is None else torch.full((1,), dl, device=DEV), got, **kw)
        d, mag = moe.gate_grad(want, dw if use_dw else 0 * dw, dl or 0.0, **kw)
        out = 2.0 ** -8 if dtype is torch.bfloat16 else U
        _close(got.double().cpu(), d, out * np.abs(d) * 1.01 + (4 * _spread(x) + 100) * U * mag + 1e-37, (use_dw, dl))


def test_gate_not_numbers_and_masked_nan():
    inf, nan = np.inf, np.nan
    x = np.array([[-inf] * 4, [0, -inf, -inf, -inf], [nan, 1, 2, 0], [0, inf, 1, -inf], [nan] * 4, [5, 6, 7, 8]], np.float32)
    for valid in (None, np.array([1, 1, 0, 0, 0, 1], bool)):
        o = _gate(_t(x), 2, None if valid is None else _t(valid), loss_coef=1.0)
        want = moe.gate(x, 2, valid=valid, loss_coef=1.0)
        _check_gate(o, want, x, 6)
        assert np.isnan(want["loss"]) == (valid is None)
        got = torch.empty(6, 4, device=DEV)
        dg.dg_moe_gate_bwd(_t(x), o["topk_idx"], o["topk_w"], o["counts"], torch.ones(6, 2, device=DEV), None, got, loss_coef=1.0)
        g = got.cpu().numpy()
        assert not g[[0, 4]].any() and np.isfinite(g[[0, 1, 5]]).all()
        assert np.isnan(g[[2, 3]]).all() if valid is None else not g[2:5].any()


def test_gate_no_tokens_and_all_masked():
    for T, valid in ((0, None), (50, torch.zeros(50, dtype=torch.uint8, device=DEV))):
        o = _gate(torch.full((T, 12), float("nan"), device=DEV), 3, valid, loss_coef=1.0)
        assert o["loss"].item() == 0 and not o["counts"].any() and not o["prob_sum"].any()
        assert (o["topk_idx"] == -1).all() and not o["topk_w"].any()


def test_gate_repeats_bit_identical_and_workspace_reusable():
    rng = np.random.default_rng(7)
    ws = _ws(dg.DG_OP_MOE_GATE, 9000, 256, 8)
    for T, E in ((9000, 256), (40, 8), (9000, 256), (700, 256)):
        X = _t(rng.standard_normal((T, E)).astype(np.float32))
        first = _gate(X, 8, ws=ws, loss_coef=0.5)
        again = _gate(X, 8, ws=_ws(dg.DG_OP_MOE_GATE, T, E, 8), loss_coef=0.5)
        for n in first:
            assert torch.equal(first[n], again[n]), n
        assert int(first["counts"][:E].sum()) == 8 * T


def test_gate_gradient_against_differences():
    """The GPU's own forward, differenced in directions, against its gradient (fp32: steps of 2^-6)."""
    rng = np.random.default_rng(11)
    T, E, k = 40, 24, 4
    x = rng.standard_normal((T, E)).astype(np.float32) * 2
    dw = _t(rng.standard_normal((T, k)).astype(np.float32))
    kw = dict(renorm=True, w_scale=1.5, loss_coef=0.7)
    o = _gate(_t(x), k, **kw)
    d = torch.empty(T, E, device=DEV)
    dg.dg_moe_gate_bwd(_t(x), o["topk_idx"], o["topk_w"], o["counts"], dw, torch.ones(1, device=DEV), d, **kw)
    top = np.sort(x, 1)[:, ::-1]
    safe = top[:, k - 1] - top[:, k] > 0.1  # rows whose choice a step cannot change, nor the order within it
    safe &= (top[:, :k - 1] - top[:, 1:k]).min(1) > 0.1
    assert safe.sum() > 3
    for _ in range(6):
        v = rng.uniform(-1, 1, (T, E)).astype(np.float32) * safe[:, None]
        h = 2.0 ** -6
        f = [(_gate(_t(x + s * h * v), k, **kw)) for s in (1, -1)]
        assert torch.equal(f[0]["topk_idx"], f[1]["topk_idx"])
        num = ((f[0]["topk_w"].double() - f[1]["topk_w"].double()) * dw.double()).sum() + (f[0]["loss"] - f[1]["loss"]).double().sum()
        num = num.item() / (2 * h)
        ana = (d.double().cpu().numpy() * v).sum()
        # third derivatives of a softmax weight are below 1: h^2 / 6 of the sum of |v|^3 |dw|, and fp32 noise of the two values
        tol = h * h / 6 * 2 * float(dw.abs().sum()) * 1.5 + 2 * (T * k * 1.5 * 60 * U) / (2 * h)
        assert abs(num - ana) <= tol


LAYOUT = [(1, 1, 1, 0, 1), (5, 2, 8, 0, 8), (64, 8, 256, 64, 32), (300, 8, 256, 0, 256), (1000, 3, 60, 7, 40), (4097, 8, 64, 0, 64), (700, 16, 1024, 0, 1024),
          (9000, 1, 4, 1, 2)]


@pytest.mark.parametrize("T,k,E,first,G", LAYOUT)
def test_layout(T, k, E, first, G):
    rng = np.random.default_rng(T + E)
    p = rng.random(E) ** 2 + 1e-3
    idx = np.argsort(-(np.log(p) + rng.gumbel(size=(T, E))), 1)[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < 0.1] = -1
    ws = _ws(dg.DG_OP_MOE_LAYOUT, T, 0, k, G)
    full = (T * k + 127 * G + 127) // 128 * 128
    for M in (full, max(128, full // 256 * 128), 0):  # enough rows, too few, none
        want = moe.layout(idx, first, G, rows=M)
        o = dict(counts=G, m_indices=M, row_token=M, row_of=(T, k))
        o = {n: torch.full((s,) if isinstance(s, int) else s, 77, dtype=torch.int32, device=DEV) for n, s in o.items()}
        dg.dg_moe_layout_contiguous(_t(idx), *o.values(), first_expert=first, workspace=ws)
        for n in o:
            assert np.array_equal(o[n].cpu().numpy(), want[n]), (n, M)
    for max_m in (1, 64, 130):
        want = moe.layout(idx, first, G, max_m=max_m)
        o = dict(counts=(G,), row_token=(G, max_m), row_of=(T, k))
        o = {n: torch.full(s, 77, dtype=torch.int32, device=DEV) for n, s in o.items()}
        dg.dg_moe_layout_masked(_t(idx), *o.values(), first_expert=first, workspace=ws)
        for n in o:
            assert np.array_equal(o[n].cpu().numpy().ravel(), want[n].ravel()), (n, max_m)


@pytest.mark.parametrize("T,k,E,first,G", [(40000, 4, 96, 0, 96), (70001, 4, 48, 8, 32)])
def test_layout_of_many_choices(T, k, E, first, G):
    """Blocks of several runs of choices each: two of them, and more than are kept in registers."""
    idx = np.argsort(np.random.default_rng(T).random((T, E)), 1)[:, :k].astype(np.int32)
    ws = _ws(dg.DG_OP_MOE_LAYOUT, T, 0, k, G)
    i32 = dict(dtype=torch.int32, device=DEV)
    M = (T * k + 127 * G + 127) // 128 * 128
    for _ in range(2):
        o = dict(counts=torch.full((G,), 77, **i32), m_indices=torch.full((M,), 77, **i32), row_token=torch.full((M,), 77, **i32), row_of=torch.full((T, k), 77, **i32))
        dg.dg_moe_layout_contiguous(_t(idx), *o.values(), first_expert=first, workspace=ws)
        want = moe.layout(idx, first, G, rows=M)
        for n in o:
            assert np.array_equal(o[n].cpu().numpy(), want[n]), n
    max_m = T * k // E
    m, rt, ro = torch.full((G,), 77, **i32), torch.full((G, max_m), 77, **i32), torch.full((T, k), 77, **i32)
    dg.dg_moe_layout_masked(_t(idx), m, rt, ro, first_expert=first, workspace=ws)
    want = moe.layout(idx, first, G, max_m=max_m)
    for got, n in ((m, "counts"), (rt, "row_token"), (ro, "row_of")):
        assert np.array_equal(got.cpu().numpy().ravel(), want[n].ravel()), n


def test_layout_no_tokens_and_one_expert_takes_all():
    i32 = dict(dtype=torch.int32, device=DEV)
    ws = _ws(dg.DG_OP_MOE_LAYOUT, 5000, 0, 2, 3)
    o = [torch.full(s, 7, **i32) for s in ((3,), (256,), (256,), (0, 2))]
    dg.dg_moe_layout_contiguous(torch.empty(0, 2, **i32), *o, workspace=ws)
    assert not o[0].any() and (o[1] == -1).all() and (o[2] == -1).all()
    idx = torch.ones(5000, 2, **i32)
    o = [torch.full(s, 7, **i32) for s in ((3,), (10240,), (10240,), (5000, 2))]
    dg.dg_moe_layout_contiguous(idx, *o, workspace=ws)
    assert o[0].tolist() == [0, 10000, 0]
    assert torch.equal(o[3].flatten(), torch.arange(10000, **i32))


COMBINE = [(1, 1, 16), (5, 2, 272), (40, 8, 2064), (17, 16, 4096), (3, 3, 7168), (130, 6, 528)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,N", COMBINE)
def test_combine_and_gradient(T, k, N, dtype):
    rng = np.random.default_rng(T + k + N)
    R = T * k + 37
    rows = _t(rng.standard_normal((R, N)).astype(np.float32)).to(torch.bfloat16)
    row_of = rng.permutation(R)[: T * k].reshape(T, k).astype(np.int32)
    row_of[rng.random((T, k)) < 0.15] = -1
    if T > 2:
        row_of[1] = -1       # a token without rows
        row_of[2, 0] = R + 5  # and a row that does not exist
    unused = np.setdiff1d(np.arange(R), row_of)
    rows[_t(unused)] = float("nan")  # never read
    w = rng.standard_normal((T, k)).astype(np.float32)
    r64 = np.nan_to_num(rows.double().cpu().numpy())
    y = torch.full((T, N), 7.0, dtype=dtype, device=DEV)
    dg.dg_moe_combine(rows, _t(row_of), _t(w), y)
    want, mag = moe.combine(r64, row_of, w.astype(np.float64))
    out = 2.0 ** -8 if dtype is torch.bfloat16 else U
    _close(y.double().cpu(), want, out * 1.01 * np.abs(want) + (k + 1) * U * mag, "y")
    dy = _t(rng.standard_normal((T, N)).astype(np.float32)).to(dtype)
    drows = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, k), 7.0, device=DEV)
    dg.dg_moe_combine_bwd(dy, rows, _t(row_of), _t(w), drows, dw)
    wr, wd, wm = moe.combine_grad(dy.double().cpu().numpy(), r64, row_of, w.astype(np.float64))
    got = drows.double().cpu().numpy()
    assert np.all(got[unused] == 7.0)
    wr = np.where(np.isnan(wr), 7.0, wr)
    _close(got, wr, (2.0 ** -8 * 1.01 + U) * np.abs(wr), "drows")
    _close(dw.cpu(), wd, (N / 256 + 20) * U * wm, "dw")


def test_refusals():
    i32, f = dict(dtype=torch.int32, device=DEV), dict(device=DEV)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)

    def gate(T=4, E=8, k=2, x=None, ws=ws, idx=None, **kw):
        dg.dg_moe_gate(torch.zeros(T, E, **f) if x is None else x, torch.empty(T, k, **i32) if idx is None else idx, torch.empty(T, k, **f),
                       torch.empty(E + 1, **i32), torch.empty(E, **f), torch.empty(1, **f), workspace=ws, **kw)

    gate()
    for kw, err in ((dict(k=9), dg.DGError), (dict(E=1025), dg.DGError), (dict(E=32, k=17), dg.DGError), (dict(ws=None), dg.DGError),
                    (dict(ws=ws[:16]), dg.DGError), (dict(w_scale=0.0), dg.DGError), (dict(w_scale=float("nan")), dg.DGError),
                    (dict(x=torch.zeros(4, 8, dtype=torch.float16, **f)), TypeError), (dict(x=torch.zeros(4, 8)), ValueError),
                    (dict(x=torch.zeros(8, 4, **f).t()), ValueError), (dict(idx=torch.empty(4, 2, dtype=torch.int64, **f)), TypeError),
                    (dict(valid=torch.ones(5, dtype=torch.bool, **f)), ValueError), (dict(valid=torch.ones(4, **f)), TypeError)):
        with pytest.raises(err):
            gate(**kw)
    lay = lambda G=2, k=2, **kw: dg.dg_moe_layout_contiguous(  # noqa: E731
        torch.zeros(4, k, **i32), torch.empty(G, **i32), torch.empty(256, **i32), torch.empty(256, **i32), torch.empty(4, k, **i32), **kw)
    lay(workspace=ws)
    for kw, err in ((dict(), dg.DGError), (dict(workspace=ws, first_expert=-1), dg.DGError), (dict(workspace=ws, G=1025), dg.DGError),
                    (dict(workspace=ws, k=17), dg.DGError), (dict(workspace=ws[1:]), dg.DGError)):
        with pytest.raises(err):
            lay(**kw)
    with pytest.raises(dg.DGError):  # no capacity
        dg.dg_moe_layout_masked(torch.zeros(4, 2, **i32), torch.empty(2, **i32), torch.empty(2, 0, **i32), torch.empty(4, 2, **i32), workspace=ws)
    comb = lambda N=16, k=2, dt=torch.bfloat16: dg.dg_moe_combine(  # noqa: E731
        torch.zeros(9, N, dtype=torch.bfloat16, **f), torch.zeros(4, k, **i32), torch.zeros(4, k, **f), torch.empty(4, N, dtype=dt, **f))
    comb()
    for kw, err in ((dict(N=24), dg.DGError), (dict(k=17), dg.DGError), (dict(dt=torch.float16), TypeError)):
        with pytest.raises(err):
            comb(**kw)
