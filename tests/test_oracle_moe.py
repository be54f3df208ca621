"""Pins of the 64-bit mixture-of-experts and 4-bit oracles (CPU): worked values,
the quantiser against a search over all codes, gradients against differences."""

import numpy as np
import pytest

from oracle import moe, mxfp4


def test_e2m1_rounding_and_scale_choice():
    # amax 6 * 2^0: scale 1; midpoints go to the even code, sign of zero kept
    x = np.zeros((1, 128), np.float32)
    x[0, :10] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0, -5.01]
    q, s = mxfp4.quant_mxfp4(x)
    assert mxfp4.unpack_words(s)[0].tolist() == [127, 127, 127, 127]
    v = mxfp4.values_mxfp4(q, s)[0]
    assert v[:10].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -6] and np.signbit(v[8])
    # just above 6: the next power of two; at 6 exactly not
    x[0, 0] = np.nextafter(np.float32(6), np.float32(7))
    assert mxfp4.unpack_words(mxfp4.quant_mxfp4(x)[1])[0, 0] == 128
    # the extremes of fp32
    x[0, 0] = np.finfo(np.float32).max
    assert mxfp4.unpack_words(mxfp4.quant_mxfp4(x)[1])[0, 0] == 253
    x[:] = 0
    x[0, 0], x[0, 40], x[0, 70], x[0, 100] = 1e-45, 2.0 ** -126, np.nan, -np.inf
    q, s = mxfp4.quant_mxfp4(x)
    assert mxfp4.unpack_words(s)[0].tolist() == [0, 0, 255, 255]  # 2^-126 / 6 lies between 2^-129 and 2^-128: clamped
    v = mxfp4.values_mxfp4(q, s)[0]
    assert v[40] == 2.0 ** -126 and np.isnan(v[64:]).all()


def test_quantiser_is_nearest_under_the_least_scale():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((64, 128)) * 2.0 ** rng.integers(-40, 40, (64, 128))).astype(np.float32)
    q, s = mxfp4.quant_mxfp4(x)
    c = mxfp4.unpack_words(s).astype(np.float64)
    b = np.abs(x.astype(np.float64)).reshape(64, 4, 32).max(-1)
    assert np.all(6 * 2 ** (c - 127) >= b) and np.all(6 * 2 ** (c - 128) < b)
    v = mxfp4.values_mxfp4(q, s).reshape(64, 4, 32, 1)
    grid = np.concatenate([mxfp4.E2M1, -mxfp4.E2M1]) * 2 ** (c - 127)[..., None, None]
    xb = x.astype(np.float64).reshape(64, 4, 32, 1)
    assert np.all(np.abs(v[..., 0] - xb[..., 0]) <= np.abs(grid - xb).min(-1))


def test_gate_worked_row_and_ties():
    x = np.log(np.array([[1.0, 4.0, 2.0, 1.0], [1, 1, 1, 1]]))
    o = moe.gate(x, 2, loss_coef=1.0)
    assert o["topk_idx"].tolist() == [[1, 2], [0, 1]]
    assert np.allclose(o["topk_w"], [[2 / 3, 1 / 3], [0.5, 0.5]])
    assert o["counts"].tolist() == [1, 2, 1, 0, 2]
    p = np.array([1 / 8 + 1 / 4, 1 / 2 + 1 / 4, 1 / 4 + 1 / 4, 1 / 8 + 1 / 4])
    assert np.isclose(o["loss"], 4 * (np.array([1, 2, 1, 0]) / 4 * p / 2).sum())


def test_gate_rows_without_experts_and_not_numbers():
    inf, nan = np.inf, np.nan
    x = np.array([[-inf, -inf, -inf], [0, -inf, -inf], [nan, 1, 2], [0, inf, 1], [5, 6, 7]])
    o = moe.gate(x, 2, valid=[1, 1, 1, 1, 0], loss_coef=1.0)
    assert o["topk_idx"].tolist() == [[-1, -1], [0, -1], [2, 1], [1, 2], [-1, -1]]
    assert o["topk_w"][:2].tolist() == [[0, 0], [1, 0]] and np.isnan(o["topk_w"][2:4]).all()
    assert np.isnan(o["loss"]) and o["counts"].tolist() == [1, 2, 2, 3]
    o = moe.gate(x[:1], 2, loss_coef=1.0)
    assert o["loss"] == 0 and o["counts"].sum() == 0


@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    T, E, k = 5, 7, 3
    x = rng.standard_normal((T, E))
    x[1, 2] = -np.inf
    valid = np.array([1, 1, 1, 0, 1])
    dw = rng.standard_normal((T, k))
    kw = dict(renorm=renorm, w_scale=1.7, loss_coef=0.3)
    o = moe.gate(x, k, valid=valid, **kw)
    d, mag = moe.gate_grad(o, dw, 1.3, **kw)

    def f(y):
        q = moe.gate(y, k, valid=valid, **kw)
        assert (q["topk_idx"] == o["topk_idx"]).all()  # the counts are constants
        return (dw * q["topk_w"]).sum() + 1.3 * q["loss"]

    h = 1e-6
    for t in range(T):
        for e in range(E):
            if not np.isfinite(x[t, e]):
                assert d[t, e] == 0
                continue
            a, b = x.copy(), x.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((f(a) - f(b)) / (2 * h) - d[t, e]) < 1e-7
    assert np.all(np.abs(d) <= mag + 1e-15)


def test_layout_worked():
    idx = np.array([[2, 5], [5, 0], [5, 2], [-1, 9]])
    o = moe.layout(idx, 2, 4, rows=512)
    assert o["counts"].tolist() == [2, 0, 0, 3]
    assert o["row_of"].tolist() == [[0, 128], [129, -1], [130, 1], [-1, -1]]
    assert o["row_token"][[0, 1, 2, 128, 129, 130, 131]].tolist() == [0, 2, -1, 0, 1, 2, -1]
    assert o["m_indices"][[0, 1, 2, 128, 130]].tolist() == [0, 0, -1, 3, 3]
    o = moe.layout(idx, 2, 4, max_m=2)
    assert o["counts"].tolist() == [2, 0, 0, 2] and o["row_of"].tolist() == [[0, 6], [7, -1], [-1, 1], [-1, -1]]


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(4)
    rows, w = rng.standard_normal((6, 4)), rng.standard_normal((2, 3))
    row_of = np.array([[0, 5, -1], [2, 3, 1]])
    dy = rng.standard_normal((2, 4))
    drows, dw, _ = moe.combine_grad(dy, rows, row_of, w)
    f = lambda r, v: (dy * moe.combine(r, row_of, v)[0]).sum()  # noqa: E731
    h = 1e-6
    for i in range(6):
        for c in range(4):
            a, b = rows.copy(), rows.copy()
            a[i, c] += h
            b[i, c] -= h
            want = (f(a, w) - f(b, w)) / (2 * h)
            assert abs(want - (0 if np.isnan(drows[i, c]) else drows[i, c])) < 1e-8
    for t in range(2):
        for j in range(3):
            a, b = w.copy(), w.copy()
            a[t, j] += h
            b[t, j] -= h
            assert abs((f(rows, a) - f(rows, b)) / (2 * h) - dw[t, j]) < 1e-8
