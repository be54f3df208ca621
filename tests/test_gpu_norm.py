"""Root-mean-square norm, its quantised outputs and its gradient on the GPU against the 64-bit oracle.

Bounds (u = 2^-24).  A row's sum of squares is positive and passes at most 8 * 16 additions in a lane and 12 across lanes and
waves, so it is within 150 u; the mean, the addition of eps, the root and the quotient add 4: rstd is within 80 u.  v = (h r) w
adds 2: E = 82 u.  y: E and half a step of its type (bf16 2^-8).  sf: E and its division; a code: half a step of e4m3 on
v / s, 2^-4 of v or, below 2^-6 s, 2^-10 s, and E.  A power-of-two scale is the oracle's, or its neighbour where amax / 448 is
within E of a power of two.  dx: with S = r (|w dy| + |n| mean|w dy n|) + |dh|, rstd enters up to three times (240 u), the mean
adds 150 u and the rest 10: 400 u S and half a step.  dw: (M + 100) u of the sum of the magnitudes."""

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_matmul_amd import dg
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0**-24
E = 82 * U


def _step(dt):
    return torch.finfo(dt).eps / 2


def _rows(M, K, dt, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, device=DEV, generator=g)
    return (scale * torch.where(torch.rand(M, K, device=DEV, generator=g) < 0.01, 20 * x, x)).to(dt)


def _np(t):
    return t.double().cpu().numpy()


def _ws(M, K):
    # not zero, as the operator allows
    return torch.full((dg.dg_get_workspace_size(dg.DG_OP_RMS_NORM_BWD, M, 0, K),), 0x7F, dtype=torch.uint8, device=DEV)


def _near(got, want, tol, what):
    bad = ~(np.abs(_np(got) - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.max(np.abs(_np(got) - want) - tol)))


def _check_codes(q, sf, v, M, K):
    """q, sf of the fp32 or the UE8M0 form against the values v."""
    kb = K // 128
    amax = np.abs(v).reshape(M, kb, 128).max(2)
    if sf.dtype == torch.int32:
        words = sf.cpu().numpy().view(np.uint8).reshape((kb + 3) // 4, M, 4)
        codes = words.transpose(1, 0, 2).reshape(M, -1)
        assert (codes[:, kb:] == 0).all()
        s = 2.0 ** (codes[:, :kb].astype(np.float64) - 127)
        assert ((s * 448 >= amax * (1 - E)) & (s * 224 <= amax * (1 + E)) | (amax == 0) & (s == 1)).all()
    else:
        s = _np(sf).T
        want = np.where(amax == 0, 1.0, amax / 448)
        assert (np.abs(s - want) <= (E + U) * want).all()
    s = np.repeat(s, 128, 1)
    back = oracle.decode_e4m3(q.cpu().numpy()) * s
    tol = np.maximum(2.0**-4 * np.abs(v), 2.0**-10 * s) * (1 + 4 * E) + 4 * E * np.abs(v)
    bad = ~(np.abs(back - v) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())


def _norm(x, w, residual=None, kind=None, y=True, eps=1e-6, stream=None):
    M, K = x.shape
    o = {"h": torch.full_like(x, 7.0) if residual is not None else None, "y": torch.full_like(x, 7.0) if y else None,
         "rstd": torch.full((M,), 7.0, device=DEV), "q": None, "sf": None}
    if kind:
        o["q"] = torch.full((M, K), 0x55, dtype=torch.uint8, device=DEV)
        o["sf"] = torch.full((K // 128, M), 7.0, device=DEV) if kind == "f32" else torch.full(((K + 511) // 512, M), -1, dtype=torch.int32, device=DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())  # the outputs are filled there
    dg.dg_rms_norm(x, w, residual=residual, eps=eps, stream=stream, **o)
    return o


def _check_norm(o, x, w, residual, eps=1e-6):
    M, K = x.shape
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    if residual is not None:
        assert torch.equal(o["h"], h)
    v, rstd = block.rms_norm(_np(h), _np(w), eps)
    _near(o["rstd"], rstd, 80 * U * rstd, "rstd")
    if o["y"] is not None:
        _near(o["y"], v, (E + _step(x.dtype)) * np.abs(v) * (1 + 1e-3) + 1e-38, "y")
    if o["q"] is not None:
        _check_codes(o["q"], o["sf"], v, M, K)
    return h


SHAPES = [(1, 128), (1, 16384), (2, 640), (3, 7168), (5, 512), (7, 1152), (17, 2048), (64, 4224), (65, 384), (130, 8192), (33, 8320),
          (257, 256), (1021, 1024), (9, 12416), (2100, 896), (3000, 4736), (2500, 7168), (1100, 16384)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_norm(M, K, dt):
    wt = torch.float32 if (M + K // 128) % 2 else dt
    x, w = _rows(M, K, dt, 1), (1 + 0.2 * _rows(1, K, torch.float32, 2)[0]).to(wt)
    res = _rows(M, K, dt, 3) if M % 3 != 2 else None
    kind = ("f32", "ue8m0", None)[(M + K // 128) % 3]
    _check_norm(_norm(x, w, res, kind, y=kind is None or M % 2 == 0), x, w, res)


@pytest.mark.parametrize("kind", ["f32", "ue8m0"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 7168), (2500, 7168), (300, 128), (40, 16384)])
def test_norm_quantised(M, K, dt, kind):
    x, w, res = _rows(M, K, dt, 5), 1 + 0.2 * _rows(1, K, torch.float32, 6)[0], _rows(M, K, dt, 7)
    _check_norm(_norm(x, w, res, kind), x, w, res)


@pytest.mark.parametrize("M,K", [(1, 8), (3, 24), (65, 520), (200, 1000), (1000, 5000), (12, 16376)])
def test_norm_columns_of_any_eight(M, K):
    for dt in (torch.bfloat16, torch.float32):
        x, w, res = _rows(M, K, dt, 8), 1 + 0.2 * _rows(1, K, torch.float32, 9)[0], _rows(M, K, dt, 10)
        _check_norm(_norm(x, w, res), x, w, res)


def test_codes_are_those_of_the_quantiser():
    # without a residual and with a weight of ones, on rows whose factor is 1, v is x: the codes are dg_quant_1x128's
    M, K = 33, 1024
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.where(torch.rand(M, K, device=DEV, generator=g) < 0.5, -1.0, 1.0)
    x[:, ::2] *= torch.where(torch.arange(K // 2, device=DEV) % 2 == 0, 0.6, 1.28**0.5)  # mean square (0.5 + (0.36 + 1.28) / 4) differs by row of none
    w = torch.ones(K, device=DEV)
    o = _norm(x, w, None, "f32")
    v = o["y"]
    q, sf = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(K // 128, M, device=DEV)
    dg.dg_quant_1x128(v, q, sf)
    assert torch.equal(q, o["q"]) and torch.equal(sf, o["sf"])
    o = _norm(x, w, None, "ue8m0")
    sf = torch.empty((K + 511) // 512, M, dtype=torch.int32, device=DEV)
    dg.dg_quant_1x128_ue8m0(v, q, sf)
    assert torch.equal(q, o["q"]) and torch.equal(sf, o["sf"])


@pytest.mark.parametrize("K", [640, 7168])
def test_fp32_codes_equal_the_quantiser_of_y(K):
    for kind, quant in (("f32", dg.dg_quant_1x128), ("ue8m0", dg.dg_quant_1x128_ue8m0)):
        x, w, res = _rows(37, K, torch.float32, 1), 1 + 0.2 * _rows(1, K, torch.float32, 2)[0], _rows(37, K, torch.float32, 3)
        o = _norm(x, w, res, kind)
        q, sf = torch.empty_like(o["q"]), torch.empty_like(o["sf"])
        quant(o["y"], q, sf)  # in fp32, y is v
        assert torch.equal(q, o["q"]) and torch.equal(sf, o["sf"])


def test_rows_of_zeros_large_and_nonfinite():
    K = 512
    x = _rows(6, K, torch.float32, 4)
    x[1] = 0
    x[2] *= 1e-25
    x[3] *= 1e18  # sum of squares 5e38: past fp32, r = 0
    x[4, 7] = float("nan")
    x[5, 9] = float("inf")
    w = torch.ones(K, device=DEV)
    o = _norm(x, w, None, "f32")
    assert (o["y"][1] == 0).all() and (o["q"][1] & 0x7F == 0).all() and (o["sf"][:, 1] == 1).all()
    assert (o["rstd"][1] - 1e3).abs() <= 1e3 * 80 * U
    assert o["rstd"][3] == 0 and (o["y"][3] == 0).all()
    assert o["y"][4].isnan().all() and o["y"][5, 9].isnan() and (o["y"][5, :9] == 0).all()
    clean = _norm(x[:1].contiguous(), w, None, "f32")
    assert torch.equal(clean["y"][0], o["y"][0]) and torch.equal(clean["q"][0], o["q"][0])


def test_in_place_and_streams():
    M, K = 70, 2304
    w = 1 + 0.2 * _rows(1, K, torch.float32, 2)[0]
    for dt in (torch.bfloat16, torch.float32):
        x, res = _rows(M, K, dt, 1), _rows(M, K, dt, 3)
        want = _norm(x, w, res, "f32")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = _norm(x, w, res, "f32", stream=s)
        torch.cuda.current_stream().wait_stream(s)
        for n in ("h", "y", "q", "sf", "rstd"):
            assert torch.equal(got[n], want[n])
        r2, x2 = res.clone(), x.clone()
        dg.dg_rms_norm(x2, w, residual=r2, h=r2, y=x2)  # the residual stream in place, the output over x
        assert torch.equal(r2, want["h"]) and torch.equal(x2, want["y"])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 8), (2, 1024), (3, 520), (8, 512), (65, 2048), (300, 1000), (1000, 4096), (5, 8192), (700, 7168), (90, 12800),
                                 (33, 16384), (6000, 256)])
def test_norm_bwd(M, K, dt):
    h, dy, dh = _rows(M, K, dt, 1), _rows(M, K, dt, 2), _rows(M, K, dt, 3)
    w = (1 + 0.2 * _rows(1, K, torch.float32, 4)[0]).to(torch.float32 if M % 2 else dt)
    o = _norm(h, w)
    dx, dw, ws = torch.full_like(h, 7.0), torch.full((K,), 7.0, device=DEV), _ws(M, K)
    before = ws[:4096].clone()
    for extra in (dh, None):
        dg.dg_rms_norm_bwd(dy, h, w, o["rstd"], dx, dw, dh=extra, workspace=ws)
        hn, dyn, wn = _np(h), _np(dy), _np(w)
        want_x, want_w = block.rms_norm_bwd(dyn, hn, wn, 1e-6, None if extra is None else _np(extra))
        r = 1 / np.sqrt((hn * hn).mean(1, keepdims=True) + 1e-6)
        n = hn * r
        mag = r * (np.abs(wn * dyn) + np.abs(n) * np.abs(wn * dyn * n).mean(1, keepdims=True)) + (0 if extra is None else np.abs(_np(extra)))
        _near(dx, want_x, _step(dt) * np.abs(want_x) * 1.001 + 400 * U * mag, "dx")
        _near(dw, want_w, (M + 100) * U * np.abs(dyn * n).sum(0), "dw")
    assert torch.equal(ws[:4096], before)  # counters of other operators


def test_norm_bwd_against_differences():
    M, K = 4, 256
    h, dy, w = _rows(M, K, torch.float32, 1), _rows(M, K, torch.float32, 2), 1 + 0.2 * _rows(1, K, torch.float32, 3)[0]
    o = _norm(h, w, eps=1e-3)
    dx, dw = torch.empty_like(h), torch.empty(K, device=DEV)
    dg.dg_rms_norm_bwd(dy, h, w, o["rstd"], dx, dw, workspace=_ws(M, K))
    g = torch.Generator(device=DEV).manual_seed(9)
    dirx, dirw = torch.randn(M, K, device=DEV, generator=g), torch.randn(K, device=DEV, generator=g)
    t = 2.0**-7
    f = lambda a, b: (_norm(a, b, eps=1e-3)["y"].double() * dy.double()).sum()  # noqa: E731
    for grad, lo, hi in (((dx.double() * dirx.double()).sum(), f(h - t * dirx, w), f(h + t * dirx, w)),
                         ((dw.double() * dirw.double()).sum(), f(h, w - t * dirw), f(h, w + t * dirw))):
        # the difference's own error: curvature (t^2 times third derivatives of order |dy|) and fp32 roundings of y over 2 t
        assert abs((hi - lo) / (2 * t) - grad) <= (t * t + 84 * U / t) * dy.double().abs().sum() * 4


def test_norm_bwd_in_place_and_deterministic():
    M, K = 300, 2048
    h, dy, w = _rows(M, K, torch.bfloat16, 1), _rows(M, K, torch.bfloat16, 2), torch.ones(K, device=DEV)
    rstd = _norm(h, w)["rstd"]
    dx, dw, ws = torch.empty_like(h), torch.empty(K, device=DEV), _ws(M, K)
    dg.dg_rms_norm_bwd(dy, h, w, rstd, dx, dw, dh=dy, workspace=ws)
    for over in (dy, h):
        a, b = dy.clone(), h.clone()
        out = a if over is dy else b
        dw2 = torch.empty_like(dw)
        dg.dg_rms_norm_bwd(a, b, w, rstd, out, dw2, dh=dy, workspace=ws)
        assert torch.equal(out, dx) and torch.equal(dw2, dw)


def test_without_rows():
    K = 256
    x, w = torch.empty(0, K, device=DEV), torch.ones(K, device=DEV)
    dg.dg_rms_norm(x, w, y=x.clone())
    dw = torch.full((K,), 7.0, device=DEV)
    dg.dg_rms_norm_bwd(x, x, w, torch.empty(0, device=DEV), x, dw, workspace=_ws(0, K))
    assert (dw == 0).all()


def test_graph_replays():
    M, K = 50, 2048
    x, res, dy, w = (_rows(n, K, torch.bfloat16, i) for i, n in enumerate((M, M, M, 1)))
    w = w[0].contiguous()
    h, y, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    q, sf = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(K // 128, M, device=DEV)
    rstd, dw, ws = torch.empty(M, device=DEV), torch.empty(K, device=DEV), _ws(M, K)

    def step():
        dg.dg_rms_norm(x, w, residual=res, h=h, y=y, q=q, sf=sf, rstd=rstd)
        dg.dg_rms_norm_bwd(dy, h, w, rstd, dx, dw, dh=dy, workspace=ws)
        return [t.clone() for t in (h, y, q, sf, rstd, dx, dw)]

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.dg_rms_norm(x, w, residual=res, h=h, y=y, q=q, sf=sf, rstd=rstd)
        dg.dg_rms_norm_bwd(dy, h, w, rstd, dx, dw, dh=dy, workspace=ws)
    for i in range(3):
        x.copy_(_rows(M, K, torch.bfloat16, 20 + i))
        want = step()
        for t in (h, y, q, sf, rstd, dx, dw):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (h, y, q, sf, rstd, dx, dw)))


def test_binding_refusals():
    x, w = _rows(4, 256, torch.bfloat16, 1), torch.ones(256, device=DEV)
    y = torch.empty_like(x)
    with pytest.raises(ValueError, match="contiguous"):
        dg.dg_rms_norm(x.t().contiguous().t(), w, y=y)
    with pytest.raises(TypeError, match="residual"):
        dg.dg_rms_norm(x, w, residual=x.float(), h=y, y=y)
    with pytest.raises(ValueError, match="weight"):
        dg.dg_rms_norm(x, w[:128], y=y)
    with pytest.raises(TypeError, match="x must be"):
        dg.dg_rms_norm(x.half(), w, y=y)
    with pytest.raises(ValueError, match="device"):
        dg.dg_rms_norm(x.cpu(), w, y=y)
    with pytest.raises(dg.DGError, match="null"):
        dg.dg_rms_norm(x, w)
    with pytest.raises(dg.DGError, match="workspace"):
        dg.dg_rms_norm_bwd(x, x, w, torch.ones(4, device=DEV), y, torch.empty(256, device=DEV))
