"""The norm, the products' epilogue, their gradients and the experts as a program runs them together (examples/ffn_block.py and
the `few` path of examples/moe_layer.py): every stage against its 64-bit definition on the values that reached it, and the
gradients against the formula's.

Bounds as in test_gpu_norm.py, test_gpu_epilogue.py and test_gpu_experts.py.  The whole gradient: each of the quantised operands
(n, a, the two gradients, the four weights) is off by at most half a step of e4m3, 2^-4 of an element; a gradient passes five
products of two of them, whose relative errors in the 2-norm are independent of one another's signs and so add as squares, each
at most 2^-4 / sqrt(3) (an even spread over a step): sqrt(10) 2^-4 / sqrt(3) = 0.114 of the norm, with the bf16 roundings 0.12."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from helpers import acc_tolerance
from moe_grouped_matmul_amd import dg
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, B = 2.0**-24, 2.0**-8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _np(t):
    return t.double().cpu().numpy()


def _near(got, want, tol, what):
    bad = ~(np.abs(_np(got) - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist())


def _values(q, s):
    v = oracle.decode_e4m3(q.cpu().numpy())
    return v * np.repeat(_np(s).T, 128, 1)


def _weight_values(q, s):
    v = oracle.decode_e4m3(q.cpu().numpy())
    return v * np.repeat(np.repeat(_np(s), 128, 0)[: v.shape[0]], 128, 1)


def _product_tol(a, b, bias=None):
    c = None if bias is None else np.broadcast_to(bias.cpu().numpy(), (a[0].shape[0], b[0].shape[0]))
    return acc_tolerance(a[0].cpu().numpy(), a[1].cpu().numpy(), b[0].cpu().numpy(), b[1].cpu().numpy(), c)


def _block(m, H, F, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    w = dict(norm=1 + 0.1 * r(H), w1=r(F, H) / H**0.5, b1=0.1 * r(F), w2=r(H, F) / F**0.5, b2=0.1 * r(H))
    return m.DenseBlock(*w.values()), w, r


@pytest.mark.parametrize("M,H,F", [(128, 256, 384), (257, 512, 128), (1, 128, 256), (640, 384, 1024)])
def test_training_step(M, H, F):
    m = _example("ffn_block")
    b, w, r = _block(m, H, F, M)
    x, res, dy = (r(M, H).to(torch.bfloat16) for _ in range(3))
    y, kept = b.forward(x, res)
    back = b.backward(dy, kept)
    # forward, stage by stage
    assert torch.equal(kept["h"], (x.double() + res.double()).to(torch.bfloat16))
    v, rstd = block.rms_norm(_np(kept["h"]), _np(w["norm"]), 1e-6)
    _near(kept["rstd"], rstd, 80 * U * rstd, "rstd")
    s = np.repeat(_np(kept["n"][1]).T, 128, 1)
    n = _values(*kept["n"])
    assert (np.abs(n - v) <= np.maximum(2.0**-4 * np.abs(v), 2.0**-10 * s) * (1 + 400 * U) + 400 * U * np.abs(v)).all()
    t = _product_tol(kept["n"], b.w1, w["b1"])
    z = n @ _weight_values(*b.w1).T + _np(w["b1"])
    _near(kept["pre"], z, t + B * (np.abs(z) + t), "pre")
    act = block.act(z, "gelu")
    t1 = 1.2 * t + (16 + 8 * np.abs(z)) * U * np.maximum(np.abs(z), 1)
    _near(kept["a"], act, t1 + B * (np.abs(act) + t1), "a")
    qa = m._rows(kept["a"])
    out = _values(*qa) @ _weight_values(*b.w2).T + _np(w["b2"]) + _np(kept["h"])
    t = _product_tol(qa, b.w2, w["b2"]) + 2 * U * np.abs(out) + U * np.abs(_np(kept["h"]))
    _near(y, out, t + B * (np.abs(out) + t), "y")
    # backward, stage by stage
    dyn = _np(dy)
    _near(back["db2"], dyn.sum(0), (M + 40) * U * np.abs(dyn).sum(0), "db2")
    da = _values(*back["q2"]) @ _weight_values(*b.w2t).T
    t = _product_tol(back["q2"], b.w2t)
    _near(back["da"], da, t + B * (np.abs(da) + t), "da")
    dan, pre = _np(back["da"]), _np(kept["pre"])
    dz = dan * block.act_slope(pre, "gelu")
    e = (32 + 8 * np.abs(pre)) * U * np.abs(dan)
    _near(back["dz1"], dz, e + B * (np.abs(dz) + e), "dz1")
    _near(back["db1"], dz.sum(0), e.sum(0) + (M + 40) * U * np.abs(dz).sum(0), "db1")
    dn = _values(*back["q1"]) @ _weight_values(*b.w1t).T
    t = _product_tol(back["q1"], b.w1t)
    _near(back["dn"], dn, t + B * (np.abs(dn) + t), "dn")
    dnn, h = _np(back["dn"]), _np(kept["h"])
    dx, dnorm = block.rms_norm_bwd(dnn, h, _np(w["norm"]), 1e-6, dyn)
    wd, nn = np.abs(_np(w["norm"]) * dnn), np.abs(h * rstd[:, None])
    mag = rstd[:, None] * (wd + nn * (wd * nn).mean(1, keepdims=True)) + np.abs(dyn)
    _near(back["dx"], dx, B * np.abs(dx) * 1.001 + 400 * U * mag, "dx")
    _near(back["dnorm"], dnorm, (M + 100) * U * np.abs(dnn * h * rstd[:, None]).sum(0), "dnorm")


def test_gradients_are_the_formulas():
    m = _example("ffn_block")
    M, H, F = 384, 512, 640
    b, w, r = _block(m, H, F, 1)
    x, res, dy = (r(M, H).to(torch.bfloat16) for _ in range(3))
    y, kept = b.forward(x, res)
    back = b.backward(dy, kept)
    dw1, dw2 = b.weight_gradients(dy, kept, back)
    p = {k: v.double().cpu().requires_grad_(True) for k, v in w.items()}
    tx = x.double().cpu().requires_grad_(True)
    h = tx + res.double().cpu()
    n = torch.nn.functional.rms_norm(h, (H,), p["norm"], eps=1e-6)
    want = h + torch.nn.functional.gelu(n @ p["w1"].t() + p["b1"]) @ p["w2"].t() + p["b2"]
    g = torch.autograd.grad((want * dy.double().cpu()).sum(), (tx, p["norm"], p["w1"], p["b1"], p["w2"], p["b2"]))
    got = (back["dx"], back["dnorm"], dw1, back["db1"], dw2, back["db2"])
    assert (y.double().cpu() - want).norm() <= 0.12 * want.norm()
    for a, e, name in zip(got, g, ("dx", "dnorm", "dw1", "db1", "dw2", "db2")):
        assert (a.double().cpu() - e).norm() <= 0.12 * e.norm(), name


def _mxfp4(g, *shape):
    w = torch.randn(*shape, device=DEV, generator=g) / shape[-1] ** 0.5
    q = torch.empty(*shape[:-1], shape[-1] // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(shape[0], shape[-1] // 128, shape[1], dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(w, q, s)
    v = torch.empty(*shape, device=DEV)
    dg.dg_dequant_mxfp4(q, s, v)
    return (q, s), _np(v)


@pytest.mark.parametrize("T", [1, 13, 64])
def test_decode_step(T):
    m = _example("ffn_block")
    E, H, inner, k = 16, 384, 256, 4
    g = torch.Generator(device=DEV).manual_seed(T)
    gate_up, v1 = _mxfp4(g, E, 2 * inner, H)
    down, v2 = _mxfp4(g, E, H, inner)
    x, res = (torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    norm, router = 1 + 0.1 * torch.randn(H, device=DEV, generator=g), torch.randn(E, H, device=DEV, generator=g) / H**0.5
    out = m.moe_decode(x, res, norm, router, gate_up, down, k)
    assert torch.equal(out["h"], (x.double() + res.double()).to(torch.bfloat16))
    v, _ = block.rms_norm(_np(out["h"]), _np(norm), 1e-6)
    _near(out["n"], v, (82 * U + B) * np.abs(v) * 1.001, "n")
    idx, wt, n = out["idx"].cpu().numpy(), _np(out["w"]), _np(out["n"])
    assert (np.sort(idx, 1)[:, 1:] != np.sort(idx, 1)[:, :-1]).all() and (idx >= 0).all() and np.allclose(wt.sum(1), 1, atol=1e-5)
    want = block.experts(n, idx, wt, v1, v2)
    # the bound of test_gpu_experts.py, with every magnitude taken over all of a token's experts
    tol = np.zeros_like(want)
    for t in range(T):
        for j, e in enumerate(idx[t]):
            gu, mag = v1[e] @ n[t], np.abs(v1[e]) @ np.abs(n[t])
            gg, u = gu[:inner], gu[inner:]
            sg, e1 = block.act(gg, "silu"), (H + H / 128 + 8) * U
            da = 1.1 * e1 * mag[:inner] * (np.abs(u) + e1 * mag[inner:]) + np.abs(sg) * e1 * mag[inner:] + (16 + 8 * np.abs(gg)) * U * np.abs(gg * u)
            a = np.abs(sg * u)
            da = da + B * (a + da)
            tol[t] += wt[t, j] * (np.abs(v2[e]) @ da + (inner + inner / 128 + 24 + k) * U * (np.abs(v2[e]) @ (a + da)))
    _near(out["y"], want, tol + B * (np.abs(want) + tol), "y")


def test_few_tokens_and_the_grouped_products_agree():
    # The grouped path quantises tokens and inner activations to e2m1, `few` keeps them bf16.  Half a step is at most 2^-2 of an
    # element, evenly spread over a step at most r = 2^-2 / sqrt(3) = 0.144 of the norm.  The tokens' error enters the gate and the
    # up projection, the inner activations' the down projection: of a = silu(g) u, the gate's is r |g silu'(g)| / |silu(g)| in the
    # norm, over g normal sqrt(0.517 / 0.356) r = 1.206 r, the up projection's r, the inner rounding's r; as squares
    # r sqrt(1.454 + 1 + 1) = 0.268.
    layer_of = _example("moe_layer")
    g = torch.Generator(device=DEV).manual_seed(0)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    E, H, inner, k, T = 16, 512, 256, 4, 64
    layer = layer_of.MoELayer(r(E, H) / H**0.5, r(E, 2 * inner, H) / H**0.5, r(E, H, inner) / inner**0.5, k)
    x = r(T, H).to(torch.bfloat16)
    few, decode = layer.few(x), layer.decode(x, 64)
    assert torch.equal(few["idx"], decode["idx"]) and torch.equal(few["w"], decode["w"])
    assert (few["y"].double() - decode["y"].double()).norm() <= 0.268 * few["y"].double().norm()


def test_the_examples_run(capsys):
    _example("ffn_block").main()
    _example("moe_layer").main()
    text = capsys.readouterr().out
    assert "training step" in text and "decode step" in text and "few tokens" in text and "nan" not in text
