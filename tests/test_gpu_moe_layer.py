"""The operators run together (examples/moe_layer.py): each stage of the layer
against the 64-bit oracles on the stage's own inputs, both layouts, a decode
step captured and replayed with new tokens, and the training step's gradients.

Bounds as in the operators' own tests; the second product takes the layer's own
hidden rows, so its bound is a product's."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from moe_grouped_matmul_amd import dg
from oracle import moe, mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24

spec = importlib.util.spec_from_file_location(
    "moe_layer_example", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py"))


@pytest.fixture(scope="module")
def ex():
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


E, H, I, K = 12, 384, 256, 3


@pytest.fixture(scope="module")
def layer(ex):
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(s, device=DEV, generator=g)  # noqa: E731
    w = (r(E, H) / H ** 0.5, r(E, 2 * I, H) / H ** 0.5, r(E, H, I) / I ** 0.5)
    return ex.MoELayer(*w, K), [t.cpu().numpy() for t in w]


def _product(got, a, b):
    """One expert's rows: inputs in fp32 as the oracle quantises them."""
    qa, sa = mxfp4.quant_mxfp4(a)
    qb, sb = mxfp4.quant_mxfp4(b)
    ref, mag = mxfp4.gemm_mxfp4(qa, sa, qb, sb)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + (a.shape[1] / 32 + 2) * U) * mag
    assert np.all(np.abs(got - ref) <= tol)
    assert np.linalg.norm(got - ref) <= 2.0 ** -8 * np.linalg.norm(ref)


@pytest.mark.parametrize("form,T", [("prefill", 1), ("prefill", 300), ("decode", 1), ("decode", 70)])
def test_layer(layer, form, T):
    moe_layer, (router, w1, w2) = layer
    x = torch.randn(T, H, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)).to(torch.bfloat16)
    out = moe_layer.prefill(x) if form == "prefill" else moe_layer.decode(x, 32)
    xs = x.float().cpu().numpy()
    idx, row_token = out["idx"].cpu().numpy(), out["row_token"].cpu().numpy()
    lay = moe.layout(idx, 0, E, rows=row_token.size) if form == "prefill" else moe.layout(idx, 0, E, max_m=32)
    assert np.array_equal(row_token.ravel(), lay["row_token"]) and np.array_equal(out["row_of"].cpu().numpy(), lay["row_of"])
    f = {n: out[n].double().cpu().numpy().reshape(row_token.size, -1) for n in ("gate_up", "h", "rows")}
    for e in range(E):
        at = np.nonzero((lay["m_indices"] == e) & (lay["row_token"] >= 0))[0]
        if len(at):
            _product(f["gate_up"][at], xs[lay["row_token"][at]], w1[e])
            _product(f["rows"][at], f["h"][at].astype(np.float32), w2[e])
    want, mag = moe.combine(f["rows"], lay["row_of"], out["w"].double().cpu().numpy())
    assert np.all(np.abs(out["y"].double().cpu().numpy() - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + (K + 1) * U * mag)


def test_decode_operators_in_a_graph(layer):
    """Router to combine captured once, replayed on new logits and tokens, eager work between the replays."""
    moe_layer, _ = layer
    T, max_m = 16, 16
    i32 = dict(dtype=torch.int32, device=DEV)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    logits = torch.zeros(T, E, device=DEV)
    idx, w, counts = torch.empty(T, K, **i32), torch.empty(T, K, device=DEV), torch.empty(E + 1, **i32)
    load, loss = torch.empty(E, device=DEV), torch.empty(1, device=DEV)
    mm, rt, ro = torch.empty(E, **i32), torch.empty(E, max_m, **i32), torch.empty(T, K, **i32)
    q, s = torch.zeros(E, max_m, H // 2, dtype=torch.uint8, device=DEV), torch.zeros(E, H // 128, max_m, **i32)
    d, y = torch.zeros(E, max_m, 2 * I, dtype=torch.bfloat16, device=DEV), torch.empty(T, 2 * I, dtype=torch.bfloat16, device=DEV)
    wg = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, T, E, K), dtype=torch.uint8, device=DEV)
    wl = torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_LAYOUT, T, 0, K, E), dtype=torch.uint8, device=DEV)

    def step():
        dg.dg_moe_gate(logits, idx, w, counts, load, loss, loss_coef=0.1, workspace=wg)
        dg.dg_moe_layout_masked(idx, mm, rt, ro, workspace=wl)
        dg.dg_quant_mxfp4(x, q, s, row_token=rt)
        dg.dg_m_grouped_mxfp4_gemm_nt_masked(q, s, *moe_layer.gate_up, d, mm)
        dg.dg_moe_combine(d.reshape(-1, 2 * I), ro, w, y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    outs = (idx, w, counts, load, loss, mm, rt, ro, y)
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(T, H, device=DEV, generator=g))
        logits.copy_(torch.randn(T, E, device=DEV, generator=g) * (1 + seed))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, outs))


def test_training_step(ex):
    g = torch.Generator(device=DEV).manual_seed(2)
    T, N, coef = 150, 272, 0.05
    r = lambda *s: torch.randn(s, device=DEV, generator=g)  # noqa: E731
    x, logits, wt, dy = r(T, H), 2 * r(T, E), r(E, N, H) / H ** 0.5, r(T, N).to(torch.bfloat16)
    w8 = torch.empty(E, N, H, dtype=torch.uint8, device=DEV)
    sw8 = torch.empty(E, (N + 127) // 128, H // 128, dtype=torch.float32, device=DEV)
    dg.dg_quant_128x128(wt, w8, sw8)
    out = ex.train_step(x, logits, w8, sw8, dy, K, coef)
    n = {k: v.double().cpu().numpy() for k, v in out.items()}
    gate = moe.gate(logits.double().cpu().numpy(), K, loss_coef=coef)
    assert np.array_equal(n["idx"], gate["topk_idx"])
    row_of = out["row_of"].cpu().numpy()
    want, mag = moe.combine(n["rows"], row_of, n["w"])
    assert np.all(np.abs(n["y"] - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + (K + 1) * U * mag)
    drows, dw, dmag = moe.combine_grad(dy.double().cpu().numpy(), n["rows"], row_of, n["w"])
    drows = np.nan_to_num(drows)  # padding rows are zero
    assert np.all(np.abs(n["drows"] - drows) <= (2.0 ** -8 * 1.01 + U) * np.abs(drows))
    assert np.all(np.abs(n["dw"] - dw) <= (N / 256 + 20) * U * dmag)
    d, m = moe.gate_grad(gate, n["dw"], 1.0, loss_coef=coef)
    spread = float((logits.max(1, keepdim=True).values - logits).max())
    assert np.all(np.abs(n["dlogits"] - d) <= 1.01 * U * np.abs(d) + (4 * spread + 100) * U * m + 1e-37)
    assert abs(n["loss"][0] - gate["loss"]) <= 2000 * U * abs(gate["loss"])
