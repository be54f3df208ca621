"""The experts of a mixture-of-experts layer for a few tokens on the GPU against the 64-bit oracle.

Bounds (u = 2^-24, b = 2^-8 bf16's half step).  gate and up: fp32 sums of H products of values that bf16 holds exactly, at most
H + H / 128 + 8 roundings of partial sums: e1 = (H + H / 128 + 8) u of the sum of the magnitudes, m1.  (The matrix cores'
own order inside a product adds no more than a rounding per term.)  silu has a slope of at most 1.1 and its own error of
(16 + 8 |g|) u: the inner activation a = silu(g) up is off by da = 1.1 e1(g) |up| + |silu(g)| e1(up) + (16 + 8 |g|) u |g up|, and its
rounding b |a|.  y: the sum over choices of |w| (sum |W2| (da + b |a|) + (I + I / 128 + 8 + k + 16) u sum |W2 a|), and b |y|."""

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_matmul_amd import dg
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, B = 2.0**-24, 2.0**-8


def _weights(fmt, G, N, K, seed):
    """Codes and scales on the device from the library's quantisers, and the values they stand for."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randn(G, N, K, device=DEV, generator=g) / K**0.5
    if fmt == "fp8":
        q, s = torch.empty(G, N, K, dtype=torch.uint8, device=DEV), torch.empty(G, N // 128, K // 128, device=DEV)
        dg.dg_quant_128x128(w, q, s)
        sn = s.double().cpu().numpy()
        return q, s, oracle.decode_e4m3(q.cpu().numpy()) * np.repeat(np.repeat(sn, 128, 1), 128, 2)
    q, s = torch.empty(G, N, K // 2, dtype=torch.uint8, device=DEV), torch.empty(G, K // 128, N, dtype=torch.int32, device=DEV)
    dg.dg_quant_mxfp4(w, q, s)
    v = torch.empty(G, N, K, device=DEV)
    dg.dg_dequant_mxfp4(q, s, v)
    return q, s, v.double().cpu().numpy()


def _layer(fmt, G, H, inner, seed=0):
    q1, s1, v1 = _weights(fmt, G, 2 * inner, H, seed + 1)
    q2, s2, v2 = _weights(fmt, G, H, inner, seed + 2)
    return dict(fmt=fmt, args=(q1, s1, q2, s2), v1=v1, v2=v2, H=H, I=inner, G=G)


def _ws(n, H, inner):
    return torch.zeros(dg.dg_get_workspace_size(dg.DG_OP_MOE_EXPERTS, n, H, inner), dtype=torch.uint8, device=DEV)


def _run(L, x, idx, w, first=0, ws=None, y=None, stream=None):
    y = torch.full_like(x, 7.0) if y is None else y
    ws = _ws(idx.numel(), L["H"], L["I"]) if ws is None else ws
    call = dg.dg_moe_experts_fp8 if L["fmt"] == "fp8" else dg.dg_moe_experts_mxfp4
    q1, s1, q2, s2 = L["args"]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())  # y and ws are filled there
    call(x, idx, w, q1, s1, q2, s2, y, first_expert=first, workspace=ws, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    assert not ws[:4096].any()  # counters back at zero
    return y


def _check(L, x, idx, w, first=0, **kw):
    y = _run(L, x, idx, w, first, **kw)
    xn, idn, wn = x.double().cpu().numpy(), idx.cpu().numpy(), w.double().cpu().numpy()
    H, inner, k = L["H"], L["I"], idn.shape[1]
    want, tol = np.zeros_like(xn), np.zeros_like(xn)
    e1, e2 = (H + H / 128 + 8) * U, (inner + inner / 128 + 24 + k) * U
    for t in range(xn.shape[0]):
        for j, e in enumerate(idn[t] - first):
            if not 0 <= e < L["G"]:
                continue
            v1, v2 = L["v1"][e], L["v2"][e]
            gu, mag = v1 @ xn[t], np.abs(v1) @ np.abs(xn[t])
            g, u, mg, mu = gu[:inner], gu[inner:], mag[:inner], mag[inner:]
            sg = block.act(g, "silu")
            a = sg * u
            da = 1.1 * e1 * mg * (np.abs(u) + e1 * mu) + np.abs(sg) * e1 * mu + (16 + 8 * np.abs(g)) * U * np.abs(g * u)
            da = da + B * (np.abs(a) + da)
            want[t] += wn[t, j] * (v2 @ a)
            tol[t] += abs(wn[t, j]) * (np.abs(v2) @ da + e2 * (np.abs(v2) @ (np.abs(a) + da)))
    got = y.double().cpu().numpy()
    tol = tol + B * (np.abs(want) + tol)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-30))))
    return y


def _tokens(T, k, E, H, seed=0, drop=0.1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    top = torch.topk(torch.randn(T, E, device=DEV, generator=g), k, dim=1)
    idx = torch.where(torch.rand(T, k, device=DEV, generator=g) < drop, -1, top.indices).int()
    return x, idx, torch.softmax(top.values, 1)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,k,E,first,G,H,inner", [
    (1, 1, 1, 0, 1, 128, 128), (1, 4, 16, 0, 16, 1024, 512), (1, 8, 32, 16, 8, 384, 256), (2, 2, 8, 0, 8, 256, 1152), (5, 3, 60, 7, 17, 640, 384),
    (16, 8, 64, 0, 64, 512, 128), (17, 2, 4, 1, 2, 896, 640), (33, 6, 8, 0, 8, 256, 256), (64, 2, 8, 0, 8, 512, 384), (64, 16, 16, 0, 16, 256, 128),
    (64, 1, 2, 0, 2, 128, 512), (64, 8, 256, 64, 32, 384, 256), (3, 5, 300, 0, 300, 256, 128)])
def test_experts(T, k, E, first, G, H, inner, fmt):
    L = _layer(fmt, G, H, inner)
    x, idx, w = _tokens(T, k, E, H)
    _check(L, x, idx, w, first)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,k,H,inner", [(1, 2, 7168, 256), (4, 2, 256, 2048), (2, 2, 16384, 128), (2, 1, 128, 16384)])
def test_long_rows(T, k, H, inner, fmt):
    L = _layer(fmt, 3, H, inner)
    x, idx, w = _tokens(T, k, 3, H, drop=0)
    _check(L, x, idx, w)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_the_longest_rows(fmt):
    x, idx, w = _tokens(2, 1, 1, 32768, drop=0)
    _check(_layer(fmt, 1, 32768, 128), x, idx, w)
    x, idx, w = _tokens(2, 1, 1, 128, drop=0)
    _check(_layer(fmt, 1, 128, 32768), x, idx, w)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_choices_of_every_kind(fmt):
    H, inner, G = 256, 256, 4
    L = _layer(fmt, G, H, inner)
    x, _, _ = _tokens(64, 4, 4, H)
    w = torch.rand(64, 4, device=DEV) - 0.3
    one = torch.full((64, 4), -1, dtype=torch.int32, device=DEV)
    assert (_check(L, x, one, w) == 0).all()  # nobody chose anything
    one[5, 2] = 3
    y = _check(L, x, one, w)
    assert (y[:5] == 0).all() and (y[6:] == 0).all() and y[5].abs().max() > 0
    one[:] = 2  # one expert, four times a token, by everybody
    _check(L, x, one, w)
    far = torch.tensor([-2**31, 2**31 - 1, 4, 9], dtype=torch.int32, device=DEV).repeat(64, 1)
    _check(L, x, far, w)
    _check(L, x, far, w, first=9)
    _check(L, x, far, w, first=2**31 - 1 - 4)
    mixed = torch.randint(-1, 6, (64, 4), dtype=torch.int32, device=DEV)  # repeats, others' experts
    _check(L, x, mixed, w)
    _check(L, x[:1].contiguous(), mixed[:1].contiguous(), w[:1].contiguous())


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_nan_stays_with_its_token_and_expert(fmt):
    H, inner, G, T = 256, 128, 4, 6
    L = _layer(fmt, G, H, inner)
    x, idx, w = _tokens(T, 2, G, H, drop=0)
    idx[:] = torch.tensor([[0, 1], [1, 2], [2, 3], [0, 2], [2, 0], [1, 0]], device=DEV)
    clean = _run(L, x, idx, w)
    q1, s1, q2, s2 = (t.clone() for t in L["args"])
    if fmt == "fp8":
        q1[3, 5, 7] = 0x7F
    else:
        s1[3, 0, 5] = -1
    bad = _run(dict(L, args=(q1, s1, q2, s2)), x, idx, w)
    assert bad[2].isnan().all() and torch.equal(bad[[0, 1, 3, 4, 5]], clean[[0, 1, 3, 4, 5]])
    x2 = x.clone()
    x2[4, 9] = float("nan")
    bad = _run(L, x2, idx, w)
    assert bad[4].isnan().all() and torch.equal(bad[[0, 1, 2, 3, 5]], clean[[0, 1, 2, 3, 5]])
    w2 = w.clone()
    w2[0, 1] = float("inf")
    bad = _run(L, x, idx, w2)
    assert bad[0].isinf().all() and torch.equal(bad[1:], clean[1:])


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_order_of_the_tokens(fmt):
    # a token's result is the same at whichever place of a batch, and so in whichever column of the products
    H, inner, G = 512, 640, 4
    L = _layer(fmt, G, H, inner)
    for k in (1, 3):  # experts of one to four groups of 16 tokens
        x, idx, w = _tokens(64, k, G, H)
        y = _run(L, x, idx, w)
        for _ in range(5):
            perm = torch.randperm(64, device=DEV)
            assert torch.equal(y[perm], _run(L, x[perm].contiguous(), idx[perm].contiguous(), w[perm].contiguous()))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_in_place_streams_and_shared_workspace(fmt):
    H, inner, G = 512, 256, 8
    L = _layer(fmt, G, H, inner)
    x, idx, w = _tokens(20, 4, G, H)
    want = _run(L, x, idx, w)
    over = x.clone()
    assert torch.equal(_run(L, over, idx, w, y=over), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(L, x, idx, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    ws = _ws(64 * 16, H, inner)  # of a larger call, used by others between
    T, E, k = 20, 8, 4
    logits = torch.randn(T, E, device=DEV)
    gi, gw = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    for _ in range(3):
        dg.dg_moe_gate(logits, gi, gw, torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV), torch.empty(1, device=DEV), workspace=ws)
        assert torch.equal(_run(L, x, idx, w, ws=ws), want)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_graph_replays(fmt):
    H, inner, G, T, k = 512, 256, 16, 9, 4
    L = _layer(fmt, G, H, inner)
    x, idx, w = _tokens(T, k, G, H)
    ws, y = _ws(T * k, H, inner), torch.empty_like(x)
    _run(L, x, idx, w, ws=ws, y=y)
    call = dg.dg_moe_experts_fp8 if fmt == "fp8" else dg.dg_moe_experts_mxfp4
    q1, s1, q2, s2 = L["args"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, idx, w, q1, s1, q2, s2, y, workspace=ws)
    for i in range(3):
        for a, b in zip((x, idx, w), _tokens(T, k, G, H, seed=i + 5)):
            a.copy_(b)
        want = _run(L, x, idx, w)
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        assert torch.equal(y, want)


def test_many_splits_and_fewer_cus():
    L = _layer("fp8", 16, 128, 2048)  # eight column tiles: several workgroups share each
    x, idx, w = _tokens(40, 8, 16, 128)
    y = _check(L, x, idx, w)
    try:
        dg.dg_set_num_cus(16)
        _check(L, x, idx, w)
    finally:
        dg.dg_set_num_cus(0)
    assert torch.equal(y, _run(L, x, idx, w))


def test_binding_refusals():
    L = _layer("fp8", 2, 256, 128)
    x, idx, w = _tokens(3, 2, 2, 256)
    q1, s1, q2, s2 = L["args"]
    y, ws = torch.empty_like(x), _ws(6, 256, 128)
    with pytest.raises(ValueError, match="s1"):
        dg.dg_moe_experts_fp8(x, idx, w, q1, s1[:, :1].contiguous(), q2, s2, y, workspace=ws)
    with pytest.raises(TypeError, match="topk_idx"):
        dg.dg_moe_experts_fp8(x, idx.long(), w, q1, s1, q2, s2, y, workspace=ws)
    with pytest.raises(ValueError, match="w2"):
        dg.dg_moe_experts_mxfp4(x, idx, w, torch.zeros(2, 256, 128, dtype=torch.uint8, device=DEV), torch.zeros(2, 2, 256, dtype=torch.int32, device=DEV),
                                q2, torch.zeros(2, 1, 256, dtype=torch.int32, device=DEV), y, workspace=ws)
    with pytest.raises(dg.DGError, match="workspace"):
        dg.dg_moe_experts_fp8(x, idx, w, q1, s1, q2, s2, y)
    with pytest.raises(dg.DGError, match="T must be"):
        many = torch.empty(65, 256, dtype=torch.bfloat16, device=DEV)
        dg.dg_moe_experts_fp8(many, torch.zeros(65, 2, dtype=torch.int32, device=DEV), torch.ones(65, 2, device=DEV), q1, s1, q2, s2, many, workspace=ws)
