"""A mixture-of-experts layer on the library's operators, for serving and for training.

Serving (`MoELayer`): the experts' weights in microscaled 4-bit floats.
  router -> dg_moe_gate -> dg_moe_layout_{contiguous,masked} -> dg_quant_mxfp4 (tokens gathered into expert rows)
  -> grouped product (gate and up projection) -> SiLU(gate) * up -> dg_quant_mxfp4 -> grouped product (down) -> dg_moe_combine
`prefill` uses the contiguous form, `decode` the masked one (a fixed launch shape, for graph capture).

Training (`train_step`): one expert projection in block-scaled FP8 between the router and the combine, with the gradients
of the router's logits and of the expert rows.

    python examples/moe_layer.py            # both, at small sizes; prints what they agree to
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_grouped_matmul_amd import dg  # noqa: E402


def _i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def _workspace(op, *size):
    return torch.zeros(max(16, dg.dg_get_workspace_size(op, *size)), dtype=torch.uint8, device="cuda")


def quantise(x, row_token=None):
    """Codes and scale words of rows of x (gathered by row_token); rows without a token stay zero."""
    lead = tuple(x.shape[:-1]) if row_token is None else tuple(row_token.shape)
    K = x.shape[-1]
    q = torch.zeros(lead + (K // 2,), dtype=torch.uint8, device="cuda")
    sf = torch.zeros(lead[:-1] + (K // 128, lead[-1]), dtype=torch.int32, device="cuda")
    dg.dg_quant_mxfp4(x, q, sf, row_token=row_token)
    return q, sf


class MoELayer:
    """E experts of hidden size H and inner size I, k of them per token."""

    def __init__(self, router, w_gate_up, w_down, k):
        """router [E,H] fp32; w_gate_up [E,2I,H] and w_down [E,H,I] fp32, quantised once here."""
        self.router, self.k = router, k
        self.E, self.H, self.I = router.shape[0], router.shape[1], w_down.shape[2]
        self.gate_up = quantise(w_gate_up)
        self.down = quantise(w_down)

    def route(self, x):
        T = x.shape[0]
        logits = x.float() @ self.router.t()
        idx, w = _i32(T, self.k), torch.empty(T, self.k, device="cuda")
        counts, load, loss = _i32(self.E + 1), torch.empty(self.E, device="cuda"), torch.empty(1, device="cuda")
        dg.dg_moe_gate(logits, idx, w, counts, load, loss, workspace=_workspace(dg.DG_OP_MOE_GATE, T, self.E, self.k))
        return idx, w

    def _experts(self, x, row_token, product):
        """Rows of the experts' outputs; `product(A, sfa, B, sfb, D)` is the grouped form."""
        lead = tuple(row_token.shape)
        a, sa = quantise(x, row_token)
        gu = torch.zeros(lead + (2 * self.I,), dtype=torch.bfloat16, device="cuda")
        product(a, sa, *self.gate_up, gu)
        h = (torch.nn.functional.silu(gu[..., : self.I].float()) * gu[..., self.I:].float()).to(torch.bfloat16)
        q, sq = quantise(h)
        d = torch.zeros(lead + (self.H,), dtype=torch.bfloat16, device="cuda")
        product(q, sq, *self.down, d)
        return {"gate_up": gu, "h": h, "rows": d}

    def prefill(self, x):
        """x [T,H] bf16 -> y [T,H] bf16, the experts' rows in the contiguous layout."""
        T, ws = x.shape[0], _workspace(dg.DG_OP_MOE_LAYOUT, x.shape[0], 0, self.k, self.E)
        idx, w = self.route(x)
        M = (T * self.k + 127 * self.E + 127) // 128 * 128
        counts, m_indices, row_token, row_of = _i32(self.E), _i32(M), _i32(M), _i32(T, self.k)
        dg.dg_moe_layout_contiguous(idx, counts, m_indices, row_token, row_of, workspace=ws)
        out = self._experts(x, row_token,
                            lambda a, sa, b, sb, d: dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(a, sa, b, sb, d, m_indices))
        y = torch.empty_like(x)
        dg.dg_moe_combine(out["rows"], row_of, w, y)
        return dict(out, y=y, idx=idx, w=w, row_of=row_of, row_token=row_token)

    def decode(self, x, max_m):
        """The same in the masked layout, at most max_m tokens per expert (later ones are dropped)."""
        T, ws = x.shape[0], _workspace(dg.DG_OP_MOE_LAYOUT, x.shape[0], 0, self.k, self.E)
        idx, w = self.route(x)
        masked_m, row_token, row_of = _i32(self.E), _i32(self.E, max_m), _i32(T, self.k)
        dg.dg_moe_layout_masked(idx, masked_m, row_token, row_of, workspace=ws)
        out = self._experts(x, row_token,
                            lambda a, sa, b, sb, d: dg.dg_m_grouped_mxfp4_gemm_nt_masked(a, sa, b, sb, d, masked_m))
        y = torch.empty_like(x)
        dg.dg_moe_combine(out["rows"].reshape(-1, self.H), row_of, w, y)
        return dict(out, y=y, idx=idx, w=w, row_of=row_of, row_token=row_token)


def train_step(x, logits, w8, sw8, dy, k, loss_coef):
    """One FP8 expert projection between router and combine: x [T,H] fp32, logits [T,E], w8/sw8 the experts' weights
    [E,N,H] from dg_quant_128x128, dy [T,N] bf16.  Returns the outputs and the gradients of the logits (through the
    weights and the balance loss), of the expert rows and of the weights."""
    T, H = x.shape
    E, N = w8.shape[:2]
    idx, w = _i32(T, k), torch.empty(T, k, device="cuda")
    counts, load, loss = _i32(E + 1), torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    dg.dg_moe_gate(logits, idx, w, counts, load, loss, loss_coef=loss_coef, workspace=_workspace(dg.DG_OP_MOE_GATE, T, E, k))
    M = (T * k + 127 * E + 127) // 128 * 128
    seg, m_indices, row_token, row_of = _i32(E), _i32(M), _i32(M), _i32(T, k)
    dg.dg_moe_layout_contiguous(idx, seg, m_indices, row_token, row_of, workspace=_workspace(dg.DG_OP_MOE_LAYOUT, T, 0, k, E))
    gathered = x[row_token.clamp(min=0).long()]
    q = torch.empty(M, H, dtype=torch.uint8, device="cuda")
    s = torch.empty(H // 128, M, dtype=torch.float32, device="cuda")
    dg.dg_quant_1x128(gathered, q, s)
    rows = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_fp8_gemm_nt_contiguous(q, s, w8, sw8, rows, m_indices)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(rows, row_of, w, y)
    drows = torch.zeros_like(rows)  # padding rows stay zero, as the K-grouped product of the weights' gradient wants them
    dw = torch.empty_like(w)
    dg.dg_moe_combine_bwd(dy, rows, row_of, w, drows, dw)
    dlogits = torch.empty_like(logits)
    dg.dg_moe_gate_bwd(logits, idx, w, counts, dw, torch.ones(1, device="cuda"), dlogits, loss_coef=loss_coef)
    return {"y": y, "loss": loss, "rows": rows, "row_of": row_of, "idx": idx, "w": w, "drows": drows, "dw": dw, "dlogits": dlogits}


def main():
    torch.manual_seed(0)
    E, H, inner, k, T = 16, 512, 256, 4, 200
    layer = MoELayer(torch.randn(E, H, device="cuda") / math.sqrt(H), torch.randn(E, 2 * inner, H, device="cuda") / math.sqrt(H),
                     torch.randn(E, H, inner, device="cuda") / math.sqrt(inner), k)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    a, b = layer.prefill(x)["y"].float(), layer.decode(x, 128)["y"].float()
    print("prefill against decode: %.2e of the norm" % ((a - b).norm() / a.norm()).item())
    w = torch.randn(E, 256, H, device="cuda") / math.sqrt(H)
    w8 = torch.empty(E, 256, H, dtype=torch.uint8, device="cuda")
    sw8 = torch.empty(E, 2, H // 128, dtype=torch.float32, device="cuda")
    dg.dg_quant_128x128(w, w8, sw8)
    out = train_step(x.float(), torch.randn(T, E, device="cuda"), w8, sw8, torch.randn(T, 256, device="cuda").to(torch.bfloat16), k, 0.01)
    print("training step: balance loss %.5f, |dlogits| %.4f" % (out["loss"].item(), out["dlogits"].norm().item()))


if __name__ == "__main__":
    main()
