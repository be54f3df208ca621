"""A transformer's pre-norm feed-forward block on the library's operators.

Training (`DenseBlock`): y = h + gelu(n(h) W1^T + b1) W2^T + b2, h = x + residual, the products in block-scaled FP8.
  dg_rms_norm (residual added, operand quantised) -> dg_fp8_gemm_nt_epilogue (bias, gelu) -> dg_quant_1x128
  -> dg_fp8_gemm_nt_epilogue (bias, residual)
  backward: dg_epilogue_bwd (bias, operand) -> dg_fp8_gemm_nt -> dg_epilogue_bwd (gelu, bias, operand) -> dg_fp8_gemm_nt
  -> dg_rms_norm_bwd; the weights' gradients are products over the tokens of transposed, requantised operands
  (dg_k_grouped_fp8_gemm_nt_contiguous, whose operands both have row scales).
Serving (`moe_decode`): a decode step of a few tokens through a mixture-of-experts layer.
  dg_rms_norm -> router -> dg_moe_gate -> dg_moe_experts_mxfp4

    python examples/ffn_block.py            # both, at small sizes
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_grouped_matmul_amd import dg  # noqa: E402


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _workspace(op, *size):
    return torch.zeros(max(16, dg.dg_get_workspace_size(op, *size)), dtype=torch.uint8, device="cuda")


def _weight(w):
    """w [N,K] fp32 -> its e4m3 codes and block scales."""
    q, s = _empty(*w.shape, dtype=torch.uint8), _empty((w.shape[0] + 127) // 128, w.shape[1] // 128)
    dg.dg_quant_128x128(w.contiguous(), q, s)
    return q, s


def _rows(x):
    """x [M,K] -> e4m3 codes and row scales."""
    q, s = _empty(*x.shape, dtype=torch.uint8), _empty(x.shape[1] // 128, x.shape[0])
    dg.dg_quant_1x128(x.float().contiguous(), q, s)
    return q, s


def _product(a, b, M, N, K, **epilogue):
    """bf16 [M,N] = act(a . b^T + bias) + residual."""
    d = _empty(M, N, dtype=torch.bfloat16)
    dg.dg_fp8_gemm_nt_epilogue(*a, *b, d, workspace=_workspace(dg.DG_OP_GEMM_NT, M, N, K), **epilogue)
    return d


class DenseBlock:
    def __init__(self, norm, w1, b1, w2, b2):
        """norm [H]; w1 [F,H], b1 [F], w2 [H,F], b2 [H], all fp32.  The weights are quantised once here, and their transposes
        for the backward pass."""
        self.norm, self.b1, self.b2 = norm, b1, b2
        self.F, self.H = w1.shape
        self.w1, self.w2, self.w1t, self.w2t = _weight(w1), _weight(w2), _weight(w1.t()), _weight(w2.t())

    def forward(self, x, residual):
        """x, residual [M,H] bf16 -> y [M,H] bf16 and what the backward pass reads."""
        (M, H), F = x.shape, self.F
        h, rstd = torch.empty_like(x), _empty(M)
        n = (_empty(M, H, dtype=torch.uint8), _empty(H // 128, M))
        dg.dg_rms_norm(x, self.norm, residual=residual, h=h, q=n[0], sf=n[1], rstd=rstd)
        pre = _empty(M, F, dtype=torch.bfloat16)
        a = _product(n, self.w1, M, F, H, bias=self.b1, act="gelu", pre=pre)
        y = _product(_rows(a), self.w2, M, H, F, bias=self.b2, residual=h)
        return y, dict(h=h, rstd=rstd, n=n, pre=pre, a=a)

    def backward(self, dy, kept):
        """dy [M,H] bf16 -> gradients of x (and of the residual), norm, b1, b2, and of the two products' outputs, of which the
        weights' gradients are dz1^T n and dz2^T a."""
        (M, H), F = dy.shape, self.F
        q2, s2, db2 = _empty(M, H, dtype=torch.uint8), _empty(H // 128, M), _empty(H)
        dg.dg_epilogue_bwd(dy, q=q2, sf=s2, dbias=db2, workspace=_workspace(dg.DG_OP_EPILOGUE_BWD, M, H, 0))
        da = _product((q2, s2), self.w2t, M, F, H)
        dz1, q1, s1, db1 = _empty(M, F, dtype=torch.bfloat16), _empty(M, F, dtype=torch.uint8), _empty(F // 128, M), _empty(F)
        dg.dg_epilogue_bwd(da, dz1, pre=kept["pre"], act="gelu", q=q1, sf=s1, dbias=db1, workspace=_workspace(dg.DG_OP_EPILOGUE_BWD, M, F, 0))
        dn = _product((q1, s1), self.w1t, M, H, F)
        dx, dnorm = torch.empty_like(dy), _empty(H)
        dg.dg_rms_norm_bwd(dn, kept["h"], self.norm, kept["rstd"], dx, dnorm, dh=dy, workspace=_workspace(dg.DG_OP_RMS_NORM_BWD, M, 0, H))
        return dict(dx=dx, dnorm=dnorm, db1=db1, db2=db2, dz1=dz1, da=da, dn=dn, q1=(q1, s1), q2=(q2, s2))

    def weight_gradients(self, dy, kept, back):
        """dw1 [F,H] and dw2 [H,F] fp32, for a multiple of 128 tokens: products over the tokens of transposed operands."""
        M = dy.shape[0]
        out = []
        for left, right in ((back["dz1"], self._normed(kept)), (dy, kept["a"])):
            (l, ls), (r, rs) = _rows(left.t()), _rows(right.t())
            d = torch.zeros(1, left.shape[1], right.shape[1], device="cuda")
            dg.dg_k_grouped_fp8_gemm_nt_contiguous(l, ls, r, rs, None, d, torch.tensor([M], dtype=torch.int32, device="cuda"))
            out.append(d[0])
        return out

    def _normed(self, kept):
        y = torch.empty_like(kept["h"])
        dg.dg_rms_norm(kept["h"], self.norm, y=y)
        return y


def moe_decode(x, residual, norm, router, gate_up, down, k):
    """A decode step of T <= 64 tokens: h = x + residual, y = the experts' output for the normed h.  router [E,H] fp32; gate_up
    and down the experts' weights from dg_quant_mxfp4 ([E,2I,H] and [E,H,I]).  Returns h, y and what was chosen."""
    (T, H), E, inner = x.shape, router.shape[0], gate_up[0].shape[1] // 2
    h, n = torch.empty_like(x), torch.empty_like(x)
    dg.dg_rms_norm(x, norm, residual=residual, h=h, y=n)
    logits = n.float() @ router.t()
    idx, w = _empty(T, k, dtype=torch.int32), _empty(T, k)
    ws = _workspace(dg.DG_OP_MOE_GATE, T, E, k)
    dg.dg_moe_gate(logits, idx, w, _empty(E + 1, dtype=torch.int32), _empty(E), _empty(1), workspace=ws)
    y = torch.empty_like(x)
    dg.dg_moe_experts_mxfp4(n, idx, w, *gate_up, *down, y, workspace=_workspace(dg.DG_OP_MOE_EXPERTS, T * k, H, inner))
    return dict(h=h, n=n, y=y, idx=idx, w=w)


def main():
    torch.manual_seed(0)
    M, H, F = 256, 512, 1024
    block = DenseBlock(1 + 0.1 * torch.randn(H, device="cuda"), torch.randn(F, H, device="cuda") / math.sqrt(H), 0.1 * torch.randn(F, device="cuda"),
                       torch.randn(H, F, device="cuda") / math.sqrt(F), 0.1 * torch.randn(H, device="cuda"))
    x, residual, dy = (torch.randn(M, H, device="cuda").to(torch.bfloat16) for _ in range(3))
    y, kept = block.forward(x, residual)
    back = block.backward(dy, kept)
    dw1, dw2 = block.weight_gradients(dy, kept, back)
    print("training step: |y| %.3f |dx| %.3f |dw1| %.3f |dw2| %.3f" % tuple(t.float().norm().item() for t in (y, back["dx"], dw1, dw2)))
    E, inner, T, k = 16, 256, 20, 4

    def experts(*shape):
        w = torch.randn(*shape, device="cuda") / math.sqrt(shape[-1])
        q, s = _empty(*shape[:-1], shape[-1] // 2, dtype=torch.uint8), _empty(shape[0], shape[-1] // 128, shape[1], dtype=torch.int32)
        dg.dg_quant_mxfp4(w, q, s)
        return q, s

    out = moe_decode(x[:T], residual[:T], block.norm, torch.randn(E, H, device="cuda") / math.sqrt(H), experts(E, 2 * inner, H), experts(E, H, inner), k)
    print("decode step: |y| %.3f" % out["y"].float().norm().item())


if __name__ == "__main__":
    main()
