"""Gradient of the epilogue for rows of more than 2^28 columns: the bias' gradient is summed in several launches, whose threads
are counted in 32 bits.  Exact: values are small integers, so that every sum is."""

import pytest
import torch

from moe_grouped_matmul_amd import dg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M,N", [(1, 2**28), (2, 2**28 + 2**27 + 16), (3, 2**27 - 16), (3, 2**27 + 16)])
def test_columns_past_a_launch(M, N):
    print(M, N, flush=True)
    col = torch.arange(N, device=DEV, dtype=torch.int32)
    dy, pre = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for r in range(M):
        dy[r] = ((col * (5 + 2 * r) + r) % 61 - 30).to(torch.bfloat16)
        pre[r] = (col + r) % 3 - 1
    want = sum(dy[r].float() * (pre[r] > 0) for r in range(M))
    db = torch.full((N,), 7.0, device=DEV)
    ws = torch.empty(dg.dg_get_workspace_size(dg.DG_OP_EPILOGUE_BWD, M, N, 0), dtype=torch.uint8, device=DEV)
    dg.dg_epilogue_bwd(dy, pre=pre, act="relu", dbias=db, workspace=ws)
    assert torch.equal(db, want)
