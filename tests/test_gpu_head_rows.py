"""spec_head_backward of very many rows: sums of whole numbers, exact in 32 bits."""
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.mark.parametrize("N,act", [(8, "silu"), (9, "none")])
def test_backward_of_more_rows_than_a_grid_is_high(N, act):
    """65535 blocks of 64 rows and more; a few rows are not zero."""
    M, K = 64 * 65535 + 200, 8
    rows = torch.tensor([0, 63, 64, 64 * 65535 - 1, 64 * 65535, M - 1], device=DEV)
    dy, x = torch.zeros(M, N, dtype=BF16, device=DEV), torch.zeros(M, K, dtype=BF16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    dy[rows] = torch.randint(-4, 5, (len(rows), N), generator=g, device=DEV).to(BF16)
    x[rows] = torch.randint(-4, 5, (len(rows), K), generator=g, device=DEV).to(BF16)
    w = torch.randint(-4, 5, (N, K), generator=g, device=DEV).to(BF16)
    pre, code = None, sv.SPEC_ACT_NONE
    slope = 1.0
    if act == "silu":   # a slope of 1/2 where the pre-activation is 0
        pre, code, slope = torch.zeros(M, N, dtype=BF16, device=DEV), sv.SPEC_ACT_SILU, 0.5
    dx, dw, db, ws = sv.spec_head_backward(dy, x, w, pre, act=code, want_db=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    dz = slope * dy.float()
    assert torch.equal(db, dz.sum(0))
    assert torch.equal(dw.float(), (dz.t() @ x.float()).to(BF16).float())
    assert torch.equal(dx.float(), (dz @ w.float()).to(BF16).float())
