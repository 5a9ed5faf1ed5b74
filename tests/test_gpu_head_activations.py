"""Activations of the head's products and their slopes over all magnitudes that
bf16 holds."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
HALF, U32 = 2.0 ** -8, 2.0 ** -24
ACT = {"silu": sv.SPEC_ACT_SILU, "gelu": sv.SPEC_ACT_GELU}


def magnitudes():
    m = torch.tensor([0.0] + [10.0 ** e for e in range(-38, 39)] + [1.5, 5.0, 8.0, 11.0, 20.0, 90.0, 2e13, 3e19, 3.3e38])
    return torch.cat([m, -m]).to(BF16)


def value(z, act):
    """act(z) in 64 bits; GELU by (1 + tanh u) / 2 = 1 / (1 + e^-2u), as 1 + tanh u
    has no digits left at u below -19."""
    if act == "silu":
        return O.act(z, act)
    with np.errstate(over="ignore"):
        return z / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))


@pytest.mark.parametrize("act", ACT)
def test_slopes(act):
    """dz = dy act'(pre) with dy = 1: by db, which sums the one row unrounded."""
    z = magnitudes()
    N = len(z)
    dy, pre = torch.ones(1, N, dtype=BF16, device=DEV), z[None].to(DEV)
    x, w = torch.ones(1, 8, dtype=BF16, device=DEV), torch.ones(N, 8, dtype=BF16, device=DEV)
    _, dw, db, ws = sv.spec_head_backward(dy, x, w, pre, act=ACT[act], want_dx=False, want_db=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    want = O.act_slope(z.double().numpy(), act)
    got = db.double().cpu().numpy()
    # a slope's terms are at most 4 and have 32 roundings; below 2^-126 is 0
    assert np.all(np.abs(got - want) <= 32 * U32 * 4 * np.minimum(1.0, np.abs(want) + (np.abs(z.double().numpy()) < 100))
                  + 2.0 ** -126)
    col = dw.double().cpu().numpy()[:, 0]
    assert np.all(np.abs(col - got) <= HALF * np.abs(got) + 2.0 ** -134)


@pytest.mark.parametrize("act", ACT)
@pytest.mark.parametrize("M", [1, 40])
def test_values(act, M):
    """act(z) with z = x w of one factor, exact."""
    z = magnitudes()
    N = len(z)
    x = torch.zeros(M, 8, dtype=BF16, device=DEV)
    x[:, 0] = 1
    w = torch.zeros(N, 8, dtype=BF16, device=DEV)
    w[:, 0] = z.to(DEV)
    y, pre, ws = sv.spec_head_forward(x, w, act=ACT[act], want_pre=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    assert torch.equal(pre.cpu(), z[None].expand(M, N).contiguous())
    f = z.double().numpy()
    want = value(f, act)
    got = y.double().cpu().numpy()
    # the sigmoid's argument is off by 4 roundings of up to 88 before the value
    # is below 2^-126 z
    rel = 16 * U32 + 4 * U32 * 88
    assert np.all(np.abs(got - want) <= (HALF + rel) * np.abs(want) + 2.0 ** -126 * (1 + np.abs(f)))
