"""spec_adamw_step's weight decay at small lr * weight_decay, where 1 - lr *
weight_decay has few digits or none in 32 bits."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N = 1 << 20


def step(w, g, bits, lr_dev, **h):
    """One first step; f32 weights, states of zero. Returns the new weights."""
    kind = dict(dtype=torch.uint8) if bits == 8 else {}
    m, v = torch.zeros(N, device=DEV, **kind), torch.zeros(N, device=DEV, **kind)
    scales = [[torch.zeros(N // 256, device=DEV)] if bits == 8 else None for _ in range(2)]
    p = w.clone()
    tb = sv.spec_adamw_table([p], [g], [m], [v], exp_avg_scale=scales[0], exp_avg_sq_scale=scales[1])
    if lr_dev:
        lr = torch.tensor([h["lr"]], device=DEV)
        ws = sv.spec_adamw_step(tb, 1, lr_dev=lr, **{**h, "lr": 0.5})
    else:
        ws = sv.spec_adamw_step(tb, 1, **h)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    return p.cpu().numpy()


@pytest.mark.parametrize("lr_dev", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr,wd", [(1e-5, 0.01), (3e-6, 0.1), (1e-3, 0.1)])
def test_decay_alone_is_rounded_once(bits, lr_dev, lr, wd):
    """No gradient: w (1 - lr wd), off by half a step of w's and by what lr wd
    itself is off (two roundings of 32 bits)."""
    w = 0.1 * torch.randn(N, generator=torch.Generator().manual_seed(1))
    got = step(w.to(DEV), torch.zeros(N, device=DEV), bits, lr_dev, lr=lr, weight_decay=wd)
    x = w.numpy().astype(np.float64)
    want = x * (1 - lr * wd)
    off = np.abs(got - want)
    assert np.all(off <= np.spacing(np.abs(w.numpy())) / 2 + 4 * 2.0 ** -24 * lr * wd * np.abs(x))


@pytest.mark.parametrize("lr_dev", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_small_decay_beside_updates(bits, lr_dev):
    """lr wd = 2e-8 is a fraction of a step of w's: it shows in the mean change,
    whose rounding errors are even in (-1/2, 1/2) of a step (standard deviation
    0.29) and fall with the root of N; six of them are allowed."""
    g = torch.Generator().manual_seed(2)
    w = 0.5 + 0.49 * torch.rand(N, generator=g)
    grad = 0.02 * torch.randn(N, generator=g)
    # an eps of the size of the gradients spreads the first updates, which would
    # all be +-lr, over (-lr, lr)
    h = dict(lr=1e-5, beta1=0.9, beta2=0.95, eps=1e-2, weight_decay=2e-3)
    got = step(w.to(DEV), grad.to(DEV), bits, lr_dev, **h)
    zero = np.zeros(N)
    want, _, _ = O.adamw(w.numpy(), grad.numpy(), zero, zero, 1, **h)
    ulp = 2.0 ** -24   # a step in [0.5, 1)
    assert abs(np.mean(got - want)) <= 6 * 0.29 * ulp / np.sqrt(N) + 32 * 2.0 ** -24 * h["lr"]
    assert 2e-8 * 0.7 > 4 * (6 * 0.29 * ulp / np.sqrt(N) + 32 * 2.0 ** -24 * h["lr"])   # the decay is seen
