"""spec_adamw_step with gradients that are infinite, NaN or whose squares overflow:
what they do to their own weights stays theirs, step after step."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24
H = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
N = 700   # two whole blocks and one that is not


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype,bits", [(torch.float32, 8), (torch.bfloat16, 8), (torch.float32, 32)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan"), 1e25])
def test_neighbours_of_a_bad_gradient_go_on(bad, dtype, bits, shift):
    g = torch.Generator().manual_seed(4)
    at = lambda x: torch.cat([x[:1], x]).to(DEV)[1:] if shift else x.to(DEV)   # noqa: E731
    w = torch.randn(N, generator=g).to(dtype)
    grads = [(0.02 * torch.randn(N, generator=g)).to(dtype) for _ in range(3)]
    hit = torch.tensor([10, 300, 699])
    rest = torch.ones(N, dtype=torch.bool)
    rest[hit] = False

    def run(first):
        """Three steps; the weights, and the states' values."""
        p, grad = at(w.clone()), at(first.clone())
        kind = dict(dtype=torch.uint8 if bits == 8 else torch.float32)
        m, v = at(torch.zeros(N, **kind)), at(torch.zeros(N, **kind))
        scales = [[torch.zeros(3, device=DEV)] if bits == 8 else None for _ in range(2)]
        tb = sv.spec_adamw_table([p], [grad], [m], [v], exp_avg_scale=scales[0], exp_avg_sq_scale=scales[1])
        for t in range(3):
            grad.copy_(first if t == 0 else grads[t])
            assert sv.spec_get_status(sv.spec_adamw_step(tb, t + 1, **H)) == sv.SPEC_OK
        states = [x.view(torch.float8_e4m3fn).float() * s[0].repeat_interleave(256)[:N] if bits == 8 else x
                  for x, s in zip((m, v), scales)]
        return [x.cpu() for x in (p, *states)]

    hurt, gone = grads[0].clone(), grads[0].clone()
    hurt[hit], gone[hit] = bad, 0.0
    got, want = run(hurt), run(gone)
    if np.isfinite(bad):   # its m is finite: a block's largest, beside which 8 bits hold the others as 0
        assert bool(torch.isfinite(got[0][rest]).all()) and torch.equal(got[2][rest], want[2][rest])
    else:
        assert all(torch.equal(x[rest], y[rest]) for x, y in zip(got, want))
        assert not bool(torch.isfinite(got[0][hit]).any())
