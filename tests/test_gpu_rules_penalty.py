"""The repetition penalty of spec_process_logits over the whole range of its factor."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V = 4096


OUTSIDE = [1e-45, 1e-39, 8.6e37, 3e38]


@pytest.mark.parametrize("rho", [2.0 ** -126, 2e-38, 1e-20, 0.3, 1.0, 1.05, 1.3, 7.0, 1e20, 2.0 ** 126] + OUTSIDE)
def test_repetition(rho):
    g = torch.Generator().manual_seed(1)
    z = torch.randn(1, V, generator=g) * torch.exp(3 * torch.randn(1, V, generator=g))
    z *= min(1.0, rho * 1e32, 1e32 / rho)
    r = torch.tensor([rho], dtype=torch.float32)
    assert float(r) > 0
    out, ws = sv.spec_process_logits(
        z.to(DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV), max_rows=1,
        history=torch.arange(V, dtype=torch.int32, device=DEV),
        cu_history=torch.tensor([0, V], dtype=torch.int32, device=DEV), repetition=r.to(DEV),
        prompt_len=torch.tensor([V], dtype=torch.int32, device=DEV))
    if rho in OUTSIDE:   # the reciprocal is no normal number
        assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG
        return
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    x, f = z.numpy()[0], r.numpy()[0]
    # (beyond f32 the result is infinite; magnitudes here stay below)
    x, f = x.astype(np.float64), float(f)
    want = np.where(x > 0, x / f, x * f)
    assert np.all(np.abs(want) < 3e38)
    # the reciprocal's, the quotient's and the product's roundings, or a step of the
    # smallest values
    assert np.all(np.abs(out.cpu().numpy()[0] - want) <= 3 * 2.0 ** -24 * np.abs(want) + 2.0 ** -149)
