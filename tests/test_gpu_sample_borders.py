"""spec_sample on the GPU where its sums decide: rows of values that go by the histogram, the same
results in every row and every run, and borders far down in a row's tail."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("filters", ["none", "top_p", "top_k"])
@pytest.mark.parametrize("R,V", [(4, 50257), (700, 9001)])
def test_equal_rows_have_equal_results(R, V, filters):
    """One row over and over, by its values' histogram, whose first warps have most of the work and
    whose last ones come late: the same result in every row and call."""
    rng = np.random.default_rng(V)
    z = torch.tensor(2.5 * rng.normal(size=V) - 1.1 * np.log(rng.permutation(V) + 1)).to(BF16).to(DEV)
    z = z.expand(R, V).contiguous()
    law = dict(temperature=torch.full((R,), 0.9, device=DEV))
    if filters == "top_p":
        law["top_p"] = torch.full((R,), 0.93, device=DEV)
    elif filters == "top_k":
        law["top_k"] = torch.full((R,), 4000, dtype=torch.int32, device=DEV)
    u = torch.full((R,), 0.77, device=DEV)
    first = None
    for _ in range(20):
        *got, ws = sv.spec_sample(z, u, want_kept=True, **law)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        got = [t for t in got if t is not None]
        first = first or [t[:1].clone() for t in got]
        for t, f in zip(got, first):
            assert torch.equal(t, f.expand(R))
