"""Masks without rows in spec_process_logits: a row that goes by one is never
left without its mask."""
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V = 100
CU = [0, 2, 3]


def call(**r):
    z = torch.randn(3, V, device=DEV)
    out, ws = sv.spec_process_logits(z, torch.tensor(CU, dtype=torch.int32, device=DEV), max_rows=2, **r)
    return z, out, sv.spec_get_status(ws)


def masks(n):
    return torch.zeros(n, (V + 31) // 32, dtype=torch.int32, device=DEV)


def rows(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n", [0, 2])
def test_fewer_mask_rows_than_rows_are_refused(n):
    with pytest.raises((ValueError, sv.SpecError)):
        call(mask=masks(n))


@pytest.mark.parametrize("checked", [True, False])
@pytest.mark.parametrize("n,which", [(0, (-1, 0, -1)), (0, (5, -1, -1)), (2, (0, 1, 2))])
def test_a_row_of_a_mask_that_is_not_there_is_reported(n, which, checked):
    sv.use_checked_library(checked)
    try:
        assert call(mask=masks(n), mask_rows=rows(*which))[2] == sv.SPEC_ERR_INVALID_ARG
    finally:
        sv.use_checked_library(False)


def test_no_row_goes_by_a_mask():
    z, out, status = call(mask=masks(0), mask_rows=rows(-1, -1, -1))
    assert status == sv.SPEC_OK and torch.equal(z, out)
