"""The head's products on the bounds-checked build: no access of its kernels (other
than by the tensor maps, which bound theirs) leaves the call's buffers, at the sizes
of the other tests, odd ones among them."""
import pytest

import speculative_decoding_rejection_gb300 as sv
import test_gpu_head as H

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def checked():
    sv.use_checked_library(True)
    yield
    sv.use_checked_library(False)


@pytest.mark.parametrize("M,K,N,act,bias,residual", H.FORWARD + [(5, 2196, 6827, "silu", 1, 1)])
def test_forward_checked(M, K, N, act, bias, residual):
    H.test_forward(M, K, N, act, bias, residual)


@pytest.mark.parametrize("M,K,N,act", H.BACKWARD + [(6, 6437, 1803, "gelu"), (1156, 261, 68, "silu")])
def test_backward_checked(M, K, N, act):
    H.test_backward(M, K, N, act)


def test_parts_and_nothing_checked():
    H.test_backward_parts_alone()
    H.test_backward_of_nothing_is_ok()
    H.test_no_rows()
    H.test_residual_in_place()
