"""CPU tests of the 64-bit reference of the draft operators where its own
intermediate values leave the range of 64 bits."""
import numpy as np

from oracle import draft_oracle as O


def test_distill_of_a_draft_that_is_almost_certain():
    """A draft probability below the smallest 64-bit value has a logarithm."""
    for low in (-1e4, -1e9, -3.0e38):
        loss, grad, terms = O.distill(np.zeros((2, 2)), np.array([[0.0, low]]), np.array([0, 1]))
        want = -np.log(2) - 0.5 * low
        assert abs(loss[0] - want) <= 1e-15 * abs(want) * 4 and np.isfinite(terms[0])
        assert np.allclose(grad, [[0.5, -0.5]], atol=0, rtol=1e-15)


def test_distill_of_masked_targets():
    """Masks in the target alone take no part, whatever their value is."""
    t, d = np.array([[1.0, 2.0, 0.0], [0.0, 0.0, 0.0]]), np.array([[0.5, 0.25, 3.0]])
    want = None
    for low in (-np.inf, -3.3e38, -1e9, -1e4):
        t[0, 2] = low
        loss, _, _ = O.distill(t, d, np.array([0, 1]))
        want = loss[0] if want is None else want
        assert loss[0] == want
    for low in (-1e4, -1e9):   # and the draft may then be 0 there
        t[0, 2], d[0, 2] = low, -np.inf
        assert np.isfinite(O.distill(t, d, np.array([0, 1]))[0][0])
    t[0, 2] = -50.0
    assert O.distill(t, d, np.array([0, 1]))[0][0] == np.inf
