"""The 4-bit head's product on the GPU for rows of x of any magnitude in each of its kernels (up to 8
rows whole and in slices of the columns, 9 to 64 rows whole and in slices), and its sequences
of kernels in a captured graph."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O
from test_gpu_head4 import bf, f64, weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def reference(x, w, group, bias=0.0, residual=0.0, act="none"):
    """(y, tolerance): sums in 32 bits, a step of 2^-22 of the magnitudes for each instruction, group,
    warp and slice that they go through, x within 2^-40 of its row's largest, an activation of slope
    1.13 at most within 2^-20, one rounding to bf16, half a step of its smallest number where y is
    below its normal range."""
    K = x.shape[1]
    z, size = x @ w.T + bias, np.abs(x) @ np.abs(w).T + np.abs(bias)
    steps = group // 16 + -(-K // group) + 16 + -(-K // 128)
    lost = 2.0 ** -40 * np.abs(x).max(1, initial=0)[:, None] * np.abs(w).sum(1)[None]
    y = O.act(z, act)
    err = 1.2 * (steps * 2.0 ** -22 * size + lost) + 2.0 ** -20 * np.abs(y)
    return y + residual, err + 2.0 ** -8 * (np.abs(y + residual) + err) + 2.0 ** -134


SHAPES = [(100, 520, 64), (64, 14400, 128), (40, 2880, 32)]


@pytest.mark.parametrize("N,K,group", SHAPES)
@pytest.mark.parametrize("M", [1, 6, 8, 9, 12, 40, 64])
@pytest.mark.parametrize("scale", [1e-37, 1e-12, 1.0, 1e20, 1e35])
def test_rows_of_any_size(M, scale, N, K, group):
    """Rows of one magnitude each, over 60 binades, of a single value, and of zeros."""
    rng = np.random.default_rng(M + K)
    w, ref_w = weight(rng, N, K, group, 1)
    x = rng.normal(size=(M, K)) * scale
    x *= 2.0 ** rng.integers(-12, 1, (M, 1))
    for m in range(M):
        if m % 5 == 1:
            x[m] *= 2.0 ** rng.integers(-60, 0, K)
        elif m % 5 == 2:
            x[m, 3:] = 0
        elif m % 5 == 3:
            x[m] = 0
    x = bf(x)
    y, ws = sv.spec_head4_forward(x, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    want, tol = reference(f64(x), ref_w, group)
    off = np.abs(f64(y) - want) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    assert bool((y[3::5] == 0).all())


@pytest.mark.parametrize("M", [1, 3, 8, 12, 40])
@pytest.mark.parametrize("power", [20, 28, 60])
def test_slices_of_different_magnitudes(M, power):
    """Columns whose magnitude rises or falls by 2^power from one end of a row to the other: each slice
    has a largest value of its own."""
    rng = np.random.default_rng(M + power)
    N, K, group = 64, 14400, 128
    w, ref_w = weight(rng, N, K, group, 1)
    step = np.floor(np.linspace(-power, 0, K))
    x = rng.normal(size=(M, K))
    x[0::2] *= 2.0 ** step
    x[1::2] *= 2.0 ** step[::-1]
    x = bf(x)
    y, ws = sv.spec_head4_forward(x, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    want, tol = reference(f64(x), ref_w, group)
    assert (np.abs(f64(y) - want) <= tol).all()


@pytest.mark.parametrize("M", [1, 8, 32])
def test_an_infinity_in_one_slice(M):
    rng = np.random.default_rng(5)
    w, ref_w = weight(rng, 50, 14400, 64, 1)
    x = bf(rng.normal(size=(M, 14400)))
    clean, _ = sv.spec_head4_forward(x, w)
    for value in (float("inf"), float("nan")):
        x[0, 14000] = value
        y, _ = sv.spec_head4_forward(x, w)
        on = torch.tensor(ref_w[:, 14000] != 0, device=DEV)
        assert bool((~torch.isfinite(y[0][on])).all()) and torch.equal(y[1:], clean[1:])


@pytest.mark.parametrize("M,N,K,group", [(32, 2880, 2880, 32), (12, 400, 4096, 64), (64, 5000, 300, 128),
                                         (8, 64, 14400, 128), (1, 4096, 4096, 128)])
def test_sequences_of_kernels_in_a_graph(M, N, K, group):
    """x's conversion, the product and the join, each begun before the one before it has ended, replayed
    one behind the other with new x."""
    rng = np.random.default_rng(M)
    w, ref_w = weight(rng, N, K, group, 1)
    b, r = rng.normal(size=N), rng.normal(size=(M, N))
    b, r = bf(b), bf(r)
    x, y = torch.empty(M, K, dtype=BF16, device=DEV), torch.empty(M, N, dtype=BF16, device=DEV)
    ws = torch.empty(sv.spec_head4_forward_workspace(M, N, K), dtype=torch.uint8, device=DEV)
    call = lambda: sv.spec_head4_forward(x, w, b, r, act=sv.SPEC_ACT_SILU, out=y, workspace=ws)   # noqa: E731
    x.copy_(bf(rng.normal(size=(M, K))))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    inputs = [bf(rng.normal(size=(M, K)) * 4.0 ** k) for k in (-3, 0, 2)]
    outputs = []
    for k in range(6):          # without a wait between
        x.copy_(inputs[k % 3])
        graph.replay()
        outputs.append(y.clone())
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    for k in range(6):
        want, tol = reference(f64(inputs[k % 3]), ref_w, group, f64(b), f64(r), "silu")
        assert (np.abs(f64(outputs[k]) - want) <= tol).all(), k
        x.copy_(inputs[k % 3])
        call()
        assert torch.equal(y, outputs[k])
