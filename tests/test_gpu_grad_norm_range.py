"""The gradients' norm on the GPU at magnitudes where a thread's sums, the root or the scaled norm
leave 32 bits, against the 64-bit reference."""
import math

import pytest
import torch

import speculative_decoding_rejection_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
# chains of eight squares and a tree of two (ten roundings, half of them in the root), sums of
# those in two words, one rounding of the norm
TOL = 6 * 2.0 ** -24


def table_of(grads):
    n = [g.numel() for g in grads]
    return sv.spec_adamw_table([torch.zeros_like(g) for g in grads], grads,
                               *[[torch.zeros(k, device=DEV) for k in n] for _ in range(2)])


def norm_of(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check_norm_and_clip(grads):
    norm = norm_of(grads)
    out, ws = sv.spec_grad_norm(table_of(grads), max_norm=0.25 * norm)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    assert abs(float(out[0]) - norm) <= TOL * norm, (float(out[0]), norm)
    assert abs(float(out[1]) - 0.25) <= 2 * TOL
    keep = [g.clone() for g in grads]
    out, ws = sv.spec_clip_grads(table_of(grads), max_norm=0.25 * norm)
    assert sv.spec_get_status(ws) == sv.SPEC_OK and abs(float(out[1]) - 0.25) <= 2 * TOL
    for g, k in zip(grads, keep):
        assert torch.equal(g, (k.float() * out[1]).to(g.dtype))


@pytest.mark.parametrize("where", [(0, 1024), (3, 1027, 2047), (5,)])
def test_two_large_gradients_of_a_thread(where):
    """Squares of 2.25e38 each are f32 numbers, two of them are not: elements 1024 apart of a tensor of
    2048 are one thread's."""
    g = torch.zeros(2048, device=DEV)
    g[list(where)] = 1.5e19
    check_norm_and_clip([g])
    check_norm_and_clip([g.fill_(1.5e19)])


@pytest.mark.parametrize("dtype,n,scale", [(F32, 12_000_001, 1e18), (F32, 12_000_001, 4e18), (F32, 12_000_001, 1e16),
                                           (BF16, 20_000_003, 2e18), (BF16, 20_000_003, 3e17)])
def test_many_large_gradients(dtype, n, scale):
    """Several items of every CTA: a thread adds many sums that f32 holds one by one."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    flat = torch.empty(n, device=DEV).normal_(generator=gen)
    check_norm_and_clip([(flat * scale).to(dtype), torch.full((77,), 3.0, dtype=dtype, device=DEV)])


def test_a_large_gradient_among_ordinary_ones():
    g = torch.randn(3_000_000, device=DEV)
    for at, v in ((0, 1.5e19), (1, -1.2e19), (2_999_999, 3e38)):
        g[at] = v
        check_norm_and_clip([g.clone()])
