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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,value,scale", [
    (5000, 3e38, 1e-3), (5000, 3e38, 1e-30), (4, 2e38, 2.0 ** -16), (4, 2e38, -2.0 ** -16), (3, 1e38, 1e-38),
    (5000, 1e-38, 2.0 ** 100), (3, 1e-30, 1e-5), (3000, 7e-39, 3e38), (4097, 1.0, 0.37), (2, 0.6, 1e-44)])
def test_a_scale_that_brings_the_norm_into_range(n, value, scale, dtype):
    """The norm of the scaled gradients is held where the norm of the gradients is not, or has lost digits."""
    g = torch.full((n,), value, dtype=dtype, device=DEV)
    g[::2] *= -0.75
    s = torch.tensor([scale], device=DEV)
    norm = abs(float(s)) * norm_of([g])
    tiny = 2.0 ** -148      # two roundings of a norm that is no normal number
    for inf in (False, True):
        want = abs(float(s)) * float(g.double().abs().max()) if inf else norm
        if want > 3.4e38:
            continue
        out, ws = sv.spec_grad_norm(table_of([g]), max_norm=0.5 * want + 2e-38, inf=inf, grad_scale=s)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        factor = float(s) * min(1.0, (0.5 * want + 2e-38) / (want + 1e-6))
        assert abs(float(out[0]) - want) <= TOL * want + tiny, (float(out[0]), want)
        assert abs(float(out[1]) - factor) <= 2 * TOL * abs(factor) + tiny, (float(out[1]), factor)


def test_denormal_gradients_under_a_scale():
    g = torch.full((900,), 1e-42, device=DEV)
    s = torch.tensor([2.0 ** 16], device=DEV)
    norm = 2.0 ** 16 * norm_of([g])
    out, _ = sv.spec_grad_norm(table_of([g]), grad_scale=s)
    assert abs(float(out[0]) - norm) <= TOL * norm and float(out[1]) == 2.0 ** 16
    keep = g.clone()
    out, _ = sv.spec_clip_grads(table_of([g]), max_norm=1.0, grad_scale=s)
    assert float(out[1]) == 2.0 ** 16 and torch.equal(g, keep * 2.0 ** 16)


def test_scales_that_are_no_ordinary_numbers():
    g = torch.full((50,), 2.0, device=DEV)
    big = torch.full((50,), float("inf"), device=DEV)
    for x, s, want in ((g, 0.0, 0.0), (g, -0.0, 0.0), (g, math.inf, math.inf), (g, math.nan, math.nan),
                       (g * 0, math.inf, math.nan), (g * 0, 0.0, 0.0), (big, 0.0, math.nan), (big, 1e-30, math.inf),
                       (g * 1e-38, math.inf, math.inf), (g, -3.0, 6 * math.sqrt(50))):
        for inf in (False, True):
            if inf and math.isfinite(want) and want > 0:
                want = 6.0
            out, ws = sv.spec_grad_norm(table_of([x]), inf=inf, grad_scale=torch.tensor([s], device=DEV))
            assert sv.spec_get_status(ws) == sv.SPEC_OK
            got = float(out[0])
            assert (math.isnan(got) and math.isnan(want)) or got == want or abs(got - want) <= TOL * want, (s, inf, got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-12, 2e-13, 1e-14, 1e-20, 1e-30, 1e-37, 3e-40])
def test_many_small_gradients(scale, dtype):
    """Squares that are no normal numbers of f32, a few hundred thousand of a CTA's threads and more."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    g = (torch.empty(6_000_001, device=DEV).normal_(generator=gen) * scale).to(dtype)
    norm = norm_of([g])
    out, ws = sv.spec_grad_norm(table_of([g]))
    assert sv.spec_get_status(ws) == sv.SPEC_OK and float(out[1]) == 1.0
    assert abs(float(out[0]) - norm) <= TOL * norm + 2.0 ** -149
    # next to ones of every size
    rest = [torch.full((33,), v, dtype=dtype, device=DEV) for v in (0.0, 1e-38, 1e-25, norm, -norm)]
    norm = norm_of([g] + rest)
    out, _ = sv.spec_grad_norm(table_of(rest + [g]))
    assert abs(float(out[0]) - norm) <= TOL * norm + 2.0 ** -149


def test_gradients_of_every_magnitude():
    """Threads that take sums of all three kinds in turn."""
    gen = torch.Generator(device=DEV).manual_seed(6)
    for top in (-60, -20, 0, 40, 62, 70, 126):
        power = torch.randint(-148, top, (4_000_000,), generator=gen, device=DEV)
        power = power.view(-1, 16)[:, :1].expand(-1, 16).reshape(-1)       # alike in a thread's vectors
        g = torch.ldexp(torch.rand(power.numel(), generator=gen, device=DEV, dtype=torch.float64) + 1, power).float()
        if norm_of([g]) < 3e38:
            check_norm_and_clip([g]) if top > 0 else None
            out, _ = sv.spec_grad_norm(table_of([g]))
            assert abs(float(out[0]) - norm_of([g])) <= TOL * norm_of([g])
        else:
            s = torch.tensor([2.0 ** -20], device=DEV)
            out, _ = sv.spec_grad_norm(table_of([g]), grad_scale=s)
            assert abs(float(out[0]) - 2.0 ** -20 * norm_of([g])) <= TOL * 2.0 ** -20 * norm_of([g])


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_an_infinity_among_large_and_small_ones(value):
    for base in (1e-20, 1.0, 1.5e19):
        g = torch.full((3_000_000,), base, device=DEV)
        g[1_234_567] = value
        out, ws = sv.spec_grad_norm(table_of([g]), max_norm=1.0)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        if math.isnan(value):
            assert math.isnan(float(out[0])) and math.isnan(float(out[1]))
        else:
            assert math.isinf(float(out[0])) and float(out[1]) == 0
        g[17] = math.nan
        assert math.isnan(float(sv.spec_grad_norm(table_of([g]))[0][0]))
