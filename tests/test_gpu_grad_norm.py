"""The norm over the gradients of an optimizer's table and their clipping on the GPU
against the 64-bit reference: ragged, unaligned, empty and mixed tensors, values whose squares
leave 32 bits, infinities, and the step that takes the factor."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
# 32 squares in chains of eight and a tree of two (10 roundings of the sum, half of
# them in the root), sums of those in two words, one rounding of the norm
TOL = 6 * 2.0 ** -24


def table_of(grads, bits=32):
    params = [torch.zeros_like(g) for g in grads]
    n = [g.numel() for g in grads]
    if bits == 8:
        codes = [[torch.zeros(k, dtype=torch.uint8, device=DEV) for k in n] for _ in range(2)]
        scales = [[torch.zeros(-(-k // 256), device=DEV) for k in n] for _ in range(2)]
        return sv.spec_adamw_table(params, grads, *codes, exp_avg_scale=scales[0], exp_avg_sq_scale=scales[1])
    return sv.spec_adamw_table(params, grads, *[[torch.zeros(k, device=DEV) for k in n] for _ in range(2)])


def f64(t):
    return t.double().cpu().numpy()


def make(rng, sizes, dtype="mixed", scale=1.0):
    out = []
    for i, n in enumerate(sizes):
        dt = (BF16, F32)[i % 2] if dtype == "mixed" else dtype
        flat = torch.empty(n + i % 3, dtype=dt, device=DEV)[i % 3:]     # elements off a boundary
        flat.copy_(torch.tensor(rng.normal(size=n) * scale))
        out.append(flat)
    return out


SIZES = [[1], [7], [4096], [4097, 3], [1, 2, 3, 5, 8, 13], [20000, 1, 12289, 4095], [300001],
         [100] * 400, [9000000, 17, 2500001]]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("dtype", ["mixed", F32, BF16])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_factor(sizes, dtype, inf, bits):
    rng = np.random.default_rng(sum(sizes))
    grads = make(rng, sizes, dtype)
    table = table_of(grads, bits)
    keep = [g.clone() for g in grads]
    scale = torch.tensor([0.37], device=DEV)
    for max_norm in (1e-3, 1e9):
        out, ws = sv.spec_grad_norm(table, max_norm=max_norm, inf=inf, grad_scale=scale)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        norm, factor = O.grad_norm([f64(g) for g in grads], max_norm, float(scale), inf)
        got = f64(out)
        assert abs(got[0] - norm) <= TOL * norm and abs(got[1] - factor) <= 2 * TOL * factor
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", ["mixed", F32, BF16])
def test_clip(sizes, dtype):
    rng = np.random.default_rng(sum(sizes) + 1)
    grads = make(rng, sizes, dtype)
    guards = [torch.empty(0, dtype=g.dtype, device=DEV).set_(g.untyped_storage()) for g in grads]
    before = [g.clone() for g in guards]
    keep = [g.clone() for g in grads]
    table = table_of(grads)
    norm = O.grad_norm([f64(g) for g in keep])[0]
    out, ws = sv.spec_clip_grads(table, max_norm=0.5 * norm)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    assert abs(float(out[0]) - norm) <= TOL * norm and abs(float(out[1]) - 0.5 * norm / (norm + 1e-6)) <= TOL
    # by the factor that it reports: one product in 32 bits, one rounding
    for g, k in zip(grads, keep):
        assert torch.equal(g, (k.float() * out[1]).to(g.dtype))
    for i, (a, b) in enumerate(zip(guards, before)):
        bits = torch.int16 if a.dtype is BF16 else torch.int32
        assert torch.equal(a[:i % 3].view(bits), b[:i % 3].view(bits))     # what lies before a tensor
    # the clipped gradients' norm is the bound
    again, _ = sv.spec_grad_norm(table)
    assert abs(float(again[0]) - 0.5 * norm) <= (2.0 ** -8 + TOL) * norm
    # nothing to clip: the bits stay
    keep = [g.clone() for g in grads]
    out, _ = sv.spec_clip_grads(table, max_norm=10 * norm)
    assert float(out[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(grads, keep))
    # a scale alone is applied
    out, _ = sv.spec_clip_grads(table, max_norm=math.inf, grad_scale=torch.tensor([0.25], device=DEV))
    assert float(out[1]) == 0.25 and all(torch.equal(a, (b.float() * 0.25).to(a.dtype)) for a, b in zip(grads, keep))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-30, 1e-25, 1e-18, 1e18, 1e25, 1e32])
def test_squares_that_leave_32_bits(scale, dtype):
    rng = np.random.default_rng(3)
    grads = make(rng, [5000, 4100, 11], dtype, scale)
    out, _ = sv.spec_grad_norm(table_of(grads))
    norm = O.grad_norm([f64(g) for g in grads])[0]
    assert abs(float(out[0]) - norm) <= TOL * norm
    # next to ordinary ones they keep their share
    grads.append(torch.full((3,), 2.0, dtype=dtype, device=DEV))
    out, _ = sv.spec_grad_norm(table_of(grads))
    norm = O.grad_norm([f64(g) for g in grads])[0]
    assert abs(float(out[0]) - norm) <= TOL * norm


def test_zero_gradients():
    for dtype in (F32, BF16):
        g = torch.zeros(70000, dtype=dtype, device=DEV)
        g[::2] = -0.0
        for inf in (False, True):
            out, ws = sv.spec_grad_norm(table_of([g]), max_norm=1.0, inf=inf)
            assert f64(out).tolist() == [0.0, 1.0] and sv.spec_get_status(ws) == sv.SPEC_OK
    g[12345] = 1e-20
    out, _ = sv.spec_grad_norm(table_of([g]))
    assert abs(float(out[0]) / float(g[12345]) - 1) <= TOL


@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [5, 40000])
def test_infinities_and_nan(n, dtype, inf):
    g = torch.randn(n, device=DEV).to(dtype)
    g[n // 2] = -float("inf")
    out, _ = sv.spec_grad_norm(table_of([g]), max_norm=1.0, inf=inf)
    assert math.isinf(float(out[0])) and float(out[1]) == 0
    g[n - 1] = float("nan")
    out, ws = sv.spec_grad_norm(table_of([g]), max_norm=1.0, inf=inf)
    assert math.isnan(float(out[0])) and math.isnan(float(out[1])) and sv.spec_get_status(ws) == sv.SPEC_OK
    out, _ = sv.spec_clip_grads(table_of([g]), max_norm=1.0, inf=inf)
    assert bool(torch.isnan(g).all())


def test_no_elements_and_tables_that_do_not_fit():
    empty = [torch.zeros(0, device=DEV)]
    out, ws = sv.spec_grad_norm(table_of(empty), max_norm=1.0)
    assert f64(out).tolist() == [0.0, 1.0] and sv.spec_get_status(ws) == sv.SPEC_OK
    g = torch.ones(10000, device=DEV)
    table = table_of([torch.zeros(0, device=DEV), g, torch.zeros(0, device=DEV)])
    out, _ = sv.spec_clip_grads(table, max_norm=50.0)
    assert abs(float(out[0]) - 100) <= 100 * TOL and abs(float(g[77]) - 0.5) <= 1e-6
    for change in (dict(n_items=table.n_items + 1), dict(state_bits=8)):
        bad = table_of([g])
        for k, v in change.items():
            setattr(bad, k, v)
        for f in (sv.spec_grad_norm, sv.spec_clip_grads):
            keep = g.clone()
            out, ws = f(bad, max_norm=1.0)
            assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG and bool(torch.isnan(out).all())
            assert torch.equal(g, keep)


def test_the_same_bits_every_time():
    rng = np.random.default_rng(8)
    table = table_of(make(rng, [700001, 33, 123457]))
    first, _ = sv.spec_grad_norm(table, max_norm=1.0)
    for _ in range(5):
        assert torch.equal(sv.spec_grad_norm(table, max_norm=1.0)[0], first)


@pytest.mark.parametrize("clip", [False, True])
def test_replays_in_a_graph(clip):
    rng = np.random.default_rng(9)
    grads = make(rng, [5000, 70001])
    table = table_of(grads)
    f = sv.spec_clip_grads if clip else sv.spec_grad_norm
    ws = torch.empty(sv.spec_grad_norm_workspace(), dtype=torch.uint8, device=DEV)
    out = torch.empty(2, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f(table, max_norm=1e9, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f(table, max_norm=3.0, out=out, workspace=ws)
    for k in range(3):
        for x in grads:
            x.copy_(torch.tensor(rng.normal(size=x.numel()) * (k + 1)))
        norm, factor = O.grad_norm([f64(x) for x in grads], 3.0)
        g.replay()
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        assert abs(float(out[0]) - norm) <= TOL * norm and abs(float(out[1]) - factor) <= 2 * TOL * factor


@pytest.mark.parametrize("dtype,bits", [(F32, 32), (BF16, 8)])
def test_the_optimizer_takes_the_factor(dtype, bits):
    """A step by the factor and a step on clipped gradients: the same up to the gradients'
    rounding (none in f32: each product is one rounding in both)."""
    rng = np.random.default_rng(10)
    grads = make(rng, [3000, 513], dtype, 5.0)
    copies = [g.clone() for g in grads]
    a, b = table_of(grads, bits), table_of(copies, bits)
    h = dict(lr=1e-2, weight_decay=0.0)
    out, _ = sv.spec_grad_norm(a, max_norm=1.0)
    sv.spec_adamw_step(a, 1, grad_scale=out[1:], **h)
    sv.spec_clip_grads(b, max_norm=1.0)
    sv.spec_adamw_step(b, 1, **h)
    for i in range(2):
        p, q = a.tensors[0][i], b.tensors[0][i]
        if dtype is F32:
            assert torch.equal(p, q)
        else:   # a first step is lr in size whatever the gradient's
            assert float((p.float() - q.float()).abs().max()) <= 2.0 ** -7 * 1e-2


def test_on_a_stream_and_wrong_tensors():
    grads = make(np.random.default_rng(1), [5000])
    table = table_of(grads)
    ref, _ = sv.spec_grad_norm(table, max_norm=1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _ = sv.spec_grad_norm(table, max_norm=1.0, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    with pytest.raises(ValueError):
        sv.spec_grad_norm(table, out=torch.empty(1, device=DEV))
    with pytest.raises(TypeError):
        sv.spec_grad_norm(table, grad_scale=torch.ones(1, dtype=torch.float64, device=DEV))
    with pytest.raises(sv.SpecError):
        sv.spec_grad_norm(table, max_norm=0.0)
