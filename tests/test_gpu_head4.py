"""The head's products with weights of 4 bits on the GPU against the 64-bit reference:
layout, rounding to 4 bits and back, and products of one to 64 rows at sizes, groups and
columns where chunks, tiles, panels and groups end."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
HALF = 2.0 ** -8    # half a step of bf16
ACT = {"none": sv.SPEC_ACT_NONE, "silu": sv.SPEC_ACT_SILU, "gelu": sv.SPEC_ACT_GELU}


def f64(t):
    return t.double().cpu().numpy()


def bf(a):
    return torch.tensor(a).to(BF16).to(DEV)


def weight(rng, N, K, group, zeros):
    """(SpecHead4, its values in 64 bits)."""
    G = -(-K // group)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = bf(rng.uniform(0.2, 2.0, (N, G)) / np.sqrt(K))
    z = rng.integers(0, 16, (N, G)).astype(np.uint8) if zeros else None
    even = codes if K % 2 == 0 else np.concatenate([codes, np.full((N, 1), 13, np.uint8)], 1)
    rows = even[:, 0::2] | (even[:, 1::2] << 4)
    w = sv.spec_head4_pack(torch.tensor(rows, device=DEV), scales,
                           None if z is None else torch.tensor(z, device=DEV), K=K, group=group)
    return w, O.dequantize4(codes, f64(scales), z, group)


def reference(x, w, bias, residual, act, group):
    """(y, tolerance): sums of K products in 32 bits, a step of 2^-22 of the magnitudes for each
    instruction, group, warp and slice that they go through (the tensor cores' sums may be cut, not
    rounded), x within 2^-40 of its row's largest, an activation of slope 1.13 at most within 2^-20,
    one rounding to bf16."""
    K = x.shape[1]
    z, size = x @ w.T, np.abs(x) @ np.abs(w).T
    steps = group // 16 + -(-K // group) + 16 + -(-K // 128)
    lost = 2.0 ** -40 * np.abs(x).max(1, initial=0)[:, None] * np.abs(w).sum(1)[None]
    if bias is not None:
        z, size = z + bias, size + np.abs(bias)
    y = O.act(z, act)
    err = 1.2 * (steps * 2.0 ** -22 * size + lost) + 2.0 ** -20 * np.abs(y)
    if residual is not None:
        y = y + residual
    return y, err + HALF * (np.abs(y) + err) + 1e-38


FORWARD = [
    (1, 1, 1, 32, 0, "none", 0, 0), (1, 128, 16, 128, 0, "none", 1, 0), (1, 4096, 1000, 128, 0, "none", 1, 0),
    (2, 100, 33, 32, 1, "silu", 1, 1), (3, 127, 17, 64, 1, "gelu", 0, 1), (4, 129, 50, 128, 0, "none", 0, 0),
    (5, 1025, 700, 64, 0, "silu", 1, 1), (7, 2880, 301, 32, 1, "none", 1, 1), (8, 640, 2500, 128, 1, "gelu", 1, 0),
    (9, 333, 129, 32, 0, "none", 0, 1), (16, 1000, 260, 64, 1, "silu", 1, 1), (17, 520, 90, 128, 0, "none", 1, 0),
    (31, 96, 1030, 32, 1, "none", 0, 0), (32, 2880, 400, 32, 1, "silu", 1, 1), (33, 64, 47, 64, 0, "gelu", 1, 1),
    (64, 4100, 300, 128, 1, "none", 1, 1), (64, 31, 5000, 32, 0, "silu", 0, 0), (40, 7000, 64, 64, 1, "none", 0, 0),
    (8, 14400, 40, 128, 0, "none", 0, 1), (1, 70000, 24, 128, 1, "none", 1, 0)]


@pytest.mark.parametrize("M,K,N,group,zeros,act,bias,residual", FORWARD)
def test_forward(M, K, N, group, zeros, act, bias, residual):
    rng = np.random.default_rng(M * 7 + K + N)
    w, ref_w = weight(rng, N, K, group, zeros)
    x = bf(rng.normal(size=(M, K)))
    b = bf(rng.normal(size=N)) if bias else None
    r = bf(rng.normal(size=(M, N))) if residual else None
    guard = torch.full((M * N + 64,), 3.0, dtype=BF16, device=DEV)
    y = guard[:M * N].view(M, N)
    _, ws = sv.spec_head4_forward(x, w, b, r, act=ACT[act], out=y)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    want, tol = reference(f64(x), ref_w, None if b is None else f64(b), None if r is None else f64(r), act, group)
    off = np.abs(f64(y) - want) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    assert bool((guard[M * N:] == 3).all())
    again, _ = sv.spec_head4_forward(x, w, b, r, act=ACT[act])
    assert torch.equal(again, y)


def test_many_tiles():
    """More tiles than CTAs, so that each takes several; rows of x one by one give the same."""
    rng = np.random.default_rng(4)
    for K, N, group in ((384, 40000, 64), (1024, 20011, 128)):
        w, ref_w = weight(rng, N, K, group, 1)
        x = bf(rng.normal(size=(3, K)))
        y, _ = sv.spec_head4_forward(x, w)
        want, tol = reference(f64(x), ref_w, None, None, "none", group)
        assert (np.abs(f64(y) - want) <= tol).all()
        for m in range(3):
            assert torch.equal(sv.spec_head4_forward(x[m:m + 1], w)[0], y[m:m + 1])


@pytest.mark.parametrize("scale", [1e-37, 1e-12, 1e20, 3e37])
def test_rows_of_any_size(scale):
    """x of few and of many binades: rows are brought to fp16's range."""
    rng = np.random.default_rng(8)
    w, ref_w = weight(rng, 100, 520, 64, 1)
    x = rng.normal(size=(6, 520)) * min(scale, 1e36)
    x[1] *= 2.0 ** rng.integers(-60, 0, 520)
    x[2, 3:] = 0
    x[3] = 0
    x[4, 100] *= 2.0 ** 30 if scale < 1e20 else 4
    x = bf(x)
    y, _ = sv.spec_head4_forward(x, w)
    want, tol = reference(f64(x), ref_w, None, None, "none", 64)
    assert (np.abs(f64(y) - want) <= tol).all()
    assert bool((y[3] == 0).all())


@pytest.mark.parametrize("M", [1, 12, 64])
def test_infinities_stay_in_their_row(M):
    rng = np.random.default_rng(5)
    w, ref_w = weight(rng, 50, 300, 64, 1)
    x = bf(rng.normal(size=(M, 300)))
    clean, _ = sv.spec_head4_forward(x, w)
    x[0, 7] = float("inf")
    y, _ = sv.spec_head4_forward(x, w)
    col = ref_w[:, 7]
    on = torch.tensor(col != 0, device=DEV)
    assert bool((~torch.isfinite(y[0][on])).all())
    assert torch.equal(y[1:], clean[1:])


def test_residual_in_place_and_no_rows():
    rng = np.random.default_rng(6)
    w, _ = weight(rng, 64, 256, 32, 0)
    x, r = bf(rng.normal(size=(4, 256))), bf(rng.normal(size=(4, 64)))
    want, _ = sv.spec_head4_forward(x, w, None, r)
    got = r.clone()
    sv.spec_head4_forward(x, w, None, got, out=got)
    assert torch.equal(got, want)
    y, ws = sv.spec_head4_forward(x[:0], w)
    assert y.shape == (0, 64) and sv.spec_get_status(ws) == sv.SPEC_OK


def test_rows_that_are_not_aligned():
    """Bias, residual and y at any element; codes, scales and zeros too."""
    rng = np.random.default_rng(7)
    N, K, group = 70, 200, 32

    def moved(t):
        out = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        out.copy_(t)
        return out

    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales, zeros = bf(rng.uniform(0.01, 0.1, (N, 7))), rng.integers(0, 16, (N, 7)).astype(np.uint8)
    w = sv.spec_head4_pack(moved(torch.tensor(codes[:, 0::2] | codes[:, 1::2] << 4, device=DEV)), moved(scales),
                           moved(torch.tensor(zeros, device=DEV)), K=K, group=group)
    ref_w = O.dequantize4(codes, f64(scales), zeros, group)
    x, b, r = bf(rng.normal(size=(5, K))), moved(bf(rng.normal(size=N))), moved(bf(rng.normal(size=(5, N))))
    y = moved(torch.zeros(5, N, dtype=BF16, device=DEV))
    sv.spec_head4_forward(x, w, b, r, out=y)
    want, tol = reference(f64(x), ref_w, f64(b), f64(r), "none", group)
    assert (np.abs(f64(y) - want) <= tol).all()


@pytest.mark.parametrize("N,K,group,zeros", [(1, 1, 32, 0), (3, 31, 32, 1), (5, 128, 64, 0), (7, 129, 128, 1),
                                             (40, 1000, 64, 1), (33, 2880, 32, 0)])
def test_unpack(N, K, group, zeros):
    w, ref_w = weight(np.random.default_rng(N + K), N, K, group, zeros)
    got = sv.spec_head4_unpack(w)
    assert got.shape == (N, K) and np.array_equal(f64(got), O.to_bf16(ref_w))


@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (3, 31, 32), (5, 128, 64), (9, 129, 128), (40, 1000, 64),
                                       (33, 2880, 32), (70, 4096, 128), (6, 33, 128)])
def test_quantize(N, K, group):
    rng = np.random.default_rng(N * K)
    x = rng.normal(size=(N, K)) * 2.0 ** rng.integers(-30, 30, (N, 1))
    x[0, : K // 2] = 0.0
    x[N // 2] = rng.integers(-14, 15, K) / 2.0      # many exact ties
    if N > 2:
        x[2] = 0.0
    wt = bf(x)
    q, ws = sv.spec_head4_quantize(wt, group=group)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    codes, scales = O.quantize4(f64(wt), group)
    assert np.array_equal(f64(sv.spec_head4_unpack(q)), O.to_bf16(O.dequantize4(codes, scales, None, group)))
    # no value further than half a step, a little more where the scale was rounded down
    err = np.abs(f64(wt) - O.dequantize4(codes, scales, None, group))
    assert (err <= (0.5 + 7 * HALF) * np.repeat(scales, group, 1)[:, :K] + 1e-300).all()
    # again into the same weight
    wt2 = bf(rng.normal(size=(N, K)))
    sv.spec_head4_quantize(wt2, group=group, out=q)
    fresh, _ = sv.spec_head4_quantize(wt2, group=group)
    assert torch.equal(fresh.packed, q.packed)


def test_quantize_reports_what_is_not_finite():
    wt = bf(np.random.default_rng(0).normal(size=(6, 200)))
    clean, _ = sv.spec_head4_quantize(wt, group=32)
    wt[3, 70] = float("nan")
    wt[4, 5] = -float("inf")
    q, ws = sv.spec_head4_quantize(wt, group=32)
    assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG
    got, ref = sv.spec_head4_unpack(q), sv.spec_head4_unpack(clean)
    assert float(got[3, 70]) == 0 and float(got[4, 5]) == 0 and bool(torch.isfinite(got).all())
    keep = torch.ones(6, 200, dtype=torch.bool, device=DEV)
    keep[3, 64:96] = keep[4, :32] = False       # their groups
    assert torch.equal(got[keep], ref[keep])


def test_quantize_of_the_smallest_weights():
    wt = torch.full((2, 64), 2.0 ** -126, dtype=BF16, device=DEV)    # their scale is no normal number
    wt[1] = 2.0 ** -120
    q, ws = sv.spec_head4_quantize(wt, group=64)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    got = sv.spec_head4_unpack(q)
    assert bool((got[0] == 0).all()) and abs(float(got[1, 0]) / 2.0 ** -120 - 1) <= 7 * HALF


def test_unaligned_weights_are_quantized_alike():
    wt = bf(np.random.default_rng(1).normal(size=(5, 264)))
    odd = torch.empty(5 * 264 + 1, dtype=BF16, device=DEV)[1:].view(5, 264)
    odd.copy_(wt)
    a, _ = sv.spec_head4_quantize(wt, group=64)
    b, _ = sv.spec_head4_quantize(odd, group=64)
    assert torch.equal(a.packed, b.packed)


def test_wrong_tensors_are_refused():
    rng = np.random.default_rng(2)
    w, _ = weight(rng, 32, 96, 32, 0)
    x = bf(rng.normal(size=(4, 96)))
    for args, kw in (((x.float(), w), {}), ((x[:, :64].contiguous(), w), {}), ((x, w, torch.zeros(31, dtype=BF16, device=DEV)), {}),
                     ((x, w), dict(residual=torch.zeros(32, 4, dtype=BF16, device=DEV))),
                     ((x, w), dict(out=torch.zeros(32, 4, dtype=BF16, device=DEV)))):
        with pytest.raises((TypeError, ValueError)):
            sv.spec_head4_forward(*args, **kw)
    with pytest.raises(sv.SpecError):
        sv.spec_head4_forward(torch.zeros(65, 96, dtype=BF16, device=DEV), w)
    codes = torch.zeros(8, 16, dtype=torch.uint8, device=DEV)
    s = torch.ones(8, 1, dtype=BF16, device=DEV)
    for c, sc, z, kw in ((codes, s, None, dict(K=40, group=32)), (codes, s[:, :0], None, dict(K=32, group=32)),
                         (codes, s, codes, dict(K=32, group=32)), (codes, s, None, dict(K=32, group=48))):
        with pytest.raises((TypeError, ValueError, sv.SpecError)):
            sv.spec_head4_pack(c, sc, z, **kw)
    with pytest.raises(ValueError):
        sv.spec_head4_quantize(torch.zeros(8, 64, dtype=BF16, device=DEV), group=32, out=w)


def test_replays_in_a_graph():
    rng = np.random.default_rng(3)
    w, ref_w = weight(rng, 500, 640, 64, 1)
    x = bf(rng.normal(size=(6, 640)))
    y = torch.empty(6, 500, dtype=BF16, device=DEV)
    ws = torch.empty(sv.spec_head4_forward_workspace(6, 500, 640), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sv.spec_head4_forward(x, w, out=y, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_head4_forward(x, w, out=y, workspace=ws)
    x.copy_(bf(rng.normal(size=(6, 640))))
    g.replay()
    want, tol = reference(f64(x), ref_w, None, None, "none", 64)
    assert (np.abs(f64(y) - want) <= tol).all()


@pytest.fixture
def checked():
    sv.use_checked_library(True)
    yield
    sv.use_checked_library(False)


def test_no_access_leaves_the_call(checked):
    for case in FORWARD:
        test_forward(*case)
    test_unpack(7, 129, 128, 1)
    test_quantize(9, 129, 128)
    test_quantize(3, 31, 32)


@pytest.mark.parametrize("M,K,N,group", [(32, 256, 40000, 64), (20, 130, 48641, 32), (12, 200, 50257, 128), (64, 130, 77777, 64),
                                         (17, 384, 128256, 128), (9, 40, 39000, 32), (28, 300, 95001, 64)])
def test_many_tiles_of_more_rows(M, K, N, group):
    """Tiles that come to one round of the warps, to several, and to uneven ones."""
    rng = np.random.default_rng(M + N)
    w, ref_w = weight(rng, N, K, group, 1)
    x, b, r = bf(rng.normal(size=(M, K))), bf(rng.normal(size=N)), bf(rng.normal(size=(M, N)))
    guard = torch.full((M * N + 64,), 3.0, dtype=BF16, device=DEV)
    y, ws = sv.spec_head4_forward(x, w, b, r, act=sv.SPEC_ACT_SILU, out=guard[:M * N].view(M, N))
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    want, tol = reference(f64(x), ref_w, f64(b), f64(r), "silu", group)
    assert (np.abs(f64(y) - want) <= tol).all() and bool((guard[M * N:] == 3).all())
    # fewer rows of the same
    again, _ = sv.spec_head4_forward(x[:9], w, b, r[:9].contiguous(), act=sv.SPEC_ACT_SILU)
    want, tol = reference(f64(x[:9]), ref_w, f64(b), f64(r[:9]), "silu", group)
    assert (np.abs(f64(again) - want) <= tol).all()
