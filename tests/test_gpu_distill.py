"""spec_distill_loss on the GPU against the 64-bit reference: loss and
gradient, both types, cluster sizes and alignments, masked tokens, weights of
zero, greedy temperatures, and the gradient against differences."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make(seed, V, K, dtype, masked=0.0, zero_every=0, sigma=0.7, T=(0.5, 1.5)):
    g = torch.Generator().manual_seed(seed)
    B = len(K)
    cu = np.concatenate([[0], np.cumsum(K)]).astype(np.int32)
    R = int(cu[-1])
    t = 2 * torch.randn(R + B, V, generator=g)
    req = np.repeat(np.arange(B), K)
    d = t[torch.tensor(np.arange(R) + req)] + sigma * torch.randn(R, V, generator=g)
    if masked:
        ban = torch.rand(V, generator=g) < masked
        ban[0] = False
        t[:, ban] = -np.inf
        d[:, ban] = -np.inf
    temp = T[0] + (T[1] - T[0]) * torch.rand(B, generator=g)
    w = torch.rand(R, generator=g)
    if zero_every:
        w[::zero_every] = 0
    return t.to(dtype).to(DEV), d.to(dtype).to(DEV), cu, temp.to(DEV), w.to(DEV)


def check(t, d, cu, temp, w, loss, grad):
    n = lambda x: None if x is None else x.float().cpu().numpy()   # noqa: E731
    rl, rg, terms = O.distill(n(t), n(d), cu, n(temp), n(w))
    V = d.shape[1]
    # an exponential is off by 2 ulp and by its argument's roundings (three, of
    # an argument of at most 64 before it stops to matter); a thread sums up
    # to V/256 + 8 terms one by one, then 16 merges of three roundings each
    rel = U32 * (8 + 3 * 64 + V / 256 + 8 + 48)
    got = loss.cpu().numpy().astype(np.float64)
    both = np.isfinite(rl)
    assert np.array_equal(both, np.isfinite(got)) and np.array_equal(rl[~both], got[~both])
    assert np.all(np.abs(got - rl)[both] <= (rel * (terms + np.abs(n(w) if w is not None else 1)) +
                                             U32 * np.abs(rl))[both])
    if grad is not None:
        gg = grad.float().cpu().numpy().astype(np.float64)
        T = np.repeat(np.where(n(temp) < 0.05, 1, n(temp)) if temp is not None else np.ones(len(cu) - 1),
                      np.diff(cu))
        k = (n(w) if w is not None else np.ones(len(T))) / T
        p_plus_q = np.abs(rg) + 2 * np.minimum(*_pq(n(t), n(d), cu, T)) * k[:, None]
        before = rel * p_plus_q + 3 * U32 * np.abs(rg)
        tol = before + HALF[d.dtype] * (np.abs(rg) + before) + 1e-38
        assert np.all(np.abs(gg - rg) <= tol), np.max(np.abs(gg - rg) - tol)


def _pq(t, d, cu, T):
    req = np.repeat(np.arange(len(cu) - 1), np.diff(cu))
    zt = t[np.arange(len(d)) + req].astype(np.float64) / T[:, None]
    zd = d.astype(np.float64) / T[:, None]
    e = lambda z: np.exp(z - z.max(1, keepdims=True))   # noqa: E731
    return e(zt) / e(zt).sum(1, keepdims=True), e(zd) / e(zd).sum(1, keepdims=True)


CASES = [
    ("one token", dict(V=1, K=[1], dtype=torch.float32)),
    ("small f32", dict(V=1024, K=[4, 4, 4, 4], dtype=torch.float32)),
    ("odd f32", dict(V=1003, K=[1, 0, 3], dtype=torch.float32)),
    ("f32 two CTAs", dict(V=5000, K=[2, 1], dtype=torch.float32)),
    ("f32 eight CTAs", dict(V=20000, K=[2, 1], dtype=torch.float32)),
    ("bf16", dict(V=1000, K=[3, 2], dtype=torch.bfloat16)),
    ("bf16 shifts", dict(V=1009, K=[3, 4, 2, 5, 3], dtype=torch.bfloat16)),
    ("bf16 even shifts", dict(V=2050, K=[1, 2, 1, 3, 1, 2, 2, 1, 1], dtype=torch.bfloat16)),
    ("f32 shifts", dict(V=1022, K=[1, 3, 1, 2, 2], dtype=torch.float32)),
    ("few tokens", dict(V=9, K=[1, 3, 2, 4, 2], dtype=torch.bfloat16)),
    ("fewer than a vector", dict(V=3, K=[2, 3, 2], dtype=torch.float32)),
    ("bf16 odd", dict(V=32003, K=[1, 2], dtype=torch.bfloat16)),
    ("bf16 cluster", dict(V=32008, K=[2, 2], dtype=torch.bfloat16)),
    ("masked", dict(V=9000, K=[2, 3], dtype=torch.bfloat16, masked=0.6)),
    ("weights of zero", dict(V=40000, K=[5, 4], dtype=torch.bfloat16, zero_every=2)),
    ("far laws", dict(V=2000, K=[2], dtype=torch.float32, sigma=6.0)),
    ("greedy", dict(V=2000, K=[2, 2], dtype=torch.float32, T=(0.0, 0.04))),
    ("many requests", dict(V=64, K=[1, 2, 0] * 200, dtype=torch.float32)),
]


@pytest.mark.parametrize("checked", [False, True])
@pytest.mark.parametrize("name,case", CASES, ids=[c[0] for c in CASES])
def test_distill(name, case, checked):
    sv.use_checked_library(checked)
    try:
        t, d, cu, temp, w = make(len(name), **case)
        loss, grad, ws = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), temp, w)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        check(t, d, cu, temp, w, loss, grad)
    finally:
        sv.use_checked_library(False)


def test_distill_large_rows():
    t, d, cu, temp, w = make(3, V=201088, K=[2, 1], dtype=torch.bfloat16)
    loss, grad, ws = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), temp, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    check(t, d, cu, temp, w, loss, grad)


@pytest.mark.parametrize("V,R,dtype", [(201088, 60, torch.bfloat16), (32000, 700, torch.bfloat16),
                                       (4096, 3000, torch.bfloat16), (8, 700000, torch.float32),
                                       (50000, 200, torch.float32), (131080, 90, torch.bfloat16)])
@pytest.mark.parametrize("zero_every", [0, 3])
def test_distill_many_positions(V, R, dtype, zero_every):
    """Calls that fill the SMs: rows held by clusters of each size, some of
    one piece, ragged requests; a sample of positions against the reference,
    the rest by the gradient's zero sum and the same bits in a second call."""
    K = [(i * 7) % 5 for i in range(R)]
    cu = np.concatenate([[0], np.cumsum(K)])
    B = int(np.searchsorted(cu, R))
    cu = np.minimum(cu[:B + 1], R).astype(np.int32)
    g = torch.Generator(device=DEV).manual_seed(V + R)
    t = (2 * torch.randn(R + B, V, generator=g, device=DEV)).to(dtype)
    d = (2 * torch.randn(R, V, generator=g, device=DEV)).to(dtype)
    temp = 0.5 + torch.rand(B, generator=g, device=DEV)
    w = 0.1 + torch.rand(R, generator=g, device=DEV)
    if zero_every:
        w[::zero_every] = 0
    cu_t = torch.tensor(cu, device=DEV)
    loss, grad, ws = sv.spec_distill_loss(t, d, cu_t, temp, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    again = sv.spec_distill_loss(t, d, cu_t, temp, w)
    assert torch.equal(loss, again[0]) and torch.equal(grad, again[1])
    alone, _, _ = sv.spec_distill_loss(t, d, cu_t, temp, w, want_grad=False)
    assert torch.equal(loss, alone)
    assert bool((loss[w == 0] == 0).all()) and not bool(grad[w == 0].any())
    assert bool((loss[w != 0] > 0).all())
    # sum over x of q - p is 0: what is left are the roundings of the values and
    # the errors of p and q (each law sums to 1; see check), times w / T
    req = np.repeat(np.arange(B), np.diff(cu))
    rel = U32 * (8 + 3 * 64 + V / 256 + 8 + 48)
    left = grad.double().sum(1).abs()
    assert bool((left <= HALF[dtype] * grad.double().abs().sum(1) +
                 2 * rel * (w / temp[torch.tensor(req, device=DEV)]).double()).all())
    for r in {0, 1, R // 2, R - 1}:
        b = int(req[r])
        check(t[r + b:r + b + 2] if r + b + 2 <= R + B else t[[r + b, r + b]], d[r:r + 1], np.array([0, 1]),
              temp[b:b + 1], w[r:r + 1], loss[r:r + 1], grad[r:r + 1])


def test_distill_resident_checked():
    sv.use_checked_library(True)
    try:
        t, d, cu, temp, w = make(12, V=16384, K=[5] * 120, dtype=torch.bfloat16, zero_every=4)
        loss, grad, ws = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), temp, w)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        check(t[:6], d[:5], np.array([0, 5]), temp[:1], w[:5], loss[:5], grad[:5])
    finally:
        sv.use_checked_library(False)


def test_distill_defaults_and_loss_alone():
    t, d, cu, _, _ = make(9, V=300, K=[2, 2], dtype=torch.float32)
    loss, grad, _ = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV))
    check(t, d, cu, None, None, loss, grad)
    alone, none, _ = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), want_grad=False)
    assert none is None and torch.equal(alone, loss)


def test_distill_draft_probability_of_zero_is_an_infinite_loss():
    t, d, cu, temp, w = make(4, V=200, K=[2], dtype=torch.float32)
    d[1, 5] = -float("inf")
    loss, grad, ws = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), temp, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    assert torch.isfinite(loss[0]) and loss[1] == float("inf") and bool(torch.isfinite(grad).all())
    check(t, d, cu, temp, w, loss, grad)


def test_distill_gradient_against_differences():
    t, d, cu, temp, w = make(6, V=40, K=[2, 1], dtype=torch.float32)
    cu_t = torch.tensor(cu, device=DEV)
    _, grad, _ = sv.spec_distill_loss(t, d, cu_t, temp, w)
    h = 0.02
    for r, x in ((0, 0), (1, 17), (2, 39)):
        up, dn = d.clone(), d.clone()
        up[r, x] += h
        dn[r, x] -= h
        lu, ld = (sv.spec_distill_loss(t, q, cu_t, temp, w, want_grad=False)[0][r] for q in (up, dn))
        diff = float(lu - ld) / float(up[r, x] - dn[r, x])
        # h^2/6 of the third derivative (below w/T^3 <= 8), and the losses'
        # roundings (terms below 32, 2^-16 relative) over 2h
        assert abs(diff - float(grad[r, x])) <= h * h / 6 * 8 + 32 * 300 * U32 / (2 * h)


def test_distill_reports_bad_inputs():
    t, d, cu, temp, w = make(2, V=100, K=[2, 2], dtype=torch.float32)
    cu_t = torch.tensor(cu, device=DEV)
    call = lambda **k: sv.spec_get_status(sv.spec_distill_loss(**{**dict(   # noqa: E731
        target=t, draft=d, cu_draft=cu_t, temperature=temp, weight=w), **k})[2])
    assert call() == sv.SPEC_OK
    assert call(temperature=torch.tensor([1.0, float("nan")], device=DEV)) == sv.SPEC_ERR_INVALID_ARG
    assert call(temperature=torch.tensor([-1.0, 1.0], device=DEV)) == sv.SPEC_ERR_INVALID_ARG
    assert call(weight=torch.tensor([1, 1, float("inf"), 1], device=DEV)) == sv.SPEC_ERR_INVALID_ARG
    assert call(cu_draft=torch.tensor([0, 3, 2], dtype=torch.int32, device=DEV)) == sv.SPEC_ERR_INVALID_ARG
    assert call(cu_draft=torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)) == sv.SPEC_ERR_INVALID_ARG
    empty = d.clone()
    empty[1] = -float("inf")
    loss, grad, ws = sv.spec_distill_loss(t, empty, cu_t, temp, w)
    assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG
    assert loss[1] == 0 and not bool(grad[1].any())


def test_distill_in_a_graph():
    t, d, cu, temp, w = make(8, V=32008, K=[3, 2], dtype=torch.bfloat16)
    cu_t = torch.tensor(cu, device=DEV)
    l0, g0, ws = sv.spec_distill_loss(t, d, cu_t, temp, w)
    out = (torch.empty_like(l0), torch.empty_like(g0))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_distill_loss(t, d, cu_t, temp, w, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], l0) and torch.equal(out[1], g0)
