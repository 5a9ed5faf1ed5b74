"""spec_head_forward and spec_head_backward on the GPU against products in 64
bits: one row to many, odd sizes of every dimension, splits of the reduction,
activations, bias, residual, and the gradients against the formulas and
against differences."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = 2.0 ** -8    # half a step of bf16, relative
U32 = 2.0 ** -24
ACT = {"none": sv.SPEC_ACT_NONE, "silu": sv.SPEC_ACT_SILU, "gelu": sv.SPEC_ACT_GELU}


def rand(shape, scale, g):
    return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16).to(DEV)


def f64(x):
    return x.double().cpu().numpy()


def sum_tol(R):
    """Relative to the sum of magnitudes: a tensor-core step adds 16 products
    and the accumulator with one truncation to 24 bits (2^-23), and the parts
    of a split are added up (at most 32 more)."""
    return (R / 16 + 2 + 33) * 2 * U32


def product_tol(a, b, R):
    return sum_tol(R) * (np.abs(a) @ np.abs(b))


FORWARD = [
    (1, 64, 64, "none", 0, 0), (1, 4096, 1000, "none", 1, 0), (1, 512, 40000, "none", 0, 0),
    (3, 136, 130, "silu", 1, 1), (16, 256, 384, "gelu", 1, 0), (17, 2048, 129, "none", 1, 1),
    (5, 63, 77, "silu", 1, 1), (1, 1, 1, "none", 1, 1), (2, 9, 4099, "none", 0, 1),
    (100, 300, 520, "gelu", 0, 1), (257, 320, 1000, "silu", 1, 1), (300, 2880, 260, "none", 1, 0),
    (513, 65, 200, "gelu", 1, 1), (700, 1024, 6000, "none", 0, 0), (129, 8192, 128, "silu", 1, 0),
    (1100, 512, 9000, "gelu", 1, 1), (600, 200, 20001, "silu", 1, 1), (256, 4096, 8192, "none", 0, 0),
    (2, 5000, 3000, "gelu", 1, 1), (4, 4104, 999, "silu", 1, 0), (3, 9001, 70, "none", 1, 1), (5, 4096, 32000, "none", 0, 0),
]


@pytest.mark.parametrize("M,K,N,act,bias,residual", FORWARD)
def test_forward(M, K, N, act, bias, residual):
    g = torch.Generator().manual_seed(M * 7 + K + N)
    x, w = rand((M, K), 1.0, g), rand((N, K), K ** -0.5, g)
    b = rand((N,), 0.5, g) if bias else None
    r = rand((M, N), 1.0, g) if residual else None
    y, pre, ws = sv.spec_head_forward(x, w, b, r, act=ACT[act], want_pre=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    z = f64(x) @ f64(w).T + (f64(b) if bias else 0)
    tz = product_tol(f64(x), f64(w).T, K) + U32 * np.abs(z)
    assert np.all(np.abs(f64(pre) - z) <= tz + HALF * (np.abs(z) + tz))
    ref = O.act(z, act)
    # a slope of at most 1.13; the activation's own roundings, 16 of them
    ty = (1.13 if act != "none" else 1.0) * tz + 16 * U32 * (np.abs(ref) + (np.abs(z) if act != "none" else 0))
    ref = ref + (f64(r) if residual else 0)
    ty = ty + U32 * np.abs(ref)
    assert np.all(np.abs(f64(y) - ref) <= ty + HALF * (np.abs(ref) + ty))
    y2, none, _ = sv.spec_head_forward(x, w, b, r, act=ACT[act])
    assert none is None and torch.equal(y, y2)   # the same bits again


BACKWARD = [
    (1, 64, 64, "none"), (1, 256, 1000, "silu"), (7, 63, 65, "gelu"), (16, 520, 384, "none"),
    (100, 300, 520, "silu"), (257, 320, 1000, "gelu"), (300, 136, 2881, "none"), (513, 65, 200, "silu"),
    (64, 1024, 4096, "none"), (1000, 128, 3000, "silu"), (1, 1, 1, "gelu"), (2000, 200, 72, "none"),
    (900, 1100, 6000, "silu"), (513, 2050, 3001, "none"), (1024, 1024, 4096, "gelu"),
]


@pytest.mark.parametrize("M,K,N,act", BACKWARD)
def test_backward(M, K, N, act):
    g = torch.Generator().manual_seed(M + K * 3 + N)
    x, w, dy = rand((M, K), 1.0, g), rand((N, K), K ** -0.5, g), rand((M, N), 1.0, g)
    pre = rand((M, N), 1.5, g) if act != "none" else None
    dx, dw, db, ws = sv.spec_head_backward(dy, x, w, pre, act=ACT[act], want_db=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    dz = f64(dy) * (O.act_slope(f64(pre), act) if act != "none" else 1.0)
    # the operand: the slope's roundings (32 of values up to 4), one rounding to bf16
    td = (32 * U32 * 4 * np.abs(f64(dy)) + HALF * np.abs(dz)) if act != "none" else 0 * dz
    for got, a, b, ta, R in ((dx, dz, f64(w), td, N), (dw, dz.T, f64(x), td.T, M)):
        ref = a @ b
        t = (np.abs(ta) @ np.abs(b)) + sum_tol(R) * ((np.abs(a) + np.abs(ta)) @ np.abs(b))
        assert np.all(np.abs(f64(got) - ref) <= t + HALF * (np.abs(ref) + t))
    ref = dz.sum(0)
    t = (M / 8 + 16 + M / 64) * U32 * np.abs(dz).sum(0) + (32 * U32 * 4 * np.abs(f64(dy)).sum(0) if act != "none" else 0)
    assert np.all(np.abs(db.double().cpu().numpy() - ref) <= t + U32 * np.abs(ref))


def test_backward_parts_alone():
    g = torch.Generator().manual_seed(1)
    x, w, dy, pre = rand((33, 72), 1, g), rand((100, 72), 0.1, g), rand((33, 100), 1, g), rand((33, 100), 1, g)
    full = sv.spec_head_backward(dy, x, w, pre, act=sv.SPEC_ACT_SILU, want_db=True)[:3]
    for k in range(3):
        want = [i == k for i in range(3)]
        part = sv.spec_head_backward(dy, x, w, pre, act=sv.SPEC_ACT_SILU, want_dx=want[0], want_dw=want[1],
                                     want_db=want[2])[:3]
        for i in range(3):
            assert part[i] is None if i != k else torch.equal(part[i], full[i])


def test_backward_of_nothing_is_ok():
    x, w = torch.ones(3, 64, dtype=torch.bfloat16, device=DEV), torch.ones(8, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((1 << 16,), 255, dtype=torch.uint8, device=DEV)
    assert sv.spec_head_backward_workspace(3, 8, 64) <= ws.numel()
    sv.spec_head_backward(x[:, :8].contiguous(), x, w, out=(None, None, None), workspace=ws)
    assert sv.spec_get_status(ws) == sv.SPEC_OK


def test_no_rows():
    x, w = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV), torch.ones(40, 64, dtype=torch.bfloat16, device=DEV)
    y, _, ws = sv.spec_head_forward(x, w)
    assert y.shape == (0, 40) and sv.spec_get_status(ws) == sv.SPEC_OK
    dx, dw, db, ws = sv.spec_head_backward(y, x, w, want_db=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK and dx.shape == (0, 64)
    assert not bool(dw.any()) and not bool(db.any())


def test_infinities_and_nan_stay_in_their_rows():
    g = torch.Generator().manual_seed(2)
    x, w = rand((20, 128), 1, g), rand((200, 128), 0.1, g)
    clean = sv.spec_head_forward(x, w)[0]
    x[3, 5], x[7, 9] = float("nan"), float("inf")
    y = sv.spec_head_forward(x, w)[0]
    rows = torch.arange(20, device=DEV)
    ok = (rows != 3) & (rows != 7)
    assert torch.equal(y[ok], clean[ok])
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[7]).any())


def test_residual_in_place():
    g = torch.Generator().manual_seed(3)
    x, w, r = rand((37, 96), 1, g), rand((200, 96), 0.1, g), rand((37, 200), 1, g)
    want = sv.spec_head_forward(x, w, None, r, act=sv.SPEC_ACT_GELU)[0]
    sv.spec_head_forward(x, w, None, r, act=sv.SPEC_ACT_GELU, out=(r, None))
    assert torch.equal(r, want)


def test_gradients_against_differences():
    """L = sum(c * y); dx by central differences of the 64-bit forward at the
    kernel's own pre-activation."""
    g = torch.Generator().manual_seed(4)
    M, K, N = 3, 24, 40
    x, w, b, c = rand((M, K), 1, g), rand((N, K), 0.3, g), rand((N,), 0.3, g), rand((M, N), 1, g)
    _, pre, _ = sv.spec_head_forward(x, w, b, act=sv.SPEC_ACT_GELU, want_pre=True)
    dx, dw, db, _ = sv.spec_head_backward(c, x, w, pre, act=sv.SPEC_ACT_GELU, want_db=True)
    X, W, Bv, C = f64(x), f64(w), f64(b), f64(c)
    loss = lambda X, W, Bv: float(np.sum(C * O.act(X @ W.T + Bv, "gelu")))   # noqa: E731
    h = 1e-5

    def diff(which, at):
        a = [X.copy(), W.copy(), Bv.copy()]
        a[which][at] += h
        up = loss(*a)
        a[which][at] -= 2 * h
        return (up - loss(*a)) / (2 * h)

    # pre and dz are rounded to bf16 (a slope changes by at most 1.2 per unit
    # of pre), the results once more
    z = X @ W.T + Bv
    td = HALF * (1.2 * np.abs(z) + 1.13) * np.abs(C) + 1e-6
    for at in ((0, 0), (2, 23)):
        t = float(td[at[0]] @ np.abs(W[:, at[1]]))
        assert abs(float(dx[at]) - diff(0, at)) <= t + HALF * (abs(diff(0, at)) + t) + 1e-6
    for at in ((0, 0), (39, 5)):
        t = float(td[:, at[0]] @ np.abs(X[:, at[1]]))
        assert abs(float(dw[at]) - diff(1, at)) <= t + HALF * (abs(diff(1, at)) + t) + 1e-6
    for at in (0, 39):
        assert abs(float(db[at]) - diff(2, at)) <= float(td[:, at].sum()) + 1e-6


def test_head_in_a_graph_and_on_another_stream():
    g = torch.Generator().manual_seed(5)
    x, w, dy = rand((50, 256), 1, g), rand((600, 256), 0.1, g), rand((50, 600), 1, g)
    y, _, ws = sv.spec_head_forward(x, w)
    dx, dw, _, wb = sv.spec_head_backward(dy, x, w)
    y2, dx2, dw2 = torch.empty_like(y), torch.empty_like(dx), torch.empty_like(dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_head_forward(x, w, out=(y2, None), workspace=ws)
        sv.spec_head_backward(dy, x, w, out=(dx2, dw2, None), workspace=wb)
    for _ in range(2):   # a replay leaves its counters as it found them
        for o in (y2, dx2, dw2):
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y3, _, _ = sv.spec_head_forward(x, w, stream=s)
    s.synchronize()
    assert torch.equal(y, y3)
