"""CPU tests of sampling, the 4-bit head and the gradients' norm: the refusals of the
C ABI and of the binding, and pins of their 64-bit reference."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from speculative_decoding_rejection_gb300 import draft as D
from oracle import draft_oracle as O

FAKE = 1 << 20   # a 256-byte-aligned non-null value; never dereferenced
INV, WS, UNSUP = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_WORKSPACE, sv.SPEC_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    try:
        return sv.lib()
    except RuntimeError as e:
        pytest.fail(f"library not built: {e}")


# ---------------------------------------------------------------- sampling
SAMPLE_OK = dict(logits=FAKE, dt=1, R=4, V=1000, cu=FAKE, B=2, params=None, uniform=FAKE, tokens=FAKE,
                 prob=FAKE, kept=FAKE, filtered=FAKE + (1 << 20), ws=FAKE, ws_bytes=256, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), INV), (dict(V=0), INV), (dict(V=(1 << 24) + 1), INV), (dict(B=-1), INV), (dict(B=0), INV),
    (dict(dt=2), INV), (dict(cu=None), INV), (dict(cu=None, B=5), INV), (dict(logits=None), INV),
    (dict(R=(1 << 27) + 1), INV), (dict(logits=FAKE + 8), INV), (dict(filtered=FAKE + 4), INV),
    (dict(filtered=FAKE + 64), INV),                           # overlaps the logits
    (dict(uniform=None), INV), (dict(uniform=None, tokens=None), INV), (dict(tokens=None), INV),
    (dict(uniform=FAKE + 2), INV), (dict(kept=FAKE + 1), INV), (dict(cu=FAKE + 2), INV),
    (dict(params=dict(temperature=FAKE + 2)), INV), (dict(params=dict(top_k=FAKE + 1)), INV),
    (dict(params=dict(top_p=FAKE + 3)), INV), (dict(params=dict(min_p=FAKE + 2)), INV),
    (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(ws_bytes=255), WS)])
def test_sample_refuses_bad_arguments(L, kw, code):
    a = {**SAMPLE_OK, **kw}
    if a["params"] is not None:
        a["params"] = ctypes.byref(D.SpecSampling(**a["params"]))
    assert L.spec_sample(*a.values()) == code


def test_sample_workspace():
    assert sv.spec_sample_workspace(3, 100) >= 256 and sv.spec_sample_workspace(0, 1) >= 256
    assert sv.spec_sample_workspace(-1, 100) == 0 and sv.spec_sample_workspace(1, 0) == 0


def test_sample_refuses_host_tensors():
    with pytest.raises(ValueError):
        sv.spec_sample(torch.zeros(2, 8), torch.zeros(2))


# --------------------------------------------------------------- 4-bit head
HEAD4_OK = dict(x=FAKE, packed=FAKE, zeros=0, bias=None, residual=None, M=4, N=64, K=64, group=32, act=0,
                y=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=(1 << 24) + 1), INV),
    (dict(M=sv.SPEC_HEAD4_MAX_ROWS + 1), UNSUP), (dict(group=16), INV), (dict(group=48), INV),
    (dict(group=256), INV), (dict(act=3), INV), (dict(x=None), INV), (dict(packed=None), INV),
    (dict(y=None), INV), (dict(x=FAKE + 8), INV), (dict(packed=FAKE + 4), INV),
    (dict(bias=FAKE + 1), INV), (dict(y=FAKE + 1), INV), (dict(ws=None), WS), (dict(ws=FAKE + 64), WS),
    (dict(ws_bytes=8), WS), (dict(M=64, K=8192, ws_bytes=256), WS)])
def test_head4_forward_refuses_bad_arguments(L, kw, code):
    assert L.spec_head4_forward(*{**HEAD4_OK, **kw}.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(group=96), INV),
    (dict(packed=None), INV), (dict(packed=FAKE + 8), INV), (dict(scales=FAKE + 1), INV),
    (dict(N=1 << 24, K=1 << 24), UNSUP)])
def test_head4_pack_refuses_bad_arguments(L, kw, code):
    a = dict(codes=FAKE, scales=FAKE, zeros=None, N=4, K=64, group=32, packed=FAKE, stream=None)
    assert L.spec_head4_pack(*{**a, **kw}.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), INV), (dict(w=FAKE + 1), INV), (dict(N=0), INV), (dict(group=100), INV),
    (dict(packed=FAKE + 2), INV), (dict(ws=None), WS), (dict(ws_bytes=0), WS)])
def test_head4_quantize_refuses_bad_arguments(L, kw, code):
    a = dict(w=FAKE, N=4, K=64, group=32, packed=FAKE, ws=FAKE, ws_bytes=256, stream=None)
    assert L.spec_head4_quantize(*{**a, **kw}.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(packed=None), INV), (dict(out=None), INV), (dict(group=0), INV), (dict(out=FAKE + 1), INV),
    (dict(K=-3), INV)])
def test_head4_unpack_refuses_bad_arguments(L, kw, code):
    a = dict(packed=FAKE, zeros=0, N=4, K=64, group=32, out=FAKE, stream=None)
    assert L.spec_head4_unpack(*{**a, **kw}.values()) == code


def test_head4_sizes(L):
    size = L.spec_head4_packed_bytes      # two blocks of 16 rows and 128 columns, scales and zeros behind each
    assert size(3, 1, 128, 0) == 2 * (1024 + 32) and size(33, 129, 32, 0) == 8 * (1024 + 128)
    assert size(32, 128, 64, 1) == 2 * (1024 + 64 + 32) and size(0, 8, 32, 0) == 0 and size(8, 8, 8, 0) == 0
    assert sv.spec_head4_forward_workspace(0, 4, 4) >= 256
    assert sv.spec_head4_forward_workspace(65, 4, 4) == 0


# ------------------------------------------------------- the gradients' norm
NORM_OK = dict(table=FAKE, n_items=1, bits=32, inf=0, max_norm=1.0, grad_scale=None, out=FAKE, ws=FAKE,
               ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), INV), (dict(table=FAKE + 8), INV), (dict(n_items=-1), INV), (dict(bits=16), INV),
    (dict(max_norm=0.0), INV), (dict(max_norm=-1.0), INV), (dict(max_norm=float("nan")), INV),
    (dict(out=None), INV), (dict(out=FAKE + 2), INV), (dict(grad_scale=FAKE + 1), INV),
    (dict(grad_scale=FAKE), INV), (dict(grad_scale=FAKE + 4), INV),      # is `out`
    (dict(ws=None), WS), (dict(ws=FAKE + 16), WS), (dict(ws_bytes=256), WS)])
def test_norm_refuses_bad_arguments(L, kw, code):
    for f in (L.spec_grad_norm, L.spec_clip_grads):
        assert f(*{**NORM_OK, **kw}.values()) == code


def test_norm_refuses_gradients_that_moved():
    p = torch.zeros(4, requires_grad=True)
    p.grad = torch.ones(4)
    table = D.SpecAdamwTable(None, 1, 32, ([p], [p.grad], [], []))
    p.grad = None
    for f in (sv.spec_grad_norm, sv.spec_clip_grads):
        with pytest.raises(ValueError, match="gradient"):
            f(table, max_norm=1.0)


# ------------------------------------------------------- the reference's pins
def test_reference_sample_by_hand():
    # weights 4, 2, 1, 1 of 8 in the order 2, 0, 1, 3 (equal ones by id)
    z = np.log([2.0, 1.0, 4.0, 1.0])
    r = O.sample_row(z, 0.5)
    assert r["order"].tolist() == [2, 0, 1, 3] and np.allclose(r["law"], [0.5, 0.25, 0.125, 0.125])
    tokens = [O.sample_row(z, u)["token"] for u in (0.0, 0.49, 0.51, 0.74, 0.76, 0.87, 0.88, 0.99)]
    assert tokens == [2, 2, 0, 0, 1, 1, 3, 3]
    assert O.sample_row(z, 0.99, top_k=3)["order"].tolist() == [2, 0, 1]
    assert O.sample_row(z, 0.99, top_p=0.6)["order"].tolist() == [2, 0]
    assert O.sample_row(z, 0.0, top_p=0.0)["order"].tolist() == [2]
    assert O.sample_row(z, 0.0, min_p=0.3)["order"].tolist() == [2, 0]
    assert O.sample_row(z, 0.9, T=0.04)["token"] == 2
    # top-p's fraction is of what top-k left: 4 of 6 reach 0.6, of 8 they would not
    assert O.sample_row(z, 0.0, top_k=2, top_p=0.6)["order"].tolist() == [2]
    masked = np.array([-np.inf, 0.0, -np.inf, 0.0])
    assert [O.sample_row(masked, u)["token"] for u in (0.4, 0.6)] == [1, 3]


def test_reference_sample_law_over_the_lattice_of_u():
    rng = np.random.default_rng(0)
    z = rng.normal(size=50) * 2
    n = 4000
    drawn = np.bincount([O.sample_row(z, (i + 0.5) / n, T=0.8, top_p=0.9)["token"] for i in range(n)], minlength=50)
    r = O.sample_row(z, 0.0, T=0.8, top_p=0.9)
    want = np.zeros(50)
    want[r["order"]] = r["law"]
    assert np.abs(drawn / n - want).max() <= 1.0 / n   # each token's run of the lattice


def test_reference_quantize_by_hand():
    w = np.array([[7.0, 3.5, -7.0, 2.5, -2.5, 0.25, 0.0, 6.4]])
    codes, scales = O.quantize4(w, 32)
    assert scales.tolist() == [[1.0]]
    assert codes.tolist() == [[15, 12, 1, 10, 6, 8, 8, 14]]       # ties to even: 3.5 to 4, 2.5 to 2
    assert O.dequantize4(codes, scales, None, 32).tolist() == [[7, 4, -7, 2, -2, 0, 0, 6]]
    assert O.to_bf16(np.array([1 + 2 ** -8, 1 + 3 * 2.0 ** -8, 0.1])).tolist() == [1.0, 1 + 2.0 ** -6, 0.10009765625]


def test_reference_norm_by_hand():
    n, f = O.grad_norm([np.array([3.0, 0.0]), np.array([[4.0]])], 1.0, 0.5)
    assert n == 2.5 and abs(f - 0.5 / 2.500001) < 1e-15
    assert O.grad_norm([np.array([3.0, -4.0])], 1e9, inf=True) == (4.0, 1.0)
