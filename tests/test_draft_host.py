"""CPU tests of the operators around a draft head: the header's functions are
exported, the refusals of the C ABI, and the 64-bit reference against
differences and closed forms."""
import ctypes

import numpy as np
import pytest

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


def test_exports_every_declared_function(L):
    names = sv.header_functions(sv.DRAFT_HEADER)
    assert set(names) == set(sv._DRAFT_SIGS)
    for n in names:
        assert hasattr(L, n), n


# ------------------------------------------------------------------- rules
RULES_OK = dict(logits=FAKE, dt=1, R=8, V=1000, cu=FAKE, B=2, max_rows=5, rules=None,
                out=FAKE + (1 << 20), ws=FAKE, ws_bytes=256, stream=None)


def rules(**kw):
    return ctypes.byref(D.SpecLogitsRules(**kw))


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), INV), (dict(V=0), INV), (dict(V=(1 << 24) + 1), INV), (dict(B=-1), INV),
    (dict(B=0), INV), (dict(dt=2), INV), (dict(max_rows=0), INV), (dict(max_rows=4097), INV),
    (dict(cu=None), INV), (dict(cu=FAKE + 2), INV), (dict(logits=None), INV),
    (dict(out=None), INV), (dict(logits=FAKE + 8), INV), (dict(out=FAKE + (1 << 20) + 4), INV),
    (dict(out=FAKE + 64), INV),                                    # overlaps the logits
    (dict(ws=None), WS), (dict(ws=FAKE + 16), WS), (dict(ws_bytes=255), WS),
    (dict(rules=dict(history=FAKE)), INV), (dict(rules=dict(cu_history=FAKE)), INV),
    (dict(rules=dict(prompt_len=FAKE)), INV), (dict(rules=dict(tokens=FAKE)), INV),
    (dict(rules=dict(cu_tokens=FAKE)), INV), (dict(rules=dict(parent=FAKE)), INV),
    (dict(rules=dict(parent=FAKE, tokens=FAKE, cu_tokens=FAKE)), INV),
    (dict(rules=dict(bias_ids=FAKE, bias_values=FAKE)), INV),
    (dict(rules=dict(bias_values=FAKE, cu_bias=FAKE)), INV),
    (dict(rules=dict(mask_rows=FAKE)), INV),
    (dict(rules=dict(mask=FAKE, n_mask=7)), INV),                  # fewer mask rows than rows
    (dict(rules=dict(mask=FAKE, n_mask=-1, mask_rows=FAKE)), INV),
    (dict(rules=dict(repetition=FAKE + 2)), INV),
])
def test_rules_refuses_bad_arguments(L, kw, code):
    a = dict(RULES_OK)
    a.update(kw)
    if a["rules"] is not None:
        a["rules"] = rules(**a["rules"])
    assert L.spec_process_logits(*a.values()) == code


# ----------------------------------------------------------------- distill
DISTILL_OK = dict(target=FAKE, draft=FAKE, dt=1, R=8, V=1000, cu=FAKE, B=2, temp=FAKE, weight=FAKE,
                  loss=FAKE, grad=FAKE, ws=FAKE, ws_bytes=256, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), INV), (dict(V=0), INV), (dict(B=-2), INV), (dict(B=0), INV), (dict(dt=7), INV),
    (dict(cu=None), INV), (dict(target=None), INV), (dict(draft=None), INV), (dict(loss=None), INV),
    (dict(target=FAKE + 4), INV), (dict(draft=FAKE + 2), INV), (dict(grad=FAKE + 8), INV),
    (dict(loss=FAKE + 1), INV), (dict(weight=FAKE + 2), INV), (dict(temp=FAKE + 2), INV),
    (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(ws_bytes=0), WS),
    (dict(R=(1 << 27) + 1, V=1), UNSUP),
])
def test_distill_refuses_bad_arguments(L, kw, code):
    a = dict(DISTILL_OK)
    a.update(kw)
    assert L.spec_distill_loss(*a.values()) == code


def test_distill_workspace():
    assert sv.spec_distill_loss_workspace(5, 100) >= 256
    assert sv.spec_distill_loss_workspace(-1, 100) == 0
    assert sv.spec_distill_loss_workspace(5, 0) == 0


# ------------------------------------------------------------------- AdamW
def tensor(**kw):
    a = dict(param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, n=10, dtype=0)
    a.update(kw)
    return D.SpecAdamwTensor(**a)


@pytest.mark.parametrize("kw,bits,code", [
    (dict(), 16, INV), (dict(n=-1), 32, INV), (dict(n=1 << 40), 32, INV), (dict(dtype=3), 32, INV),
    (dict(param=None), 32, INV), (dict(grad=None), 32, INV), (dict(exp_avg=None), 32, INV),
    (dict(exp_avg_sq=None), 32, INV), (dict(param=FAKE + 2), 32, INV), (dict(grad=FAKE + 1), 32, INV),
    (dict(exp_avg=FAKE + 2), 32, INV), (dict(master=FAKE), 32, INV),   # a master of f32 weights
    (dict(exp_avg_scale=FAKE), 32, INV), (dict(), 8, INV),             # scales missing
    (dict(exp_avg_scale=FAKE), 8, INV),
    (dict(n=(1 << 40) - 1), 32, sv.SPEC_OK),
])
def test_adamw_table_checks_its_tensors(L, kw, bits, code):
    rows = (D.SpecAdamwTensor * 1)(tensor(**kw))
    n = L.spec_adamw_table_bytes(rows, 1, bits)
    if code != sv.SPEC_OK:
        assert n == 0
        items = ctypes.c_int64(0)
        buf = ctypes.create_string_buffer(4096)
        assert L.spec_adamw_table(rows, 1, bits, buf, 4096, ctypes.byref(items)) == code
    else:
        assert n > 0


def test_adamw_table_counts_items(L):
    rows = (D.SpecAdamwTensor * 3)(tensor(n=1), tensor(n=0, param=None), tensor(n=8193))
    n = L.spec_adamw_table_bytes(rows, 3, 32)
    buf = ctypes.create_string_buffer(n + 16)
    at = (ctypes.addressof(buf) + 15) // 16 * 16
    items = ctypes.c_int64(0)
    assert L.spec_adamw_table(rows, 3, 32, at, n, ctypes.byref(items)) == sv.SPEC_OK
    assert items.value == 1 + 0 + 3
    assert L.spec_adamw_table(rows, 3, 32, at, n - 1, ctypes.byref(items)) == WS


HYPER_OK = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)


@pytest.mark.parametrize("kw,code", [
    (dict(lr=-1.0), INV), (dict(lr=float("nan")), INV), (dict(beta1=1.0), INV), (dict(beta2=-0.1), INV),
    (dict(eps=-1e-8), INV), (dict(weight_decay=float("inf")), INV), (dict(step=0), INV),
    (dict(grad_scale=FAKE + 1), INV), (dict(step_dev=FAKE + 2), INV)])
def test_adamw_step_refuses_bad_hyperparameters(L, kw, code):
    h = D.SpecAdamwHyper(**{**HYPER_OK, **kw})
    assert L.spec_adamw_step(FAKE, 1, 32, ctypes.byref(h), FAKE, 256, None) == code


@pytest.mark.parametrize("table,items,bits,ws,ws_bytes,code", [
    (None, 1, 32, FAKE, 256, INV), (FAKE + 8, 1, 32, FAKE, 256, INV), (FAKE, -1, 32, FAKE, 256, INV),
    (FAKE, 1, 4, FAKE, 256, INV), (FAKE, 1, 32, None, 256, WS), (FAKE, 1, 32, FAKE, 100, WS)])
def test_adamw_step_refuses_bad_arguments(L, table, items, bits, ws, ws_bytes, code):
    h = D.SpecAdamwHyper(**HYPER_OK)
    assert L.spec_adamw_step(table, items, bits, ctypes.byref(h), ws, ws_bytes, None) == code
    assert L.spec_adamw_step(FAKE, 1, 32, None, FAKE, 256, None) == INV


# ------------------------------------------------- the reference's own pins
def test_reference_gradient_against_differences():
    rng = np.random.default_rng(3)
    cu = np.array([0, 2, 5])
    t, d = rng.normal(size=(7, 11)), rng.normal(size=(5, 11))
    T, w = np.array([0.7, 1.4]), rng.random(5)
    _, grad, _ = O.distill(t, d, cu, T, w)
    h = 1e-6
    for r, x in ((0, 3), (2, 0), (4, 10)):
        up, dn = d.copy(), d.copy()
        up[r, x] += h
        dn[r, x] -= h
        diff = (O.distill(t, up, cu, T, w)[0][r] - O.distill(t, dn, cu, T, w)[0][r]) / (2 * h)
        assert abs(diff - grad[r, x]) < 1e-8    # h^2 of the third derivative, 1e-16 / h of rounding


def test_reference_rules_by_hand():
    z = np.array([[1.0, -2.0, 3.0, 0.5], [1.0, -2.0, 3.0, 0.5]])
    case = dict(history=np.array([0, 1, 1]), cu_history=np.array([0, 3]), prompt_len=np.array([1]),
                tokens=np.array([2]), cu_tokens=np.array([0, 1]), repetition=np.array([2.0]),
                frequency=np.array([0.25]), presence=np.array([0.5]),
                bias_ids=np.array([3, 3]), bias_values=np.array([9.0, 1.0]), cu_bias=np.array([0, 2]))
    out, _ = O.process_logits(z, [0, 2], case)
    assert np.allclose(out, [[0.5, -4 - 0.5 - 0.5, 3.0, 1.5], [0.5, -5.0, 1.5 - 0.75, 1.5]], atol=0, rtol=0)


def test_reference_e4m3_rounds_to_nearest_even():
    assert O.to_e4m3(np.array([448.0, 500.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == \
        [448.0, 448.0, 1.0, 1.25, 0.0, 2 * 2.0 ** -9]


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_reference_activation_slopes(name):
    z = np.linspace(-5, 5, 41)
    h = 1e-6
    diff = (O.act(z + h, name) - O.act(z - h, name)) / (2 * h)
    assert np.max(np.abs(diff - O.act_slope(z, name))) < 1e-8


# -------------------------------------------------------------------- head
FORWARD_OK = dict(x=FAKE, w=FAKE, bias=None, residual=None, M=4, N=64, K=64, act=0, y=FAKE, pre=None,
                  ws=FAKE, ws_bytes=1 << 30, stream=None)
BACKWARD_OK = dict(dy=FAKE, x=FAKE, w=FAKE, pre=FAKE, M=4, N=64, K=64, act=1, dx=FAKE, dw=FAKE, db=FAKE,
                   ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=(1 << 24) + 1), INV),
    (dict(act=3), INV), (dict(act=-1), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV),
    (dict(x=FAKE + 8), INV), (dict(w=FAKE + 2), INV), (dict(y=FAKE + 4), INV), (dict(bias=FAKE + 1), INV),
    (dict(ws=None), WS), (dict(ws=FAKE + 64), WS), (dict(ws_bytes=128), WS)])
def test_head_forward_refuses_bad_arguments(L, kw, code):
    assert L.spec_head_forward(*{**FORWARD_OK, **kw}.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(act=9), INV), (dict(dy=None), INV), (dict(pre=None), INV),
    (dict(w=None), INV), (dict(x=None), INV), (dict(dx=FAKE + 8), INV), (dict(dw=FAKE + 2), INV),
    (dict(db=FAKE + 2), INV), (dict(ws=None), WS), (dict(ws_bytes=256), WS)])
def test_head_backward_refuses_bad_arguments(L, kw, code):
    assert L.spec_head_backward(*{**BACKWARD_OK, **kw}.values()) == code


def test_head_workspaces():
    for f in (sv.spec_head_forward_workspace, sv.spec_head_backward_workspace):
        assert f(1, 32000, 4096) >= 256 and f(0, 10, 10) >= 256
        assert f(-1, 10, 10) == 0 and f(1, 0, 10) == 0 and f(1, 10, 0) == 0
    # padded copies of odd operands are part of it
    assert sv.spec_head_forward_workspace(4, 64, 63) >= 2 * 64 * (64 + 4)
