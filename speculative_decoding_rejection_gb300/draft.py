"""Binding of the operators around a draft head (include/specdraft.h): rules
on the logits, the distillation loss, the head's products and AdamW. As in
the package's other calls, the functions here only marshal arguments and raise
on a non-zero return code; the kernels of libspecverify.so do the work.
"""
from __future__ import annotations

import ctypes

import speculative_decoding_rejection_gb300 as _sv

SPEC_ADAMW_BLOCK = 256
SPEC_ACT_NONE, SPEC_ACT_SILU, SPEC_ACT_GELU = 0, 1, 2

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


class SpecLogitsRules(ctypes.Structure):
    """spec_logits_rules of include/specdraft.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("history", "cu_history", "prompt_len", "tokens", "cu_tokens", "parent",
                 "repetition", "frequency", "presence", "bias_ids", "bias_values", "cu_bias",
                 "mask", "mask_rows")] + [("n_mask", ctypes.c_int32)]


class SpecAdamwTensor(ctypes.Structure):
    """spec_adamw_tensor of include/specdraft.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale",
                 "master")] + [("n", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class SpecAdamwHyper(ctypes.Structure):
    """spec_adamw_hyper of include/specdraft.h."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("grad_scale", ctypes.c_void_p), ("lr_dev", ctypes.c_void_p),
        ("step_dev", ctypes.c_void_p)]


SIGS = {
    "spec_process_logits_workspace": (_sz, []),
    "spec_process_logits": (_i32, [_vp, _i32, _i32, _i32, _vp, _i32, _i32,
                                   ctypes.POINTER(SpecLogitsRules), _vp, _vp, _sz, _vp]),
    "spec_distill_loss_workspace": (_sz, [_i32, _i32]),
    "spec_distill_loss": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                 _sz, _vp]),
    "spec_adamw_table_bytes": (_sz, [ctypes.POINTER(SpecAdamwTensor), _i32, _i32]),
    "spec_adamw_table": (_i32, [ctypes.POINTER(SpecAdamwTensor), _i32, _i32, _vp, _sz,
                                ctypes.POINTER(_i64)]),
    "spec_head_forward_workspace": (_sz, [_i32, _i32, _i32]),
    "spec_head_forward": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "spec_head_backward_workspace": (_sz, [_i32, _i32, _i32]),
    "spec_head_backward": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz,
                                  _vp]),
    "spec_adamw_step": (_i32, [_vp, _i64, _i32, ctypes.POINTER(SpecAdamwHyper), _vp, _sz, _vp]),
}


def _want(name, t, dtype, numel=None, device=None):
    """A tensor of the dtype and size that the call reads; None passes."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, {numel} are needed")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")


def _begin(device, stream, tensors):
    """The stream of the call and a context in which its buffers are
    allocated. Where that is not torch's current stream, the tensors the
    caller made elsewhere are marked as in use there, so that their memory is
    not handed out before the call's work is done."""
    torch = _sv._torch()
    cur = torch.cuda.current_stream(device)
    s = cur if stream is None else stream
    if s != cur:
        for t in tensors:
            if t is not None:
                t.record_stream(s)
    return s, torch.cuda.stream(s)


def _bytes(t):
    return ctypes.c_size_t(t.numel() * t.element_size())


# ------------------------------------------------------- rules on the logits
def spec_process_logits_workspace() -> int:
    return int(_sv.lib().spec_process_logits_workspace())


def spec_process_logits(logits, cu_rows, *, max_rows: int, history=None, cu_history=None,
                        prompt_len=None, tokens=None, cu_tokens=None, parent=None,
                        repetition=None, frequency=None, presence=None, bias_ids=None,
                        bias_values=None, cu_bias=None, mask=None, mask_rows=None,
                        workspace=None, out=None, stream=None):
    """Repetition, frequency and presence penalties, biases and grammar masks
    on the rows of a linear batch (tokens, cu_tokens: the drafts) or of trees
    (tokens, parent: the nodes). Pass out=logits to work in place. See
    include/specdraft.h for the semantics.

    Returns (out [R, V], workspace).
    """
    torch = _sv._torch()
    R, V = logits.shape
    B = cu_rows.numel() - 1
    dev = logits.device
    i32, f32 = torch.int32, torch.float32
    _want("cu_rows", cu_rows, i32, 1, dev)
    _want("history", history, i32, None, dev)
    _want("cu_history", cu_history, i32, B + 1, dev)
    _want("prompt_len", prompt_len, i32, B, dev)
    _want("tokens", tokens, i32, R if parent is not None else None, dev)
    _want("cu_tokens", cu_tokens, i32, B + 1, dev)
    _want("parent", parent, i32, R, dev)
    _want("repetition", repetition, f32, B, dev)
    _want("frequency", frequency, f32, B, dev)
    _want("presence", presence, f32, B, dev)
    _want("bias_ids", bias_ids, i32, None, dev)
    _want("bias_values", bias_values, f32, bias_ids.numel() if bias_ids is not None else None, dev)
    _want("cu_bias", cu_bias, i32, B + 1, dev)
    _want("mask_rows", mask_rows, i32, R, dev)
    _want("out", out, logits.dtype, R * V, dev)
    if mask is not None:
        _want("mask", mask, i32, None, dev)
        if mask.dim() != 2 or mask.shape[1] != (V + 31) // 32:
            raise ValueError(f"mask must be [n, {(V + 31) // 32}] int32 words")
    ptr = _sv._ptr
    rules = SpecLogitsRules(
        ptr(history), ptr(cu_history), ptr(prompt_len), ptr(tokens), ptr(cu_tokens), ptr(parent),
        ptr(repetition), ptr(frequency), ptr(presence), ptr(bias_ids), ptr(bias_values),
        ptr(cu_bias), ptr(mask), ptr(mask_rows), 0 if mask is None else mask.shape[0])
    # an empty list has no address: without entries the step is left out
    for names in (("history", "cu_history", "prompt_len"), ("tokens", "cu_tokens", "parent"),
                  ("bias_ids", "bias_values", "cu_bias")):
        first = dict(history=history, tokens=tokens, bias_ids=bias_ids)[names[0]]
        if first is not None and first.numel() == 0:
            for n in names:
                setattr(rules, n, None)
    if mask is not None and mask.numel() == 0 and mask_rows is not None:
        rules.mask = rules.mask_rows = None
        rules.n_mask = 0
    s, ctx = _begin(dev, stream, (logits, cu_rows, history, cu_history, prompt_len, tokens,
                                  cu_tokens, parent, repetition, frequency, presence, bias_ids,
                                  bias_values, cu_bias, mask, mask_rows, workspace, out))
    with ctx:
        ws = _sv._workspace(256, dev, workspace)
        if out is None:
            out = torch.empty_like(logits)
        code = _sv.lib().spec_process_logits(
            ptr(logits), _sv._dtype_code(logits), R, V, ptr(cu_rows), B, int(max_rows),
            ctypes.byref(rules), ptr(out), ptr(ws), _bytes(ws), _sv._stream(s))
    _sv._check(code, "spec_process_logits")
    return out, ws


# ------------------------------------------------------- distillation loss
def spec_distill_loss_workspace(R_d: int, V: int) -> int:
    return int(_sv.lib().spec_distill_loss_workspace(R_d, V))


def spec_distill_loss(target, draft, cu_draft, temperature=None, weight=None, *, want_grad=True,
                      workspace=None, out=None, stream=None):
    """The weighted KL(p || q) of every draft position and its gradient with
    respect to the draft logits. See include/specdraft.h for the semantics.

    Returns (loss [R_d] f32, grad [R_d, V] or None, workspace).
    """
    torch = _sv._torch()
    R, V = draft.shape
    B = cu_draft.numel() - 1
    dev = draft.device
    if target.dtype != draft.dtype:
        raise TypeError("target and draft logits must have the same type")
    if target.shape[1] != V or target.shape[0] < R + B:
        raise ValueError(f"target must be [{R + B}, {V}] logits")
    _want("target", target, draft.dtype, None, dev)
    _want("cu_draft", cu_draft, torch.int32, 1, dev)
    _want("temperature", temperature, torch.float32, B, dev)
    _want("weight", weight, torch.float32, R, dev)
    loss, grad = (None, None) if out is None else out
    _want("loss", loss, torch.float32, R, dev)
    _want("grad", grad, draft.dtype, R * V, dev)
    ptr = _sv._ptr
    s, ctx = _begin(dev, stream, (target, draft, cu_draft, temperature, weight, workspace, loss,
                                  grad))
    with ctx:
        ws = _sv._workspace(256, dev, workspace)
        if out is None:
            loss = torch.empty(R, dtype=torch.float32, device=dev)
            grad = torch.empty_like(draft) if want_grad else None
        code = _sv.lib().spec_distill_loss(
            ptr(target), ptr(draft), _sv._dtype_code(draft), R, V, ptr(cu_draft), B,
            ptr(temperature), ptr(weight), ptr(loss), ptr(grad), ptr(ws), _bytes(ws),
            _sv._stream(s))
    _sv._check(code, "spec_distill_loss")
    return loss, grad, ws


# --------------------------------------------------------- a head's products
def spec_head_forward_workspace(M: int, N: int, K: int) -> int:
    return int(_sv.lib().spec_head_forward_workspace(M, N, K))


def spec_head_backward_workspace(M: int, N: int, K: int) -> int:
    return int(_sv.lib().spec_head_backward_workspace(M, N, K))


def _head_sizes(x, weight):
    torch = _sv._torch()
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"weight must be [N, {K}]")
    _want("x", x, torch.bfloat16)
    _want("weight", weight, torch.bfloat16, None, x.device)
    return M, N, K


def _head_workspace(size, where, device, workspace):
    if workspace is not None:
        return workspace
    if size == 0:
        raise _sv.SpecError(_sv.SPEC_ERR_INVALID_ARG, where)
    return _sv._workspace(size, device)


def spec_head_forward(x, weight, bias=None, residual=None, *, act: int = SPEC_ACT_NONE,
                      want_pre=False, workspace=None, out=None, stream=None):
    """y = act(x weight^T + bias) + residual in bf16, x [M, K], weight [N, K].
    With `want_pre` the pre-activation is returned too, for
    spec_head_backward. See include/specdraft.h.

    Returns (y [M, N], pre [M, N] or None, workspace).
    """
    torch = _sv._torch()
    M, N, K = _head_sizes(x, weight)
    dev, bf = x.device, torch.bfloat16
    _want("bias", bias, bf, N, dev)
    _want("residual", residual, bf, M * N, dev)
    y, pre = (None, None) if out is None else out
    _want("y", y, bf, M * N, dev)
    _want("pre", pre, bf, M * N, dev)
    ptr = _sv._ptr
    s, ctx = _begin(dev, stream, (x, weight, bias, residual, y, pre, workspace))
    with ctx:
        ws = _head_workspace(0 if workspace is not None else spec_head_forward_workspace(M, N, K),
                             "spec_head_forward_workspace", dev, workspace)
        if out is None:
            y = torch.empty(M, N, dtype=bf, device=dev)
            pre = torch.empty_like(y) if want_pre else None
        code = _sv.lib().spec_head_forward(
            ptr(x), ptr(weight), ptr(bias), ptr(residual), M, N, K, act, ptr(y), ptr(pre), ptr(ws),
            _bytes(ws), _sv._stream(s))
    _sv._check(code, "spec_head_forward")
    return y, pre, ws


def spec_head_backward(dy, x, weight, pre=None, *, act: int = SPEC_ACT_NONE, want_dx=True,
                       want_dw=True, want_db=False, workspace=None, out=None, stream=None):
    """The gradients of spec_head_forward given dy [M, N]; `pre` is the
    pre-activation it returned (not needed without an activation). See
    include/specdraft.h.

    Returns (dx [M, K], dw [N, K], db [N] f32, workspace), None for what is
    not wanted.
    """
    torch = _sv._torch()
    M, N, K = _head_sizes(x, weight)
    dev, bf = x.device, torch.bfloat16
    if tuple(dy.shape) != (M, N):
        raise ValueError(f"dy must be [{M}, {N}]")
    _want("dy", dy, bf, M * N, dev)
    _want("pre", pre, bf, M * N, dev)
    dx, dw, db = (None, None, None) if out is None else out
    _want("dx", dx, bf, M * K, dev)
    _want("dw", dw, bf, N * K, dev)
    _want("db", db, torch.float32, N, dev)
    ptr = _sv._ptr
    s, ctx = _begin(dev, stream, (dy, x, weight, pre, dx, dw, db, workspace))
    with ctx:
        ws = _head_workspace(0 if workspace is not None else spec_head_backward_workspace(M, N, K),
                             "spec_head_backward_workspace", dev, workspace)
        if out is None:
            dx = torch.empty(M, K, dtype=bf, device=dev) if want_dx else None
            dw = torch.empty(N, K, dtype=bf, device=dev) if want_dw else None
            db = torch.empty(N, dtype=torch.float32, device=dev) if want_db else None
        code = _sv.lib().spec_head_backward(
            ptr(dy), ptr(x), ptr(weight), ptr(pre), M, N, K, act, ptr(dx), ptr(dw), ptr(db), ptr(ws),
            _bytes(ws), _sv._stream(s))
    _sv._check(code, "spec_head_backward")
    return dx, dw, db, ws


# ------------------------------------------------------------------- AdamW
class SpecAdamwTable:
    """The device table of spec_adamw_table, with the tensors it names."""

    def __init__(self, data, n_items, state_bits, tensors):
        self.data, self.n_items, self.state_bits, self.tensors = data, n_items, state_bits, tensors


def spec_adamw_table(params, grads, exp_avg, exp_avg_sq, *, exp_avg_scale=None,
                     exp_avg_sq_scale=None, master=None) -> SpecAdamwTable:
    """The table of tensors that spec_adamw_step goes by, built once: lists of
    weights (f32 or bf16), their gradients (the same type), and states. States
    are f32 tensors, or torch.float8_e4m3fn (or uint8) codes with lists of f32
    scales, one per SPEC_ADAMW_BLOCK elements. `master` lists f32 copies of
    bf16 weights (entries may be None). The tensors' addresses must stay as
    they are while the table is used."""
    torch = _sv._torch()
    n = len(params)
    if not (len(grads) == len(exp_avg) == len(exp_avg_sq) == n):
        raise ValueError("params, grads and states must be lists of the same length")
    for name, extra in (("exp_avg_scale", exp_avg_scale), ("exp_avg_sq_scale", exp_avg_sq_scale),
                        ("master", master)):
        if extra is not None and len(extra) != n:
            raise ValueError(f"{name} must be a list of the same length")
    if n == 0:
        raise ValueError("no tensors")
    dev = params[0].device
    codes = (torch.float8_e4m3fn, torch.uint8)
    bits = 8 if exp_avg[0].dtype in codes else 32
    pick = lambda xs, i: None if xs is None else xs[i]   # noqa: E731
    rows = (SpecAdamwTensor * n)()
    for i in range(n):
        p, g, m, v = params[i], grads[i], exp_avg[i], exp_avg_sq[i]
        ms, vs, w = pick(exp_avg_scale, i), pick(exp_avg_sq_scale, i), pick(master, i)
        size = p.numel()
        blocks = -(-size // SPEC_ADAMW_BLOCK)
        _want(f"grads[{i}]", g, p.dtype, size, dev)
        for name, s in (("exp_avg", m), ("exp_avg_sq", v)):
            if s.dtype not in (codes if bits == 8 else (torch.float32,)):
                raise TypeError(f"{name}[{i}] must hold states of {bits} bits, got {s.dtype}")
            _want(f"{name}[{i}]", s, s.dtype, size, dev)
        _want(f"exp_avg_scale[{i}]", ms, torch.float32, blocks, dev)
        _want(f"exp_avg_sq_scale[{i}]", vs, torch.float32, blocks, dev)
        _want(f"master[{i}]", w, torch.float32, size, dev)
        rows[i] = SpecAdamwTensor(*(x if x is None else x.value for x in map(
            _sv._ptr, (p, g, m, v, ms, vs, w))), size, _sv._dtype_code(p))
    L = _sv.lib()
    nbytes = L.spec_adamw_table_bytes(rows, n, bits)
    if nbytes == 0:
        raise _sv.SpecError(_sv.SPEC_ERR_INVALID_ARG, "spec_adamw_table_bytes")
    host = torch.empty(nbytes, dtype=torch.uint8)
    items = ctypes.c_int64(0)
    _sv._check(L.spec_adamw_table(rows, n, bits, host.data_ptr(), nbytes, ctypes.byref(items)),
               "spec_adamw_table")
    keep = (list(params), list(grads), list(exp_avg), list(exp_avg_sq), exp_avg_scale,
            exp_avg_sq_scale, master)
    return SpecAdamwTable(host.to(dev), items.value, bits, keep)


def spec_adamw_step(table, step: int = 1, *, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                    eps: float = 1e-8, weight_decay: float = 0.01, grad_scale=None, lr_dev=None,
                    step_dev=None, workspace=None, stream=None):
    """One AdamW step over the tensors of `table`, in place. `grad_scale`,
    `lr_dev` (f32) and `step_dev` (int32) are one-element device tensors read
    when the kernel runs. See include/specdraft.h for the semantics. Returns
    the workspace."""
    torch = _sv._torch()
    dev = table.data.device
    _want("grad_scale", grad_scale, torch.float32, 1, dev)
    _want("lr_dev", lr_dev, torch.float32, 1, dev)
    _want("step_dev", step_dev, torch.int32, 1, dev)
    ptr = _sv._ptr
    hyper = SpecAdamwHyper(lr, beta1, beta2, eps, weight_decay, int(step), ptr(grad_scale),
                           ptr(lr_dev), ptr(step_dev))
    used = [table.data, grad_scale, lr_dev, step_dev, workspace]
    if stream is not None:
        used += [t for group in table.tensors if group is not None for t in group]
    s, ctx = _begin(dev, stream, used)
    with ctx:
        ws = _sv._workspace(256, dev, workspace)
        code = _sv.lib().spec_adamw_step(
            ptr(table.data), table.n_items, table.state_bits, ctypes.byref(hyper), ptr(ws),
            _bytes(ws), _sv._stream(s))
    _sv._check(code, "spec_adamw_step")
    return ws
