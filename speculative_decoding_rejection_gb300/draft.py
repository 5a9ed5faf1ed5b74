"""Binding of the operators around a draft head (include/specdraft.h): rules
on the logits, the distillation loss, the head's products and AdamW. As in
the package's other calls, the functions here only marshal arguments and raise
on a non-zero return code; the kernels of libspecverify.so do the work.
"""
from __future__ import annotations

import ctypes
import struct

import torch

import speculative_decoding_rejection_gb300 as _sv

# the current stream's handle without a Stream object (less host time per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

SPEC_ADAMW_BLOCK = 256
_INT_MAX = 0x7fffffff
SPEC_ACT_NONE, SPEC_ACT_SILU, SPEC_ACT_GELU = 0, 1, 2

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


class SpecLogitsRules(ctypes.Structure):
    """spec_logits_rules of include/specdraft.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("history", "cu_history", "prompt_len", "tokens", "cu_tokens", "parent",
                 "repetition", "frequency", "presence", "bias_ids", "bias_values", "cu_bias",
                 "mask", "mask_rows")] + [(n, ctypes.c_int32) for n in
                                          ("n_mask", "n_history", "n_tokens", "n_bias")]


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


# the two records as they lie in memory, for calls (less host time than a
# Structure's fields)
_RULES = struct.Struct("@14P4i")
_HYPER = struct.Struct("@5dq3P")
assert _RULES.size == ctypes.sizeof(SpecLogitsRules)
assert _HYPER.size == ctypes.sizeof(SpecAdamwHyper)

SIGS = {
    "spec_process_logits_workspace": (_sz, []),
    "spec_process_logits": (_i32, [_vp, _i32, _i32, _i32, _vp, _i32, _i32,
                                   _vp, _vp, _vp, _sz, _vp]),
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
    "spec_adamw_step": (_i32, [_vp, _i64, _i32, _vp, _vp, _sz, _vp]),
}


def _arg(name, t, dtype, numel, dev):
    """The address of a tensor the call reads or writes (None passes): of the
    dtype, at least that many elements, contiguous, on device `dev`."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and (not numel or t.numel() >= numel) and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _sv._ptr(t)   # raises for a host tensor and for one that is not contiguous
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{dev}")
    raise ValueError(f"{name} has {t.numel()} elements, {numel} are needed")


def _matrix(name, t, dtype, rows, width, dev):
    """The address of `rows` rows of `width` elements: a flat buffer, or a tensor
    whose trailing dimensions make up a row."""
    if t is not None:
        shape = t.shape
        if shape and shape[-1] != width and len(shape) > 1:
            row = 1
            for n in reversed(shape):
                row *= n
                if row == width:
                    break
            else:
                raise ValueError(f"{name} must have rows of {width} elements, its shape is {tuple(shape)}")
    return _arg(name, t, dtype, rows * width, dev)


def _device(name, t):
    """The CUDA device index of the call's first tensor."""
    dev = t.get_device()
    if dev < 0:
        _sv._ptr(t)   # raises
        raise ValueError(f"{name} must live on a CUDA device")
    return dev


class _Call:
    """The stream of a call, as a context in which its buffers are allocated and
    its device is the current one (the default stream's handle is the same on
    every device). Where the stream is not torch's current stream, the tensors
    the caller made elsewhere are marked as in use there, so that their memory
    is not handed out before the call's work is done."""

    __slots__ = ("raw", "ctx")

    def __init__(self, dev, stream, tensors):
        self.ctx = None
        if stream is None:
            if _current_device() != dev:
                self.ctx = torch.cuda.device(dev)
            self.raw = torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None \
                else _raw_stream(dev)
            return
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the call runs on cuda:{dev}")
        self.raw = stream.cuda_stream
        if stream != torch.cuda.current_stream(dev):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        self.ctx = torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self

    def __exit__(self, *e):
        if self.ctx is not None:
            self.ctx.__exit__(*e)


def _scratch(size, dev, workspace):
    """(workspace, address, bytes); one of `size` bytes where the caller has none."""
    if workspace is None:
        workspace = torch.empty(max(size, 256), dtype=torch.uint8, device=f"cuda:{dev}")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _sv._ptr(workspace)
        raise ValueError("the workspace is on another device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _f32_or_bf16(t):
    d = t.dtype
    return _sv.SPEC_BF16 if d is torch.bfloat16 else _sv.SPEC_F32 if d is torch.float32 \
        else _sv._dtype_code(t)


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
    R, V = logits.shape
    B = cu_rows.numel() - 1
    dev = _device("logits", logits)
    i32, f32 = torch.int32, torch.float32
    n_mask = 0
    if mask is not None:
        n_mask, words = mask.shape
        if words != (V + 31) // 32:
            raise ValueError(f"mask must be [n, {(V + 31) // 32}] int32 words")
        if mask_rows is None and n_mask < R:
            raise ValueError(f"mask has {n_mask} rows, the logits {R}")
    cu_history_at = _arg("cu_history", cu_history, i32, B + 1, dev) or 0
    cu_tokens_at = _arg("cu_tokens", cu_tokens, i32, B + 1, dev) or 0
    cu_bias_at = _arg("cu_bias", cu_bias, i32, B + 1, dev) or 0
    # an empty list has no address: its offsets' stands for it, unread (entries: -1)
    history_at = n_history = tokens_at = n_tokens = bias_at = n_bias = 0
    if history is not None:
        n_history = history.numel()
        if n_history:
            history_at = _arg("history", history, i32, 0, dev)
        else:
            history_at, n_history = cu_history_at, -1
    if parent is not None:
        tokens_at, n_tokens = _arg("tokens", tokens, i32, R, dev) or 0, R
    elif tokens is not None:
        n_tokens = tokens.numel()
        if n_tokens:
            tokens_at = _arg("tokens", tokens, i32, 0, dev)
        else:
            tokens_at, n_tokens = cu_tokens_at, -1
    if bias_ids is not None:
        n_bias = bias_ids.numel()
    if n_bias or bias_ids is None:
        bias_at = _arg("bias_ids", bias_ids, i32, 0, dev) or 0
        values_at = _arg("bias_values", bias_values, f32, n_bias, dev) or 0
    else:
        bias_at = values_at = cu_bias_at
        n_bias = -1
    if n_history + n_tokens + n_bias > _INT_MAX:   # a list may be longer than offsets reach
        n_history, n_tokens, n_bias = (min(n, _INT_MAX) for n in (n_history, n_tokens, n_bias))
    mask_rows_at = _arg("mask_rows", mask_rows, i32, R, dev) or 0
    mask_at = _arg("mask", mask, i32, 0, dev) or 0
    if mask_at == 0 and mask is not None:   # no rows: an address that is not read
        mask_at = mask_rows_at
    rules = _RULES.pack(
        history_at, cu_history_at,
        0 if history is not None and not history_at else _arg("prompt_len", prompt_len, i32, B, dev) or 0,
        tokens_at, cu_tokens_at,
        _arg("parent", parent, i32, R, dev) or 0,
        _arg("repetition", repetition, f32, B, dev) or 0,
        _arg("frequency", frequency, f32, B, dev) or 0,
        _arg("presence", presence, f32, B, dev) or 0,
        bias_at, values_at, cu_bias_at,
        mask_at, mask_rows_at, n_mask, n_history, n_tokens, n_bias)
    used = () if stream is None else (
        logits, cu_rows, history, cu_history, prompt_len, tokens, cu_tokens, parent, repetition,
        frequency, presence, bias_ids, bias_values, cu_bias, mask, mask_rows, workspace, out)
    with _Call(dev, stream, used) as call:
        ws, ws_at, ws_bytes = _scratch(256, dev, workspace)
        if out is None:
            out = torch.empty_like(logits, memory_format=torch.contiguous_format)
        code = _sv.lib().spec_process_logits(
            _arg("logits", logits, logits.dtype, 0, dev), _f32_or_bf16(logits), R, V,
            _arg("cu_rows", cu_rows, i32, 1, dev), B, max_rows, rules,
            _matrix("out", out, logits.dtype, R, V, dev), ws_at, ws_bytes, call.raw)
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
    R, V = draft.shape
    B = cu_draft.numel() - 1
    dev, dt, f32 = _device("draft", draft), draft.dtype, torch.float32
    if target.dtype is not dt:
        raise TypeError("target and draft logits must have the same type")
    if target.shape[1] != V or target.shape[0] < R + B:
        raise ValueError(f"target must be [{R + B}, {V}] logits")
    loss, grad = (None, None) if out is None else out
    with _Call(dev, stream, (target, draft, cu_draft, temperature, weight, workspace, loss,
                             grad)) as call:
        ws, ws_at, ws_bytes = _scratch(
            0 if workspace is not None else spec_distill_loss_workspace(R, V), dev, workspace)
        if out is None:
            loss = torch.empty(R, dtype=f32, device=draft.device)
            grad = torch.empty_like(draft, memory_format=torch.contiguous_format) if want_grad else None
        code = _sv.lib().spec_distill_loss(
            _arg("target", target, dt, 0, dev), _arg("draft", draft, dt, 0, dev),
            _f32_or_bf16(draft), R, V, _arg("cu_draft", cu_draft, torch.int32, 1, dev), B,
            _arg("temperature", temperature, f32, B, dev), _arg("weight", weight, f32, R, dev),
            _arg("loss", loss, f32, R, dev), _matrix("grad", grad, dt, R, V, dev), ws_at, ws_bytes,
            call.raw)
    _sv._check(code, "spec_distill_loss")
    return loss, grad, ws


# --------------------------------------------------------- a head's products
def spec_head_forward_workspace(M: int, N: int, K: int) -> int:
    return int(_sv.lib().spec_head_forward_workspace(M, N, K))


def spec_head_backward_workspace(M: int, N: int, K: int) -> int:
    return int(_sv.lib().spec_head_backward_workspace(M, N, K))


def _head_sizes(x, weight):
    M, K = x.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"weight must be [N, {K}]")
    return M, N, K


def _head_workspace(query, M, N, K, workspace):
    """What a call without a workspace of its own has to allocate."""
    if workspace is not None:
        return 0
    size = query(M, N, K)
    if size == 0:
        raise _sv.SpecError(_sv.SPEC_ERR_INVALID_ARG, query.__name__)
    return size


def spec_head_forward(x, weight, bias=None, residual=None, *, act: int = SPEC_ACT_NONE,
                      want_pre=False, workspace=None, out=None, stream=None):
    """y = act(x weight^T + bias) + residual in bf16, x [M, K], weight [N, K].
    With `want_pre` the pre-activation is returned too, for
    spec_head_backward. See include/specdraft.h.

    Returns (y [M, N], pre [M, N] or None, workspace).
    """
    M, N, K = _head_sizes(x, weight)
    dev, bf = _device("x", x), torch.bfloat16
    y, pre = (None, None) if out is None else out
    with _Call(dev, stream, (x, weight, bias, residual, y, pre, workspace)) as call:
        ws, ws_at, ws_bytes = _scratch(
            _head_workspace(spec_head_forward_workspace, M, N, K, workspace), dev, workspace)
        if out is None:
            y = torch.empty(M, N, dtype=bf, device=x.device)
            pre = torch.empty_like(y) if want_pre else None
        code = _sv.lib().spec_head_forward(
            _arg("x", x, bf, 0, dev), _arg("weight", weight, bf, 0, dev),
            _arg("bias", bias, bf, N, dev), _matrix("residual", residual, bf, M, N, dev), M, N, K,
            act, _matrix("y", y, bf, M, N, dev), _matrix("pre", pre, bf, M, N, dev), ws_at, ws_bytes,
            call.raw)
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
    M, N, K = _head_sizes(x, weight)
    dev, bf = _device("x", x), torch.bfloat16
    if tuple(dy.shape) != (M, N):
        raise ValueError(f"dy must be [{M}, {N}]")
    dx, dw, db = (None, None, None) if out is None else out
    with _Call(dev, stream, (dy, x, weight, pre, dx, dw, db, workspace)) as call:
        ws, ws_at, ws_bytes = _scratch(
            _head_workspace(spec_head_backward_workspace, M, N, K, workspace), dev, workspace)
        if out is None:
            dx = torch.empty(M, K, dtype=bf, device=x.device) if want_dx else None
            dw = torch.empty(N, K, dtype=bf, device=x.device) if want_dw else None
            db = torch.empty(N, dtype=torch.float32, device=x.device) if want_db else None
        code = _sv.lib().spec_head_backward(
            _arg("dy", dy, bf, M * N, dev), _arg("x", x, bf, 0, dev),
            _arg("weight", weight, bf, 0, dev), _matrix("pre", pre, bf, M, N, dev), M, N, K, act,
            _matrix("dx", dx, bf, M, K, dev), _matrix("dw", dw, bf, N, K, dev),
            _arg("db", db, torch.float32, N, dev), ws_at, ws_bytes, call.raw)
    _sv._check(code, "spec_head_backward")
    return dx, dw, db, ws


# ------------------------------------------------------------------- AdamW
class SpecAdamwTable:
    """The device table of spec_adamw_table, with the tensors it names (weights and
    gradients first)."""

    def __init__(self, data, n_items, state_bits, tensors):
        self.data, self.n_items, self.state_bits, self.tensors = data, n_items, state_bits, tensors
        # weights whose gradient is autograd's own: it may be replaced behind the table
        self.followed = [(p, g.data_ptr()) for p, g in zip(*tensors[:2])
                         if p.is_leaf and p.grad is not None and p.grad.data_ptr() == g.data_ptr()]

    def check(self):
        """Raises where a weight's .grad is no longer the tensor of the table."""
        for p, at in self.followed:
            if p.grad is None or p.grad.data_ptr() != at:
                raise ValueError("the gradient of a weight is not the table's tensor any more: keep the "
                                 "gradients (zero_grad(set_to_none=False)) or build the table anew")


def spec_adamw_table(params, grads, exp_avg, exp_avg_sq, *, exp_avg_scale=None,
                     exp_avg_sq_scale=None, master=None) -> SpecAdamwTable:
    """The table of tensors that spec_adamw_step goes by, built once: lists of
    weights (f32 or bf16), their gradients (the same type), and states. States
    are f32 tensors, or torch.float8_e4m3fn (or uint8) codes with lists of f32
    scales, one per SPEC_ADAMW_BLOCK elements. `master` lists f32 copies of
    bf16 weights (entries may be None). The tensors' addresses must stay as
    they are while the table is used: gradients are zeroed in place
    (zero_grad(set_to_none=False)), not dropped. A step refuses a weight whose
    .grad was the table's and has been replaced."""
    n = len(params)
    if not (len(grads) == len(exp_avg) == len(exp_avg_sq) == n):
        raise ValueError("params, grads and states must be lists of the same length")
    for name, extra in (("exp_avg_scale", exp_avg_scale), ("exp_avg_sq_scale", exp_avg_sq_scale),
                        ("master", master)):
        if extra is not None and len(extra) != n:
            raise ValueError(f"{name} must be a list of the same length")
    if n == 0:
        raise ValueError("no tensors")
    dev = _device("params[0]", params[0])
    f32 = torch.float32
    codes = (torch.float8_e4m3fn, torch.uint8)
    bits = 8 if exp_avg[0].dtype in codes else 32
    rows = (SpecAdamwTensor * n)()
    for i in range(n):
        p, m, v = params[i], exp_avg[i], exp_avg_sq[i]
        ms = exp_avg_scale[i] if exp_avg_scale is not None else None
        vs = exp_avg_sq_scale[i] if exp_avg_sq_scale is not None else None
        w = master[i] if master is not None else None
        size = p.numel()
        blocks = -(-size // SPEC_ADAMW_BLOCK)
        for name, s in (("exp_avg", m), ("exp_avg_sq", v)):
            if s.dtype not in (codes if bits == 8 else (f32,)):
                raise TypeError(f"{name}[{i}] must hold states of {bits} bits, got {s.dtype}")
        rows[i] = SpecAdamwTensor(
            _arg(f"params[{i}]", p, p.dtype, 0, dev), _arg(f"grads[{i}]", grads[i], p.dtype, size, dev),
            _arg(f"exp_avg[{i}]", m, m.dtype, size, dev),
            _arg(f"exp_avg_sq[{i}]", v, v.dtype, size, dev),
            _arg(f"exp_avg_scale[{i}]", ms, f32, blocks, dev),
            _arg(f"exp_avg_sq_scale[{i}]", vs, f32, blocks, dev),
            _arg(f"master[{i}]", w, f32, size, dev), size, _f32_or_bf16(p))
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
    return SpecAdamwTable(host.to(params[0].device), items.value, bits, keep)


def spec_adamw_step(table, step: int = 1, *, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                    eps: float = 1e-8, weight_decay: float = 0.01, grad_scale=None, lr_dev=None,
                    step_dev=None, workspace=None, stream=None):
    """One AdamW step over the tensors of `table`, in place. `grad_scale`,
    `lr_dev` (f32) and `step_dev` (int32) are one-element device tensors read
    when the kernel runs. See include/specdraft.h for the semantics. Returns
    the workspace."""
    if table.followed:
        table.check()
    dev, f32 = table.data.get_device(), torch.float32
    hyper = _HYPER.pack(lr, beta1, beta2, eps, weight_decay, step,
                        _arg("grad_scale", grad_scale, f32, 1, dev) or 0,
                        _arg("lr_dev", lr_dev, f32, 1, dev) or 0,
                        _arg("step_dev", step_dev, torch.int32, 1, dev) or 0)
    used = () if stream is None else (
        table.data, grad_scale, lr_dev, step_dev, workspace,
        *(t for group in table.tensors if group is not None for t in group))
    with _Call(dev, stream, used) as call:
        ws, ws_at, ws_bytes = _scratch(256, dev, workspace)
        code = _sv.lib().spec_adamw_step(table.data.data_ptr(), table.n_items, table.state_bits,
                                         hyper, ws_at, ws_bytes, call.raw)
    _sv._check(code, "spec_adamw_step")
    return ws
