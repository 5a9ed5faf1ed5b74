"""Plain 64-bit reference of the operators around a draft head: rules on
logits, the distillation loss, the head's products, AdamW. numpy, one row or
element rule at a time, written from the formulas; shares no code with the
package."""
from __future__ import annotations

import numpy as np

NEG_INF = -np.inf


# ------------------------------------------------------- rules on the logits
def row_tokens(case, b, r, lo):
    """Draft tokens that row r (of request b, whose rows start at lo) sees."""
    if case.get("tokens") is None:
        return []
    if case.get("parent") is None:
        k0, k1 = case["cu_tokens"][b], case["cu_tokens"][b + 1]
        return list(case["tokens"][k0:min(k0 + r - lo, k1)])
    path, v = [], r - lo
    while v > 0:
        path.append(case["tokens"][lo + v])
        v = case["parent"][lo + v]
    return path


def process_logits(logits, cu_rows, case):
    """logits [R, V] (any float), cu_rows [B+1], case: dict of numpy arrays
    under the names of spec_process_logits's arguments. Returns (out f64,
    scale f64): scale bounds the magnitudes each result went through."""
    z = np.asarray(logits, dtype=np.float64)
    out, scale = z.copy(), np.abs(np.where(np.isfinite(z), z, 0.0))
    R, V = z.shape
    for b in range(len(cu_rows) - 1):
        lo, hi = int(cu_rows[b]), int(cu_rows[b + 1])
        hist = []
        if case.get("history") is not None:
            hist = list(case["history"][case["cu_history"][b]:case["cu_history"][b + 1]])
        hp = int(case["prompt_len"][b]) if case.get("prompt_len") is not None else 0
        hp = max(0, min(hp, len(hist)))
        par = lambda n, d: float(case[n][b]) if case.get(n) is not None else d   # noqa: E731
        rho, f, p = par("repetition", 1.0), par("frequency", 0.0), par("presence", 0.0)
        bias = {}
        if case.get("bias_ids") is not None:
            for j in range(int(case["cu_bias"][b]), int(case["cu_bias"][b + 1])):
                bias[int(case["bias_ids"][j])] = float(case["bias_values"][j])
        for r in range(lo, hi):
            new = row_tokens(case, b, r, lo)
            made = np.bincount(np.asarray(hist[hp:] + new, dtype=np.int64), minlength=V)
            seen = np.bincount(np.asarray(hist + new, dtype=np.int64), minlength=V) > 0
            for x in set(np.flatnonzero(seen)) | set(bias):
                v = out[r, x] + bias.get(int(x), 0.0)
                m = abs(out[r, x]) + abs(bias.get(int(x), 0.0)) if np.isfinite(v) else 0.0
                if seen[x]:
                    v = v / rho if v > 0 else v * rho
                    m *= max(rho, 1 / rho, 1.0)
                    n = int(made[x])
                    if n:
                        v = v - f * n - p
                        m += abs(f * n) + abs(p)
                out[r, x], scale[r, x] = v, m
            if case.get("mask") is not None:
                row = int(case["mask_rows"][r]) if case.get("mask_rows") is not None else r
                if row >= 0:
                    words = np.asarray(case["mask"][row]).astype(np.uint32)
                    bits = (words[:, None] >> np.arange(32, dtype=np.uint32)) & 1
                    out[r, bits.reshape(-1)[:V] == 0] = NEG_INF
    return out, scale


# ------------------------------------------------------- distillation loss
def distill(target, draft, cu, temperature=None, weight=None):
    """Returns (loss [R], grad [R, V], terms [R]): terms is the sum of the
    magnitudes that the loss is put together from."""
    target, draft = np.asarray(target, np.float64), np.asarray(draft, np.float64)
    R, V = draft.shape
    loss, grad, terms = np.zeros(R), np.zeros((R, V)), np.zeros(R)
    for b in range(len(cu) - 1):
        T = 1.0 if temperature is None else float(temperature[b])
        T = 1.0 if T < 0.05 else T
        for r in range(int(cu[b]), int(cu[b + 1])):
            w = 1.0 if weight is None else float(weight[r])
            if w == 0:
                continue
            zt, zd = target[r + b] / T, draft[r] / T
            mt, md = zt.max(), zd.max()
            et, ed = np.exp(zt - mt), np.exp(zd - md)
            p, q = et / et.sum(), ed / ed.sum()
            on = p > 0
            # by the logits: a q that is 0 in 64 bits has a logarithm still
            lp, lq = zt[on] - mt - np.log(et.sum()), zd[on] - md - np.log(ed.sum())
            loss[r] = w * float(np.sum(p[on] * (lp - lq)))
            grad[r] = w / T * (q - p)
            d = np.abs(zt[on] - zd[on])
            terms[r] = abs(w) * (float(np.sum(p[on] * d)) + abs(mt - md) + np.log(et.sum()) +
                                 np.log(ed.sum()))
    return loss, grad, terms


# ------------------------------------------------------------------- AdamW
E4M3 = np.sort(np.array([s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                         for s in (1.0,) for e in range(16) for m in range(8)
                         if not (e == 15 and m == 7)]))


def to_e4m3(x):
    """The nearest e4m3 value (ties to the even mantissa), saturating."""
    a = np.abs(np.asarray(x, np.float64))
    i = np.clip(np.searchsorted(E4M3, a), 1, len(E4M3) - 1)
    lo, hi = E4M3[i - 1], E4M3[i]
    pick_hi = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    return np.sign(x) * np.where(a >= E4M3[-1], E4M3[-1], np.where(pick_hi, hi, lo))


def blocks_of(x, block=256):
    n = -(-len(x) // block) * block
    return np.concatenate([x, np.zeros(n - len(x))]).reshape(-1, block)


def pack8(x, root):
    """(values, scales) that a state of 8 bits stands for; x is m, or the root
    of v with `root`."""
    rows = blocks_of(np.asarray(x, np.float64))
    most = np.abs(rows).max(1)
    most = np.where(most < 2.0 ** -100, 0.0, most)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(most[:, None] > 0, rows * 448.0 / most[:, None], 0.0)
    if root:
        y = np.where((rows > 0) & (most[:, None] > 0), np.maximum(y, 2.0 ** -9), y)
    return (to_e4m3(y) * (most / 448.0)[:, None]).reshape(-1)[:len(x)], most / 448.0


def adamw(w, g, m, v, t, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """One step in 64 bits: (w, m, v)."""
    g = np.asarray(g, np.float64) * grad_scale
    m = beta1 * np.asarray(m, np.float64) + (1 - beta1) * g
    v = beta2 * np.asarray(v, np.float64) + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** t), v / (1 - beta2 ** t)
    return np.asarray(w, np.float64) * (1 - lr * weight_decay) - lr * mh / (np.sqrt(vh) + eps), m, v


# --------------------------------------------- product with an epilogue
def act(z, name):
    if name == "silu":
        return z / (1 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_slope(z, name):
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    if name == "gelu":
        c = np.sqrt(2 / np.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)
