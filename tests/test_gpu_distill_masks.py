"""spec_distill_loss with masks of every kind in the target, in the draft and in
both: -1e4, -1e9, the type's lowest value and -inf, over random tokens and over
runs that cover a thread's whole share, on both schedules."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from test_gpu_distill import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
# a cluster per position (with and without shifts), and persistent clusters
SCHEDULES = {"positions": (9000, [2, 3]), "odd": (9001, [2, 3]), "resident": (16384, [1] * 5 + [5] * 119)}


def fill(name, dtype):
    return {"1e4": -1e4, "1e9": -1e9, "lowest": torch.finfo(dtype).min, "inf": -INF, "none": None}[name]


def tokens(pattern, V, g):
    """The masked tokens; V - 1 is never one."""
    if pattern == "run":
        return torch.arange(V) < 2 * V // 3
    if pattern == "most":
        return torch.arange(V) < V - 7
    ban = torch.rand(V, generator=g) < 0.5
    ban[-1] = False
    return ban


def make(schedule, dtype, pattern, in_target, in_draft, T=(1.0, 1.5)):
    V, K = SCHEDULES[schedule]
    g = torch.Generator().manual_seed(V + len(in_target) * 7 + len(in_draft))
    cu = np.concatenate([[0], np.cumsum(K)]).astype(np.int32)
    R, B = int(cu[-1]), len(K)
    t = 2 * torch.randn(R + B, V, generator=g)
    d = t[torch.tensor(np.arange(R) + np.repeat(np.arange(B), K))] + 0.7 * torch.randn(R, V, generator=g)
    ban = tokens(pattern, V, g)
    for z, name in ((t, in_target), (d, in_draft)):
        if name != "none":
            z[:, ban] = fill(name, dtype)
    temp = T[0] + (T[1] - T[0]) * torch.rand(B, generator=g)
    w = 0.1 + 0.9 * torch.rand(R, generator=g)
    return t.to(dtype).to(DEV), d.to(dtype).to(DEV), cu, temp.to(DEV), w.to(DEV)


@pytest.mark.parametrize("in_target,in_draft", [
    ("1e4", "none"), ("1e9", "none"), ("lowest", "none"), ("inf", "none"),
    ("1e4", "inf"), ("1e9", "inf"), ("lowest", "inf"), ("1e9", "lowest"),
    ("lowest", "lowest"), ("1e9", "1e9"), ("inf", "lowest"), ("none", "lowest"), ("none", "inf")])
@pytest.mark.parametrize("pattern", ["run", "most", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("schedule", SCHEDULES)
def test_distill_masks(schedule, dtype, pattern, in_target, in_draft):
    t, d, cu, temp, w = make(schedule, dtype, pattern, in_target, in_draft)
    loss, grad, ws = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), temp, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    if schedule == "resident":   # the first requests are enough for the reference
        t, d, cu, temp, w = t[:25], d[:15], cu[:8], temp[:7], w[:15]
        loss, grad = loss[:15], grad[:15]
    check(t, d, cu, temp, w, loss, grad)


@pytest.mark.parametrize("schedule", SCHEDULES)
@pytest.mark.parametrize("at", [0, 5, 4000, -1])
@pytest.mark.parametrize("below,infinite", [(20.0, True), (100.0, True), (500.0, True), (1000.0, False),
                                            (1e30, False)])
def test_distill_draft_probability_of_zero(schedule, at, below, infinite):
    """A token that the draft holds at -inf: the loss is +inf as long as the
    target's probability is not 0 in 64 bits, wherever the token lies."""
    t, d, cu, _, w = make(schedule, torch.float32, "run", "none", "none")
    t[:, at] = t.amax(1) - below
    d[:, at] = -INF
    loss, grad, ws = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), None, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    assert bool(torch.isinf(loss).all()) == infinite and bool(torch.isinf(loss).any()) == infinite
    check(t[:6], d[:2], np.array([0, 2]) if schedule != "resident" else np.array([0, 1, 2]), None, w[:2], loss[:2],
          grad[:2])


def test_distill_target_row_of_the_lowest_value():
    """A target row that is the lowest bf16 value throughout is an even law."""
    t, d, cu, temp, w = make("positions", torch.bfloat16, "run", "none", "none")
    t[1] = torch.finfo(torch.bfloat16).min
    loss, grad, ws = sv.spec_distill_loss(t, d, torch.tensor(cu, device=DEV), temp, w)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    check(t, d, cu, temp, w, loss, grad)
