"""The lists of spec_process_logits (histories, drafts, biases): offsets past
their ends are reported and nothing behind them is read; empty lists."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LISTS = {"history": ("history", "cu_history"), "drafts": ("tokens", "cu_tokens"), "biases": ("bias_ids", "cu_bias")}


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rules(which, entries, offsets):
    ids, cu = LISTS[which]
    r = {ids: ints(*entries), cu: ints(*offsets)}
    if which == "biases":
        r["bias_values"] = torch.ones(len(entries), device=DEV)
    return r


def call(r, rows=(3, 3), V=200, dtype=torch.float32):
    cu = np.concatenate([[0], np.cumsum(rows)])
    z = torch.randn(int(cu[-1]), V, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    out, ws = sv.spec_process_logits(z, ints(*cu.tolist()), max_rows=max(rows),
                                     repetition=torch.full((len(rows),), 1.5, device=DEV), **r)
    return z, out, sv.spec_get_status(ws)


@pytest.mark.parametrize("checked", [True, False])
@pytest.mark.parametrize("which", LISTS)
@pytest.mark.parametrize("entries,offsets", [
    ([5, 6, 7, 8], [0, 2, 5]),        # one past the end
    ([5, 6, 7, 8], [0, 2, 1 << 28]),
    ([5, 6, 7, 8], [0, 1 << 30, (1 << 30) + 2]),
    ([], [0, 0, 2]), ([], [0, 1, 1])])
def test_offsets_past_a_list_are_reported(which, entries, offsets, checked):
    sv.use_checked_library(checked)
    try:
        assert call(rules(which, entries, offsets))[2] == sv.SPEC_ERR_INVALID_ARG
    finally:
        sv.use_checked_library(False)


@pytest.mark.parametrize("which", LISTS)
def test_offsets_up_to_the_end_are_taken(which):
    z, out, status = call(rules(which, [5, 6, 7, 8], [0, 2, 4]))
    assert status == sv.SPEC_OK and not torch.equal(z, out)


@pytest.mark.parametrize("which", LISTS)
def test_empty_lists_change_nothing(which):
    z, out, status = call(rules(which, [], [0, 0, 0]))
    assert status == sv.SPEC_OK and torch.equal(z, out)
    r = rules(which, [], [0, 0, 0])   # without offsets too
    r.pop(LISTS[which][1])
    z, out, status = call(r)
    assert status == sv.SPEC_OK and torch.equal(z, out)


def test_lists_that_end_at_the_last_offset():
    """Offsets up to 2^31 - 1: the last entries of the longest lists."""
    n, used, V = (1 << 31) - 1, 601, 5000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 26 GB")
    g = torch.Generator().manual_seed(3)
    tail = torch.randint(0, V, (used,), generator=g, dtype=torch.int32)
    ids = torch.randperm(V, generator=g)[:used].to(torch.int32)
    short = dict(history=tail, bias_ids=ids, bias_values=torch.randn(used, generator=g))
    results = []
    for size in (used, n):
        r = {}
        for name, x in short.items():
            r[name] = torch.empty(size, dtype=x.dtype, device=DEV)
            r[name][size - used:] = x.to(DEV)
        for cu in ("cu_history", "cu_bias"):
            r[cu] = ints(size - used, size)
        z, out, status = call({**r, "prompt_len": ints(100), "frequency": torch.ones(1, device=DEV)}, rows=(2,), V=V)
        assert status == sv.SPEC_OK and not torch.equal(z, out)
        results.append(out)
        del r
    assert torch.equal(*results)


def test_prompt_lengths_want_a_history():
    with pytest.raises(sv.SpecError):
        call(dict(prompt_len=ints(1, 1)))
    z, out, status = call(dict(prompt_len=ints(1, 1), history=ints()))   # an empty one, without offsets
    assert status == sv.SPEC_OK and torch.equal(z, out)
