"""spec_process_logits on the GPU against the 64-bit reference: penalties,
biases and masks on linear batches and trees, in both types, at sizes,
alignments and masks where ranges, segments and vectors end."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24   # half a step of f32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step of the type


def make(seed, V, rows, dtype, hist=20, tree=0, bias=3, mask="rows", prompt=True, repeat=False):
    """A batch of requests with the given numbers of rows."""
    rng = np.random.default_rng(seed)
    B = len(rows)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    R = int(cu[-1])
    z = (3 * rng.normal(size=(R, V))).astype(np.float32)
    z[rng.random((R, V)) < 0.02] = -np.inf
    c = {}
    if hist:
        n = rng.integers(0, hist + 1, B)
        n[0] = 0
        c["cu_history"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        c["history"] = rng.integers(0, min(V, 3 if repeat else V), int(n.sum())).astype(np.int32)
        if prompt:
            c["prompt_len"] = rng.integers(0, hist + 5, B).astype(np.int32)   # past the end too
    if tree:
        c["tokens"] = rng.integers(0, V, R).astype(np.int32)
        c["parent"] = np.concatenate([[-1 if v == 0 else int(rng.integers(max(0, v - 3), v))
                                       for v in range(n)] for n in rows if n]).astype(np.int32)
    else:
        K = [max(0, n - 1) for n in rows]
        c["cu_tokens"] = np.concatenate([[0], np.cumsum(K)]).astype(np.int32)
        c["tokens"] = rng.integers(0, min(V, 2 if repeat else V), sum(K)).astype(np.int32)
    c["repetition"] = rng.uniform(0.7, 1.6, B).astype(np.float32)
    c["frequency"] = rng.uniform(-0.5, 1.0, B).astype(np.float32)
    c["presence"] = rng.uniform(-0.5, 1.0, B).astype(np.float32)
    if bias:
        n = rng.integers(0, bias + 1, B)
        n[-1] = bias
        c["cu_bias"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        c["bias_ids"] = rng.integers(0, V, int(n.sum())).astype(np.int32)
        c["bias_values"] = rng.normal(size=int(n.sum())).astype(np.float32) * 5
        c["bias_values"][0] = -np.inf
    W = (V + 31) // 32
    if mask:
        m = rng.integers(0, 2 ** 32, (R, W), dtype=np.uint64).astype(np.uint32)
        m[::3] = 0xffffffff
        m[1::5] = 0            # rows that the mask leaves nothing
        if mask == "index":
            c["mask_rows"] = rng.integers(-1, R, R).astype(np.int32)
        c["mask"] = m.view(np.int32)
    return torch.tensor(z).to(dtype).to(DEV), cu, c


def run(z, cu, c, out=None, **kw):
    t = {k: torch.tensor(v, device=DEV) for k, v in c.items()}
    rows = np.diff(cu)
    out, ws = sv.spec_process_logits(z, torch.tensor(cu, device=DEV), max_rows=max(1, int(rows.max())),
                                     out=out, **t, **kw)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    return out


def check(z, cu, c, got):
    ref, scale = O.process_logits(z.float().cpu().numpy(), cu, c)
    g = got.float().cpu().numpy().astype(np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(g)) and np.array_equal(ref[~fin], g[~fin])
    # at most 7 roundings in 32 bits (sum, quotient or product, f n, two
    # differences, and f n's factors), then one to the type
    before = 7 * U32 * scale
    tol = before + HALF[z.dtype] * (np.abs(np.where(fin, ref, 0)) + before)
    # what no rule touches keeps its bits
    zin = z.float().cpu().numpy().astype(np.float64)
    same = fin & (ref == zin)
    assert np.array_equal(g[same], zin[same])
    off = np.abs(g[fin] - ref[fin]) - tol[fin]
    assert off.max(initial=-1) <= 0, off.max()


CASES = [
    ("one token", dict(V=1, rows=[1], dtype=torch.float32, hist=2, bias=1)),
    ("small f32", dict(V=1024, rows=[5, 5, 1, 3], dtype=torch.float32)),
    ("odd f32", dict(V=1001, rows=[2, 0, 4], dtype=torch.float32)),
    ("f32 ranges", dict(V=8192 + 2052, rows=[4, 3], dtype=torch.float32, hist=300)),
    ("bf16", dict(V=8200, rows=[6, 2, 3], dtype=torch.bfloat16, hist=500)),
    ("bf16 odd", dict(V=20011, rows=[1, 3, 2], dtype=torch.bfloat16, hist=500)),
    ("bf16 by 4", dict(V=20012, rows=[2, 3, 2], dtype=torch.bfloat16, hist=500)),
    ("bf16 by 2", dict(V=9002, rows=[6, 3, 2], dtype=torch.bfloat16, hist=300, mask="index")),
    ("f32 by 2", dict(V=5002, rows=[6, 3, 2], dtype=torch.float32, hist=300)),
    ("bf16 by 2, long", dict(V=30002, rows=[3] * 200, dtype=torch.bfloat16, hist=20)),
    ("f32 by 1, long", dict(V=12289, rows=[3] * 260, dtype=torch.float32, hist=20)),
    ("bf16 vector end", dict(V=16392, rows=[3, 3], dtype=torch.bfloat16)),
    ("mask by index", dict(V=2056, rows=[4, 4, 4], dtype=torch.bfloat16, mask="index")),
    ("no mask", dict(V=2056, rows=[4, 1], dtype=torch.bfloat16, mask=None)),
    ("mask alone", dict(V=515, rows=[4, 1], dtype=torch.float32, hist=0, bias=0)),
    ("no prompt", dict(V=700, rows=[3, 3], dtype=torch.float32, prompt=False)),
    ("repeated tokens", dict(V=64, rows=[40, 33], dtype=torch.float32, hist=90, repeat=True)),
    ("long segment", dict(V=128, rows=[100, 17, 1], dtype=torch.bfloat16)),
    ("tree", dict(V=3000, rows=[64, 1, 20], dtype=torch.bfloat16, tree=1)),
    ("tree f32 odd", dict(V=777, rows=[33, 40], dtype=torch.float32, tree=1, mask="index")),
    ("many requests", dict(V=8192, rows=[3] * 700, dtype=torch.bfloat16, hist=10)),
]


@pytest.mark.parametrize("name,case", CASES, ids=[c[0] for c in CASES])
@pytest.mark.parametrize("inplace", [False, True])
def test_rules(name, case, inplace):
    z, cu, c = make(len(name), **case)
    out = z.clone() if inplace else None
    got = run(out if inplace else z, cu, c, out=out)
    check(z, cu, c, got)


@pytest.mark.parametrize("name,case", CASES[1:9] + CASES[18:20], ids=[c[0] for c in CASES[1:9] + CASES[18:20]])
def test_rules_checked(name, case):
    """The same on the bounds-checked build: no access leaves its buffers."""
    sv.use_checked_library(True)
    try:
        z, cu, c = make(50 + len(name), **case)
        check(z, cu, c, run(z, cu, c))
    finally:
        sv.use_checked_library(False)


def test_rules_large_range_walks_wide_tables():
    """The wide ranges and 16-row segments of large calls."""
    z, cu, c = make(91, V=40000, rows=[9] * 80, dtype=torch.bfloat16, hist=40)
    got = run(z, cu, c)
    keep = [0, 1, 41, 79]   # a few requests against the reference
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in keep])
    sub = {k: v for k, v in c.items() if k in ("repetition", "frequency", "presence", "prompt_len")}
    sub = {k: v[keep] for k, v in sub.items()}
    for ids, off in (("history", "cu_history"), ("tokens", "cu_tokens"), ("bias_ids", "cu_bias")):
        parts = [c[ids][c[off][b]:c[off][b + 1]] for b in keep]
        sub[ids], sub[off] = np.concatenate(parts), np.concatenate([[0], np.cumsum([len(p) for p in parts])])
    sub["bias_values"] = np.concatenate([c["bias_values"][c["cu_bias"][b]:c["cu_bias"][b + 1]] for b in keep])
    sub["mask"] = c["mask"][rows]
    check(z[rows], np.concatenate([[0], np.cumsum([9] * 4)]), sub, got[rows])


def test_rules_masked_nan_is_minus_infinity():
    z = torch.full((1, 40), float("nan"), device=DEV)
    z[0, 7] = 2.0
    m = np.zeros((1, 2), np.uint32)
    m[0, 0] = 1 << 7
    got = run(z, np.array([0, 1], np.int32), dict(mask=m.view(np.int32)))
    want = torch.full((1, 40), -float("inf"))
    want[0, 7] = 2.0
    assert torch.equal(got.cpu(), want)


def test_rules_without_rules_copy():
    z = torch.randn(3, 100, device=DEV)
    out, ws = sv.spec_process_logits(z, torch.tensor([0, 3], dtype=torch.int32, device=DEV), max_rows=3)
    assert torch.equal(out, z) and sv.spec_get_status(ws) == sv.SPEC_OK


@pytest.mark.parametrize("name,change", [
    ("offsets", lambda cu, c: cu.__setitem__(1, 9)),
    ("token", lambda cu, c: c["history"].__setitem__(0, 300)),
    ("draft", lambda cu, c: c["tokens"].__setitem__(0, -1)),
    ("rho", lambda cu, c: c["repetition"].__setitem__(1, 0.0)),
    ("frequency", lambda cu, c: c["frequency"].__setitem__(0, np.nan)),
    ("bias id", lambda cu, c: c["bias_ids"].__setitem__(0, 300)),
    ("bias value", lambda cu, c: c["bias_values"].__setitem__(0, np.inf)),
    ("mask row", lambda cu, c: c["mask_rows"].__setitem__(2, 8)),
])
def test_rules_reports_bad_inputs(name, change):
    sv.use_checked_library(True)   # nothing leaves its buffers even so
    try:
        z, cu, c = make(7, V=300, rows=[4, 4], dtype=torch.float32, mask="index")
        c["history"] = np.arange(4, dtype=np.int32)
        c["cu_history"] = np.array([0, 2, 4], np.int32)
        change(cu, c)
        _, ws = sv.spec_process_logits(z, torch.tensor(cu, device=DEV), max_rows=4,
                                       **{k: torch.tensor(v, device=DEV) for k, v in c.items()})
        assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG
    finally:
        sv.use_checked_library(False)


@pytest.mark.parametrize("parent", [[-1, 0, 2, 1], [-1, -1, 0, 0]])
def test_rules_reports_bad_trees(parent):
    z = torch.randn(4, 50, device=DEV)
    _, ws = sv.spec_process_logits(z, torch.tensor([0, 4], dtype=torch.int32, device=DEV), max_rows=4,
                                   tokens=torch.zeros(4, dtype=torch.int32, device=DEV),
                                   parent=torch.tensor(parent, dtype=torch.int32, device=DEV))
    assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG


def test_rules_in_a_graph_and_on_another_stream():
    z, cu, c = make(5, V=4104, rows=[5, 3], dtype=torch.bfloat16)
    t = {k: torch.tensor(v, device=DEV) for k, v in c.items()}
    cu_t = torch.tensor(cu, device=DEV)
    want, ws = sv.spec_process_logits(z, cu_t, max_rows=5, **t)
    out = torch.empty_like(z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_process_logits(z, cu_t, max_rows=5, out=out, workspace=ws, **t)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = sv.spec_process_logits(z, cu_t, max_rows=5, stream=s, **t)
    s.synchronize()
    assert torch.equal(got, want)
