"""spec_sample on the GPU against the 64-bit reference: tokens, probabilities, counts and
filtered rows, in both types, at sizes, masks, values and parameters where borders, bins,
chunks and vectors end. What is whole is compared exactly."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
# Borders are within 2^-38 of the mass, the reference's sums within 2^-40. Where u is nearer
# than this to one (among tokens of less than 1e-10 each), either side of it is right:
# the token's share of the mass, widened by this, still has to hold u.
EDGE = 2.0 ** -36
U24 = 1 - 2.0 ** -24


def law_of(rng, B, kind):
    """Parameters of B requests."""
    on = lambda p: rng.random(B) < p   # noqa: E731
    T = rng.uniform(0.3, 2.0, B)
    p = dict(temperature=T)
    if kind == "none":
        return {k: v.astype(np.float32) for k, v in p.items()}
    if kind in ("top_k", "all", "mixed"):
        p["top_k"] = rng.integers(1, 80, B)
    if kind in ("top_p", "all", "mixed"):
        p["top_p"] = rng.uniform(0.05, 0.999, B)
    if kind in ("min_p", "all", "mixed"):
        p["min_p"] = rng.uniform(0.001, 0.3, B)
    if kind == "mixed":
        p["temperature"] = np.where(on(0.2), 0.01, T)
        p["top_k"] = np.where(on(0.5), rng.integers(-2, 1, B), p["top_k"])
        p["top_k"] = np.where(on(0.2), 1 << 30, p["top_k"])
        p["top_p"] = np.where(on(0.4), 1.0, p["top_p"])
        p["top_p"] = np.where(on(0.1), 0.0, p["top_p"])
        p["min_p"] = np.where(on(0.6), 0.0, p["min_p"])
        p["min_p"] = np.where(on(0.1), 1.0, p["min_p"])
    return {k: v.astype(np.int32 if k == "top_k" else np.float32) for k, v in p.items()}


def logits_of(rng, R, V, values):
    z = 2.5 * rng.normal(size=(R, V)) - 1.1 * np.log(rng.permutation(V) + 1)
    if values == "masked":
        z[rng.random((R, V)) < 0.4] = -np.inf
        z[0, 1:] = -np.inf                      # one token is allowed
        z[0, 0] = 0.0
    elif values == "finite masks":
        z[rng.random((R, V)) < 0.4] = -1e9
        z[R // 2, rng.random(V) < 0.5] = -3.3e38
    elif values == "hard masks":                # what is left is less than many a top_k
        z[rng.random((R, V)) < 1 - 5 / V] = -1e9
    elif values == "ties":
        z = rng.integers(-3, 3, (R, V)).astype(np.float64)
    elif values == "equal":
        z[:] = rng.choice([0.0, 1.5, -700.0, 30000.0], (R, 1))
    elif values == "zeros":
        z = rng.choice([0.0, -0.0, 1.0, -1.0], (R, V))
    elif values == "tiny":
        z *= 1e-7
    elif values == "denormal":
        z *= 1e-40
    elif values == "large":
        z *= 200.0
    elif values == "huge":
        z *= 1e35
    elif values == "far below":
        z -= 5000.0
    elif values == "peaked":
        z[np.arange(R), rng.integers(0, V, R)] += 30.0
    return z


def make(seed, R, V, dtype, kind, values="plain", cu=None):
    rng = np.random.default_rng(seed)
    z = torch.tensor(logits_of(rng, R, V, values)).to(dtype).to(DEV)
    B = R if cu is None else len(cu) - 1
    u = rng.random(R).astype(np.float32)
    u[::7] = 0.0
    u[3::7] = U24
    u = np.minimum(u, np.float32(U24))
    return z, u, law_of(rng, B, kind)


def run(z, u, law, cu=None, **kw):
    t = {k: torch.tensor(v, device=DEV) for k, v in law.items()}
    out = sv.spec_sample(z, None if u is None else torch.tensor(u, device=DEV),
                         None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV), **t, **kw)
    return out[:4], sv.spec_get_status(out[4])


def check(z, u, law, got, cu=None, rows=None):
    tokens, prob, kept, filtered = (None if t is None else t.float().cpu().numpy() if t.dtype is BF16 else t.cpu().numpy()
                                    for t in got)
    zz = z.float().cpu().numpy().astype(np.float64)
    R, V = zz.shape
    req = np.arange(R) if cu is None else np.repeat(np.arange(len(cu) - 1), np.diff(cu))
    for r in range(R) if rows is None else rows:
        p = {n: law[k][req[r]] for n, k in (("T", "temperature"), ("top_k", "top_k"), ("top_p", "top_p"),
                                            ("min_p", "min_p")) if k in law}
        p = {n: int(v) if n == "top_k" else float(v) for n, v in p.items()}
        ref = O.sample_row(zz[r], None if u is None else float(u[r]), **p)
        assert ref["edge"] > EDGE, (r, ref["edge"])
        if kept is not None:
            assert kept[r] == len(ref["order"]), (r, kept[r], len(ref["order"]))
        if u is not None:
            at, = np.flatnonzero(ref["order"] == tokens[r])
            if ref["edge_u"] > EDGE:
                assert tokens[r] == ref["token"], (r, tokens[r], ref["token"])
            else:
                c = np.cumsum(ref["law"])
                assert c[at] - ref["law"][at] - EDGE <= u[r] <= c[at] + EDGE
            assert abs(prob[r] - ref["law"][at]) <= 2.0 ** -23 * ref["law"][at]
        if filtered is not None:
            want = np.full(V, -np.inf)
            want[ref["order"]] = zz[r, ref["order"]]
            assert np.array_equal(filtered[r], want), r


SIZES = [(3, 1), (5, 2), (4, 7), (9, 31), (6, 256), (6, 257), (8, 1000), (7, 2049), (5, 4099), (20, 8200),
         (3, 32003), (2, 70001), (300, 515), (330, 9001)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["none", "top_k", "top_p", "min_p", "all", "mixed"])
@pytest.mark.parametrize("R,V", SIZES)
def test_sizes_and_filters(R, V, kind, dtype):
    z, u, law = make(R * 1000 + V, R, V, dtype, kind)
    got, status = run(z, u, law, want_kept=True, want_filtered=True)
    assert status == sv.SPEC_OK
    rows = None if R < 50 else range(0, R, 7)
    check(z, u, law, got, rows=rows)


VALUES = ["masked", "finite masks", "hard masks", "ties", "equal", "zeros", "tiny", "denormal", "large", "huge",
          "far below", "peaked"]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["none", "top_k", "top_p", "all", "mixed"])
@pytest.mark.parametrize("values", VALUES)
@pytest.mark.parametrize("R,V", [(12, 1003), (4, 20000)])
def test_values(R, V, values, kind, dtype):
    z, u, law = make(R + V, R, V, dtype, kind, values)
    got, status = run(z, u, law, want_kept=True, want_filtered=True)
    assert status == sv.SPEC_OK
    check(z, u, law, got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["none", "top_k", "mixed"])
def test_long_rows(kind, dtype):
    for R, V in ((2, 201088), (320, 40000)):
        z, u, law = make(V, R, V, dtype, kind)
        got, status = run(z, u, law, want_kept=True, want_filtered=True)
        assert status == sv.SPEC_OK
        check(z, u, law, got, rows=range(0, R, 61))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R", [1, 200])
def test_the_longest_row(R, dtype):
    """V = 2^24 by one CTA and by a cluster; the logits fall with the id."""
    V = 1 << 24
    if R > 1 and dtype is F32:
        R = 170
    x = torch.arange(V, device=DEV, dtype=torch.float64)
    row = (-2.0 * torch.log1p(x)).to(dtype)
    z = row.expand(R, V).contiguous()
    u = np.linspace(0, U24, R).astype(np.float32) if R > 1 else np.float32([0.9])
    law = dict(top_p=np.full(R, 0.95, np.float32), temperature=np.full(R, 1.0, np.float32))
    got, status = run(z, u, law, want_kept=True)
    assert status == sv.SPEC_OK
    w = torch.exp(row.double())          # in the order of the ids already
    c = torch.cumsum(w, 0)
    n = int((c - w < float(law["top_p"][0]) * c[-1]).sum())
    at = torch.searchsorted(c[:n], torch.tensor(u, device=DEV).double() * c[n - 1], right=True)
    assert torch.equal(got[2], torch.full((R,), n, dtype=torch.int32, device=DEV))
    assert torch.equal(got[0], at.clamp(max=n - 1).int())


def test_requests_own_their_rows():
    cu = [0, 3, 3, 4, 9, 9]
    for dtype in (BF16, F32):
        z, u, law = make(5, 9, 777, dtype, "mixed", cu=cu)
        got, status = run(z, u, law, cu, want_kept=True, want_filtered=True)
        assert status == sv.SPEC_OK
        check(z, u, law, got, cu)


def test_defaults_are_the_softmax():
    z, u, _ = make(1, 40, 300, F32, "none")
    got, status = run(z, u, {}, want_kept=True)
    assert status == sv.SPEC_OK
    check(z, u, {}, got)


def test_the_law_over_a_lattice_of_u():
    """4096 draws of one law at equal steps: every token as often as its probability says."""
    n, V = 4096, 700
    z, _, law = make(3, 1, V, BF16, "all")
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    cu = np.array([0, n])
    got, status = run(z.expand(n, V).contiguous(), u, law, cu)
    assert status == sv.SPEC_OK
    ref = O.sample_row(z[0].float().cpu().numpy(), 0.5, T=float(law["temperature"][0]), top_k=int(law["top_k"][0]),
                       top_p=float(law["top_p"][0]), min_p=float(law["min_p"][0]))
    want = np.zeros(V)
    want[ref["order"]] = ref["law"]
    assert np.abs(np.bincount(got[0].cpu().numpy(), minlength=V) / n - want).max() <= 1.0 / n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1000, 1001, 20011])
def test_filtering_alone_apart_and_in_place(V, dtype):
    z, _, law = make(V, 6, V, dtype, "mixed")
    guard = torch.full((8, V), 7.0, dtype=dtype, device=DEV)
    out = guard.view(-1)[: 6 * V].view(6, V)
    got, status = run(z, None, law, out=(None, None, None, out))
    assert status == sv.SPEC_OK and got[0] is None
    check(z, None, law, (None, None, None, out))
    assert bool((guard.view(-1)[6 * V:] == 7).all())
    same = z.clone()
    _, status = run(same, None, law, out=(None, None, None, same))
    assert status == sv.SPEC_OK and torch.equal(same, out)
    # with a draw too
    u = np.full(6, 0.7, np.float32)
    ref, _ = run(z, u, law, want_filtered=True)
    same = z.clone()
    tokens = torch.empty(6, dtype=torch.int32, device=DEV)
    _, status = run(same, u, law, out=(tokens, None, None, same))
    assert status == sv.SPEC_OK and torch.equal(same, out) and torch.equal(tokens, ref[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 30000])
def test_bad_rows_are_reported_and_the_others_right(V, dtype):
    R = 12
    for where, change in (("nan", float("nan")), ("inf", float("inf")), ("empty", None)):
        z, u, law = make(V, R, V, dtype, "mixed")
        if change is None:
            z[4] = -float("inf")
        else:
            z[4, V // 3] = change
        got, status = run(z, u, law, want_kept=True, want_filtered=True)
        assert status == sv.SPEC_ERR_INVALID_ARG, where
        assert int(got[0][4]) == -1 and float(got[1][4]) == 0 and int(got[2][4]) == 0
        assert bool((got[3][4] == -float("inf")).all())
        check(z, u, law, got, rows=[r for r in range(R) if r != 4])


@pytest.mark.parametrize("kw", [
    dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")), dict(top_p=-0.1),
    dict(top_p=1.5), dict(top_p=float("nan")), dict(min_p=-1e-3), dict(min_p=1.01), dict(min_p=float("nan")),
    dict(u=1.0), dict(u=-0.25), dict(u=float("nan"))])
def test_bad_parameters_are_reported(kw):
    z, u, law = make(2, 5, 400, BF16, "all")
    (name, value), = kw.items()
    (u if name == "u" else law[name])[3] = value
    got, status = run(z, u, law, want_kept=True)
    assert status == sv.SPEC_ERR_INVALID_ARG
    assert int(got[0][3]) == -1 and int(got[2][3]) == 0
    check(z, u, law, got, rows=[0, 1, 2, 4])


@pytest.mark.parametrize("cu", [[0, 3, 2, 5], [1, 2, 3, 5], [0, 2, 4, 4]])
def test_bad_offsets_are_reported(cu):
    z, u, law = make(2, 5, 400, BF16, "all", cu=cu)
    _, status = run(z, u, law, cu)
    assert status == sv.SPEC_ERR_INVALID_ARG


def test_a_mask_of_nan_below_the_border_is_reported_too():
    """A NaN is no logit of a token that a mask forbids: -inf is."""
    z, u, law = make(2, 3, 400, BF16, "top_k")
    z[:, 5] = float("nan")
    _, status = run(z, u, law)
    assert status == sv.SPEC_ERR_INVALID_ARG


def test_no_rows():
    z = torch.zeros(0, 50, device=DEV)
    out = sv.spec_sample(z, torch.zeros(0, device=DEV), want_kept=True)
    assert sv.spec_get_status(out[4]) == sv.SPEC_OK and out[0].numel() == 0


def test_results_do_not_go_by_the_batch():
    """The same row alone (a cluster) and among many (one CTA) has the same result."""
    z, u, law = make(9, 400, 20000, BF16, "all")
    many, _ = run(z, u, law, want_kept=True, want_filtered=True)
    for r in (0, 77, 399):
        one, _ = run(z[r:r + 1], u[r:r + 1], {k: v[r:r + 1] for k, v in law.items()}, want_kept=True,
                     want_filtered=True)
        assert all(torch.equal(a[r:r + 1], b) for a, b in zip(many, one))


def test_replays_in_a_graph_with_new_inputs():
    z, u, law = make(9, 20, 5000, BF16, "mixed")
    t = {k: torch.tensor(v, device=DEV) for k, v in law.items()}
    uu = torch.tensor(u, device=DEV)
    ws = torch.empty(sv.spec_sample_workspace(20, 5000), dtype=torch.uint8, device=DEV)
    out = (torch.empty(20, dtype=torch.int32, device=DEV), torch.empty(20, device=DEV),
           torch.empty(20, dtype=torch.int32, device=DEV), torch.empty_like(z))
    call = lambda: sv.spec_sample(z, uu, out=out, workspace=ws, **t)   # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    z2, u2, law2 = make(10, 20, 5000, BF16, "mixed")
    z.copy_(z2)
    uu.copy_(torch.tensor(u2))
    for k, v in law2.items():
        t[k].copy_(torch.tensor(v))
    g.replay()
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    check(z2, u2, law2, out)


def test_on_a_stream_of_its_own():
    z, u, law = make(11, 30, 3000, F32, "all")
    ref, _ = run(z, u, law, want_filtered=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = sv.spec_sample(z, torch.tensor(u, device=DEV), **{k: torch.tensor(v, device=DEV) for k, v in law.items()},
                         want_filtered=True, stream=s)
    s.synchronize()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[3], ref[3])


def test_wrong_tensors_are_refused():
    z, u, law = make(2, 5, 400, BF16, "top_k")
    uu = torch.tensor(u, device=DEV)
    for bad in (dict(top_k=torch.ones(5, device=DEV)), dict(top_p=torch.ones(4, device=DEV)),
                dict(temperature=torch.ones(5, dtype=torch.float64, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            sv.spec_sample(z, uu, **bad)
    with pytest.raises((TypeError, ValueError)):
        sv.spec_sample(z, uu[:3])
    with pytest.raises((TypeError, ValueError)):
        sv.spec_sample(z.half(), uu)
    with pytest.raises(ValueError):
        sv.spec_sample(z, uu, out=(torch.empty(5, dtype=torch.int32, device=DEV), None, None,
                                   torch.empty(400, 5, dtype=BF16, device=DEV)))


@pytest.fixture
def checked():
    sv.use_checked_library(True)
    yield
    sv.use_checked_library(False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,V", [(3, 1), (4, 7), (6, 257), (5, 4099), (2, 20011), (320, 515)])
def test_no_access_leaves_the_call(R, V, dtype, checked):
    for values in ("plain", "finite masks", "ties"):
        z, u, law = make(R + V, R, V, dtype, "mixed", values)
        got, status = run(z, u, law, want_kept=True, want_filtered=True)
        assert status == sv.SPEC_OK
        check(z, u, law, got, rows=range(0, R, 1 + R // 40))


@pytest.mark.parametrize("per", [200, 255, 256, 257, 511, 512, 513, 1700])
@pytest.mark.parametrize("kind", ["none", "top_p"])
def test_crowded_intervals(per, kind):
    """f32 rows whose tokens crowd in eight steps of the logits, `per` to a step, so that a
    border's neighbours are few, as many as are ranked, or too many to be."""
    rng = np.random.default_rng(per)
    step = 63 / 4096 * np.log(2)
    R, V = 6, max(8 * per, 1700)
    z = np.full((R, V), -200.0)
    for r in range(R):
        at = rng.permutation(V)[:8 * per]
        z[r, at] = -step * (np.repeat(np.arange(8) * 3, per) + rng.uniform(0.05, 0.95, 8 * per))
        z[r, at[0]] = 0.0
    z = torch.tensor(z, dtype=F32, device=DEV)
    law = dict(temperature=np.ones(R, np.float32))
    if kind == "top_p":
        law["top_p"] = rng.uniform(0.1, 0.95, R).astype(np.float32)
    u = rng.random(R).astype(np.float32)
    got, status = run(z, u, law, want_kept=True, want_filtered=True)
    assert status == sv.SPEC_OK
    check(z, u, law, got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("many", [200, 300, 510, 520, 1500])
def test_crowded_lists(many, dtype):
    """A law by min-p with many tokens next to one another and one far above them: they share an
    interval of the list."""
    rng = np.random.default_rng(many)
    R, V = 4, 6001
    z = np.full((R, V), -30.0)
    for r in range(R):
        at = rng.permutation(V)[:many + 1]
        z[r, at[:many]] = rng.uniform(1, 1 + 1e-4, many)
        z[r, at[many]] = 6.0
    z = torch.tensor(z).to(dtype).to(DEV)
    law = dict(temperature=np.ones(R, np.float32), min_p=np.full(R, 1e-3, np.float32),
               top_p=np.array([1.0, 0.3, 0.6, 0.9], np.float32), top_k=np.array([0, many // 2, 0, 400], np.int32))
    u = np.array([0.2, 0.9, 0.5, 0.7], np.float32)
    got, status = run(z, u, law, want_kept=True, want_filtered=True)
    assert status == sv.SPEC_OK
    check(z, u, law, got)
