"""spec_sample on the GPU where its sums decide: rows of values that go by the histogram, the same
results in every row and every run, and borders far down in a row's tail."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U24 = 1 - 2.0 ** -24


@pytest.mark.parametrize("filters", ["none", "top_p", "top_k"])
@pytest.mark.parametrize("R,V", [(4, 50257), (700, 9001)])
def test_equal_rows_have_equal_results(R, V, filters):
    """One row over and over, by its values' histogram, whose first warps have most of the work and
    whose last ones come late: the same result in every row and call."""
    rng = np.random.default_rng(V)
    z = torch.tensor(2.5 * rng.normal(size=V) - 1.1 * np.log(rng.permutation(V) + 1)).to(BF16).to(DEV)
    z = z.expand(R, V).contiguous()
    law = dict(temperature=torch.full((R,), 0.9, device=DEV))
    if filters == "top_p":
        law["top_p"] = torch.full((R,), 0.93, device=DEV)
    elif filters == "top_k":
        law["top_k"] = torch.full((R,), 4000, dtype=torch.int32, device=DEV)
    u = torch.full((R,), 0.77, device=DEV)
    first = None
    for _ in range(20):
        *got, ws = sv.spec_sample(z, u, want_kept=True, **law)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        got = [t for t in got if t is not None]
        first = first or [t[:1].clone() for t in got]
        for t, f in zip(got, first):
            assert torch.equal(t, f.expand(R))


def weights_of(z, T):
    """The values of a row in falling order, how many tokens each has, and the weight of one in units
    of 2^-120 (whole numbers, so that sums of millions lose nothing)."""
    values, counts = np.unique(z[z > -np.inf], return_counts=True)
    values, counts = values[::-1], counts[::-1]
    return values, counts, [int(math.exp((v - values[0]) / T) * 2.0 ** 120) for v in values]


def mass_of(counts, weights, n):
    """The weight of the first n tokens."""
    total = 0
    for c, w in zip(counts, weights):
        total += min(n, int(c)) * w
        n -= min(n, int(c))
    return total


def check_borders(z, T, top_k, top_p, u, token, prob, kept, filtered, bound):
    """Each border where exact weights put it, but for `bound` of the mass."""
    values, counts, weights = weights_of(z, T)
    all_n = int(counts.sum()) if top_k <= 0 else min(int(counts.sum()), top_k)
    mass = mass_of(counts, weights, all_n)
    e = Fraction(bound)
    p = Fraction(top_p)
    if top_p < 1:
        assert 1 <= kept <= all_n
        assert mass_of(counts, weights, kept) >= (p - e) * mass, (kept, "too few")
        assert mass_of(counts, weights, kept - 1) < (p + e) * mass, (kept, "too many")
    else:
        assert kept == all_n
    law = mass_of(counts, weights, kept)
    at = z[token]
    rank = int((z > at).sum() + (z[:token] == at).sum())
    assert rank < kept
    before, upto = mass_of(counts, weights, rank), mass_of(counts, weights, rank + 1)
    assert before <= (Fraction(u) + e) * law and upto > (Fraction(u) - e) * law, (rank, kept)
    assert abs(prob - (upto - before) / law) <= 2.0 ** -22 * prob
    if filtered is not None:
        order = np.lexsort((np.arange(len(z)), -z))[:kept]
        want = np.full(len(z), -np.inf)
        want[order] = z[order]
        assert np.array_equal(filtered, want)


def peaked(rng, V, kind):
    """A token that leads, and a tail of small weights, with values that have no bin of their own."""
    z = np.full(V, -27.75)
    if kind == "tiny":                     # one logit of 1e-7, the largest
        z[rng.integers(V)] = 1e-7
    elif kind == "tiny tail":
        z = np.where(rng.random(V) < 0.5, 1e-7, 0.0)
        z[rng.integers(V)] = 27.0
    elif kind == "large":                  # from 2048 on
        z[:] = 2976.0
        z[rng.integers(V)] = 3008.0
    elif kind == "far below":
        z[:] = -2128.0
        z[rng.integers(V)] = -2096.0
    elif kind == "spread":
        z = np.round(rng.normal(size=V) * 8) / 8 - 28
        z[rng.integers(0, V, 3)] = [1e-7, 2.0, 3.0]
    return z


LAWS = [(0, U24, 0.5), (0, 1 - 2.0 ** -21, U24), (0, 1.0, U24), (0, 1.0, 1 - 2.0 ** -20), (30000, 1.0, U24),
        (30000, U24, 1 - 2.0 ** -22), (0, 0.9, 0.3)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["tiny", "tiny tail", "large", "far below", "spread"])
@pytest.mark.parametrize("R,V", [(7, 50257), (7, 201088), (322, 50257)])
def test_borders_in_the_tail_of_a_peaked_row(R, V, kind, dtype):
    rng = np.random.default_rng(V)
    T = 1.2 if kind in ("large", "far below") else 1.0
    z = peaked(rng, V, kind)
    rows = torch.tensor(z).to(dtype).to(DEV)
    zz = rows.double().cpu().numpy()
    laws = [LAWS[r % len(LAWS)] for r in range(R)]
    top_k, top_p, u = (np.array([law[i] for law in laws]) for i in range(3))
    tokens, prob, kept, filtered, ws = sv.spec_sample(
        rows.expand(R, V).contiguous(), torch.tensor(u, dtype=F32, device=DEV),
        temperature=torch.full((R,), T, device=DEV), top_k=torch.tensor(top_k, dtype=torch.int32, device=DEV),
        top_p=torch.tensor(top_p, dtype=F32, device=DEV), want_kept=True, want_filtered=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    for r in range(len(LAWS)):
        k, p, x = laws[r]
        check_borders(zz, float(np.float32(T)), k, float(np.float32(p)), float(np.float32(x)), int(tokens[r]), float(prob[r]),
                      int(kept[r]), filtered[r].double().cpu().numpy(), 2.0 ** -37)
    for r in range(len(LAWS), R):          # the same law, the same result
        for t in (tokens, prob, kept, filtered):
            assert torch.equal(t[r], t[r % len(LAWS)])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_borders_in_the_tail_of_the_longest_row(dtype):
    V = 1 << 24
    z = torch.full((3, V), -26.0, dtype=dtype, device=DEV)
    z[:, 777] = 1e-7
    u = np.array([1 - 2.0 ** -14, U24, 0.9999])
    top_p = np.array([1.0, 1 - 2.0 ** -15, 1.0])
    tokens, prob, kept, _, ws = sv.spec_sample(
        z, torch.tensor(u, dtype=F32, device=DEV), top_p=torch.tensor(top_p, dtype=F32, device=DEV), want_kept=True)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    zz = z[0].double().cpu().numpy()
    for r in range(3):
        check_borders(zz, 1.0, 0, float(np.float32(top_p[r])), float(np.float32(u[r])), int(tokens[r]), float(prob[r]),
                      int(kept[r]), None, 2.0 ** -36)


# The value of half of a law's 256 tokens, the temperature, and a u whose part of the mass is so near to
# the other half's that the unit of the weights decides on which side of the border it falls.
NEAR = [(0.625, "0x1.a4c48p+0", "0x1.301846p-1"), (0.75, "0x1.5b43d6p+0", "0x1.450554p-1"),
        (2.625, "0x1.d608d8p-1", "0x1.e43ffep-1"), (2.75, "0x1.73a8dp+0", "0x1.bd0c4ep-1"),
        (2.875, "0x1.99f698p+0", "0x1.b71386p-1")]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gap,T,u", NEAR)
@pytest.mark.parametrize("filters", ["min_p", "min_p and top_k"])
def test_results_do_not_go_by_the_way_a_row_is_decided(gap, T, u, filters, dtype):
    """The tokens of a law all over the row, so that its list holds them and little else, and behind the
    rest of the row, whose tokens fill the list before the largest logit is seen."""
    R, V, half = 400, 60000, 128
    T, u = float.fromhex(T), float.fromhex(u)
    z = torch.full((2, V), -gap - 0.125)
    all_over = torch.arange(2 * half) * (V // (2 * half))
    for row, at in ((0, all_over), (1, torch.arange(V - 2 * half, V))):
        z[row, at[::2]] = 0.0
        z[row, at[1::2]] = -gap
    z = z.to(dtype).to(DEV).repeat(R // 2, 1)
    law = dict(temperature=torch.full((R,), T, device=DEV),
               min_p=torch.full((R,), math.exp(-(gap + 0.0625) / T), device=DEV))
    if filters != "min_p":
        law["top_k"] = torch.full((R,), 2 * half, dtype=torch.int32, device=DEV)
    tokens, prob, kept, _, ws = sv.spec_sample(z, torch.full((R,), u, device=DEV), want_kept=True, **law)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    assert bool((kept == 2 * half).all())
    drawn = z.gather(1, tokens.long()[:, None])[:, 0]
    assert bool((drawn == drawn[0]).all()) and bool((prob == prob[0]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("many", [100, 256, 257, 1000, 2540, 2560, 2561, 4000])
def test_lists_that_are_nearly_full(many, dtype):
    """Laws of as many tokens as a list may hold, and a few more or less, in rows of every order."""
    rng = np.random.default_rng(many)
    V, B = 12000, 40
    base = np.concatenate([np.round(rng.uniform(-4, 0, many) * 64) / 64, np.full(V - many, -9.0)])
    base[0] = 0.0
    z = torch.tensor(np.stack([rng.permutation(base) for _ in range(B - 1)] + [np.sort(base)])).to(dtype).to(DEV)
    z = z.repeat(10, 1)
    R = z.shape[0]
    law = dict(temperature=np.float32(0.9), min_p=np.float32(0.003), top_p=np.float32(0.97))
    u = np.float32(0.71)
    t = {k: torch.full((R,), float(v), device=DEV) for k, v in law.items()}
    tokens, prob, kept, _, ws = sv.spec_sample(z, torch.full((R,), float(u), device=DEV), want_kept=True, **t)
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    drawn = z.gather(1, tokens.long()[:, None])[:, 0]
    assert bool((drawn == drawn[0]).all()) and bool((prob == prob[0]).all()) and bool((kept == kept[0]).all())
    inside = z[0].double().cpu().numpy()
    inside[inside < -5] = -np.inf
    assert float(law["temperature"]) * math.log(float(law["min_p"])) > -9
    check_borders(inside, float(law["temperature"]), 0, float(law["top_p"]), float(u), int(tokens[0]), float(prob[0]),
                  int(kept[0]), None, 2.0 ** -37)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [2.0 ** 60, 2.0 ** 110, 3.4e38])
def test_temperatures_that_level_a_row(T, dtype):
    """Of ordinary logits every token is as likely as the next, of logits as large as T the law is the
    one of logits of about 1."""
    V, R = 9001, 5
    rng = np.random.default_rng(V)
    u = np.array([0.0, 0.25, 0.6, 0.9999, U24], np.float32)
    for large in (False, True):
        z = torch.tensor(rng.normal(size=V) * (min(T, 2.0 ** 105) if large else 1.0)).to(dtype).to(DEV)
        zz = z.double().cpu().numpy()
        for law in (dict(), dict(top_p=0.75), dict(top_k=500)):
            t = {k: torch.full((R,), v, dtype=torch.int32 if k == "top_k" else F32, device=DEV) for k, v in law.items()}
            tokens, prob, kept, _, ws = sv.spec_sample(z.expand(R, V).contiguous(), torch.tensor(u, device=DEV), want_kept=True,
                                                       temperature=torch.full((R,), T, device=DEV), **t)
            assert sv.spec_get_status(ws) == sv.SPEC_OK
            for r in range(R):
                check_borders(zz, float(np.float32(T)), law.get("top_k", 0), law.get("top_p", 1.0), float(u[r]),
                              int(tokens[r]), float(prob[r]), int(kept[r]), None, 2.0 ** -37)


@pytest.fixture
def checked():
    sv.use_checked_library(True)
    yield
    sv.use_checked_library(False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_access_leaves_the_call(dtype, checked):
    """Rows off the histogram and rows whose list is full, of odd lengths and in clusters."""
    for kind in ("tiny", "spread"):
        test_borders_in_the_tail_of_a_peaked_row(7, 50257, kind, dtype)
    for many in (2560, 4000):
        test_lists_that_are_nearly_full(many, dtype)
    test_results_do_not_go_by_the_way_a_row_is_decided(*NEAR[0], "min_p", dtype)
