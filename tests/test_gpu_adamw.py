"""spec_adamw_step on the GPU against the 64-bit reference: both weight types,
masters, states of 32 and of 8 bits, ragged and unaligned tensors in one
table, several steps, the device-side step, and the refusals."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
H = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 256, 255, 4096, 4097, 10000, 513]


def make(seed, dtype, bits, master, sizes=SIZES, shift=0):
    """Lists of tensors; `shift` elements of offset take away the alignment."""
    g = torch.Generator().manual_seed(seed)
    at = lambda x: torch.cat([torch.zeros(shift, dtype=x.dtype), x]).to(DEV)[shift:]   # noqa: E731
    p = [at((0.1 * torch.randn(n, generator=g)).to(dtype)) for n in sizes]
    grads = [at((0.02 * torch.randn(n, generator=g) * (torch.rand(n, generator=g) < 0.9)).to(dtype))
             for n in sizes]
    w = [at(0.1 * torch.randn(n, generator=g)) for n in sizes] if master else None
    if bits == 32:
        m = [at(0.01 * torch.randn(n, generator=g)) for n in sizes]
        v = [at((0.02 * torch.randn(n, generator=g)) ** 2) for n in sizes]
        return dict(p=p, g=grads, m=m, v=v, ms=None, vs=None, w=w)
    code = lambda n: at(torch.zeros(n, dtype=torch.uint8))   # noqa: E731
    scale = lambda n: torch.zeros(-(-n // 256), device=DEV)   # noqa: E731
    return dict(p=p, g=grads, m=[code(n) for n in sizes], v=[code(n) for n in sizes],
                ms=[scale(n) for n in sizes], vs=[scale(n) for n in sizes], w=w)


def table(s):
    return sv.spec_adamw_table(s["p"], s["g"], s["m"], s["v"], exp_avg_scale=s["ms"],
                               exp_avg_sq_scale=s["vs"], master=s["w"])


def f64(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def held(codes, scales, n):
    vals = codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes
    return f64(vals) * np.repeat(f64(scales), 256)[:n]


def snapshot(s, i):
    n = s["p"][i].numel()
    w = f64(s["w"][i]) if s["w"] else f64(s["p"][i])
    if s["ms"] is None:
        return w, f64(s["m"][i]), f64(s["v"][i])
    return w, held(s["m"][i], s["ms"][i], n), held(s["v"][i], s["vs"][i], n) ** 2


def check_step(s, before, t, gs, dtype):
    for i, (w0, m0, v0) in enumerate(before):
        g = f64(s["g"][i])
        w, m, v = O.adamw(w0, g, m0, v0, t, grad_scale=gs, **H)
        gm, gv = H["beta1"] * np.abs(m0) + 0.1 * np.abs(g * gs), v
        # decoding the states, the constants and the step's operations: at most
        # 8 roundings of each moment, relative to its terms
        tm, tv = 8 * U32 * gm, 8 * U32 * gv
        c1, c2 = 1 - H["beta1"] ** t, 1 - H["beta2"] ** t
        den = np.sqrt(v / c2) + H["eps"]
        upd = np.abs(H["lr"] * m / c1 / den)
        tw = 4 * U32 * np.abs(w0) + 16 * U32 * upd + H["lr"] / c1 * tm / den
        got_w, got_m, got_v = snapshot(s, i)
        if s["w"]:
            assert np.all(np.abs(got_w - w) <= tw), i
            assert np.array_equal(f64(s["p"][i]), f64(s["w"][i].to(dtype)))   # the weight: one rounding
        else:
            assert np.all(np.abs(got_w - w) <= tw + HALF[dtype] * (np.abs(w) + tw)), i
        if s["ms"] is None:
            assert np.all(np.abs(got_m - m) <= tm) and np.all(np.abs(got_v - v) <= tv), i
        else:
            for x, tol, got, scales, root in (
                    (m, tm, got_m, s["ms"][i], False),
                    (np.sqrt(v), 5 * U32 * np.sqrt(v), np.sqrt(got_v), s["vs"][i], True)):
                _, ws = O.pack8(x, root)
                sc = f64(scales)
                assert np.all(np.abs(sc - ws) <= ws * 10 * U32 + 1e-45), i
                # half a step of e4m3: 2^-4 of a normal value, half the
                # smallest step below; a root that would be zero is one step
                step = np.repeat(ws, 256)[:len(x)] * 2.0 ** -9
                half = np.maximum(np.abs(x) * 2.0 ** -4, step * (1.0 if root else 0.5))
                assert np.all(np.abs(got - x) <= (half + tol) * (1 + 32 * U32) + 1e-45), i
                # and the code is the rounding of a value within the tolerance
                # of x (12 roundings of the scale, the quotient and the decoding)
                per = np.repeat(np.where(ws > 0, ws, 1.0), 256)[:len(x)]
                d = (tol + 12 * U32 * np.abs(x)) / per
                lo, hi = O.to_e4m3(x / per - d), O.to_e4m3(x / per + d)
                if root:
                    lo, hi = (np.where((x > 0) & (per < 1), np.maximum(c, 2.0 ** -9), c) for c in (lo, hi))
                code = O.to_e4m3(got / np.repeat(np.where(sc > 0, sc, 1.0), 256)[:len(x)])
                assert np.all((lo <= code) & (code <= hi)), i


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype,bits,master", [
    (torch.float32, 32, False), (torch.bfloat16, 32, False), (torch.bfloat16, 32, True),
    (torch.float32, 8, False), (torch.bfloat16, 8, False), (torch.bfloat16, 8, True)])
def test_adamw_steps(dtype, bits, master, shift):
    s = make(11, dtype, bits, master, shift=shift)
    tb = table(s)
    scale = torch.tensor([0.5], device=DEV)
    for t in (1, 2, 3):
        before = [snapshot(s, i) for i in range(len(SIZES))]
        ws = sv.spec_adamw_step(tb, t, grad_scale=scale, **H)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        check_step(s, before, t, 0.5, dtype)


def test_adamw_tensors_of_both_types_in_one_table():
    a, b = make(1, torch.float32, 32, False, [300, 5000]), make(2, torch.bfloat16, 32, True, [300, 5000])
    tb = sv.spec_adamw_table(a["p"] + b["p"], a["g"] + b["g"], a["m"] + b["m"], a["v"] + b["v"],
                             master=[None, None] + b["w"])
    before = [[snapshot(s, i) for i in range(2)] for s in (a, b)]
    sv.spec_adamw_step(tb, 4, **H)
    check_step(a, before[0], 4, 1.0, torch.float32)
    check_step(b, before[1], 4, 1.0, torch.bfloat16)


def test_adamw_neighbours_keep_their_bits():
    """Ragged tensors cut out of one buffer: what lies between is not written."""
    for dtype, bits in ((torch.float32, 32), (torch.bfloat16, 8)):
        buf = torch.full((3000,), 7.0, dtype=dtype, device=DEV)
        p = [buf[16:16 + 1001], buf[1504:1504 + 999]]
        s = make(3, dtype, bits, False, [1001, 999])
        tb = sv.spec_adamw_table(p, s["g"], s["m"], s["v"], exp_avg_scale=s["ms"],
                                 exp_avg_sq_scale=s["vs"])
        sv.spec_adamw_step(tb, 1, **H)
        for a, b in ((0, 16), (1017, 1504), (2503, 3000)):
            assert bool((buf[a:b] == 7.0).all())


def test_adamw_states_of_zero_and_tiny_blocks():
    """A block without gradients stays zero and its weights only decay; tiny
    gradients do not divide by a root that became zero."""
    g = torch.zeros(512, device=DEV)
    g[256:] = 1e-20
    g[300] = 1.0
    s = dict(p=[torch.ones(512, device=DEV)], g=[g], m=[torch.zeros(512, dtype=torch.uint8, device=DEV)],
             v=[torch.zeros(512, dtype=torch.uint8, device=DEV)], ms=[torch.zeros(2, device=DEV)],
             vs=[torch.zeros(2, device=DEV)], w=None)
    tb = table(s)
    for t in (1, 2):
        before = [snapshot(s, 0)]
        sv.spec_adamw_step(tb, t, **H)
        check_step(s, before, t, 1.0, torch.float32)
    assert bool((s["m"][0][:256] == 0).all()) and float(s["ms"][0][0]) == 0
    assert bool(torch.isfinite(s["p"][0]).all())
    # smaller than a step would be with a root of zero (|m| / eps)
    assert float((s["p"][0] - 1).abs().max()) < 10 * H["lr"]


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_device_step_and_lr_in_a_graph(bits):
    a, b = make(5, torch.bfloat16, bits, True), make(5, torch.bfloat16, bits, True)
    ta, tb = table(a), table(b)
    step = torch.ones(1, dtype=torch.int32, device=DEV)
    lr = torch.tensor([H["lr"]], device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_adamw_step(tb, 1, step_dev=step, lr_dev=lr, workspace=ws, **{**H, "lr": 0.5})
    for t in (1, 2, 3):
        sv.spec_adamw_step(ta, t, **H)
        step.fill_(t)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(a["w"], b["w"]):
            # the device's bias corrections are off by a few roundings of 32 bits
            assert float((x - y).abs().max()) <= 40 * U32 * (0.6 + 20 * H["lr"]) * t
    step.fill_(0)
    keep = [x.clone() for x in b["w"]]
    g.replay()
    assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG
    assert all(torch.equal(x, y) for x, y in zip(keep, b["w"]))


def test_adamw_nan_stays_where_it_is():
    s = make(6, torch.float32, 8, False, [600])
    s["g"][0][10] = float("nan")
    sv.spec_adamw_step(table(s), 1, **H)
    bad = ~torch.isfinite(s["p"][0])
    assert bool(bad[10]) and int(bad.sum()) == 1


def test_adamw_table_of_another_shape_is_refused():
    s = make(7, torch.float32, 32, False, [5000])
    tb = table(s)
    tb.n_items = 1
    keep = s["p"][0].clone()
    ws = sv.spec_adamw_step(tb, 1, **H)
    assert sv.spec_get_status(ws) == sv.SPEC_ERR_INVALID_ARG and torch.equal(keep, s["p"][0])


def test_adamw_on_another_stream():
    a, b = make(8, torch.float32, 32, False), make(8, torch.float32, 32, False)
    sv.spec_adamw_step(table(a), 1, **H)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv.spec_adamw_step(table(b), 1, stream=s, **H)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a["p"], b["p"]))


def test_adamw_binding_refuses_mixed_lists():
    s = make(9, torch.float32, 32, False, [10])
    with pytest.raises(ValueError):
        sv.spec_adamw_table(s["p"], s["g"], s["m"], [])
    with pytest.raises(TypeError):
        sv.spec_adamw_table(s["p"], [s["g"][0].bfloat16()], s["m"], s["v"])
    with pytest.raises(sv.SpecError):
        sv.spec_adamw_table(s["p"], s["g"], s["m"], s["v"], master=[s["m"][0]])


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_squares_below_and_beyond_the_normal_range(bits, shift):
    """Gradients whose squares are subnormal or zero in 32 bits, one block per
    magnitude, and one that overflows: its root is infinite, so its weight only
    decays and nothing else is touched."""
    mags = 10.0 ** np.arange(-26, -14)
    n = 256 * len(mags)
    s = make(5, torch.float32, bits, False, [n + 256], shift=shift)
    for x in (s["m"], s["v"]):
        x[0].zero_()
    u = 0.5 + np.random.default_rng(5).random(n)
    g = np.zeros(n + 256, np.float32)
    g[:n] = (np.repeat(mags, 256) * u).astype(np.float32)
    g[n + 3] = 1e25
    s["g"][0].copy_(torch.from_numpy(g))
    w0 = f64(s["p"][0])
    h = dict(H, eps=1e-30)
    sv.spec_adamw_step(table(s), 1, **h)
    x = g[:n].astype(np.float64)
    w, m, v = O.adamw(w0[:n], x, 0.0 * x, 0.0 * x, 1, **h)
    # g^2 and its product are off by half of 2^-149 each where subnormal
    tv = 2.0 ** -149 + 8 * U32 * v
    got_w, got_m, got_v = snapshot(s, 0)
    r, tr = np.sqrt(v), tv / np.maximum(np.sqrt(v), 2.0 ** -75)
    if bits == 32:
        assert np.all(np.abs(got_v[:n] - v) <= tv)
    else:
        # half a step of e4m3 at the block's scale beside that
        half = np.maximum(r * 2.0 ** -4, np.repeat(r.reshape(-1, 256).max(1) / 448 * 2.0 ** -9, 256))
        assert np.all(np.abs(np.sqrt(got_v[:n]) - r) <= (half + tr) * (1 + 64 * U32))
    # where the root is known to a quarter, the weight follows
    c1, c2 = 0.1, np.sqrt(0.05)
    sure = tr <= r / 4
    upd = np.abs(H["lr"] * (m / c1) / (np.maximum(r, 1e-300) / c2))
    tw = 8 * U32 * np.abs(w0[:n]) + upd * (32 * U32 + 2 * tr / np.maximum(r, 1e-300))
    assert sure.sum() > n // 3
    assert np.all((np.abs(got_w[:n] - w) <= tw)[sure])
    assert abs(got_w[n + 3] - w0[n + 3] * (1 - H["lr"] * H["weight_decay"])) <= 4 * U32 * abs(w0[n + 3])
