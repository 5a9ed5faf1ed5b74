"""Timed cases of the operators that a draft head is served and trained with.

Next to the operators of operators.py, a speculation round uses

* sample    a token of every row's law at its request's temperature after min-p,
            top-k and top-p, by given random numbers, and the rows with what was
            dropped at -inf (spec_sample): the drafts, and the target's law that
            they are verified against;
* head4     a product of few rows with weights of 4 bits and group scales, with
            bias, activation and residual in its epilogue (spec_head4_forward):
            the draft head as it is served;
* norm      the norm over all gradients of a table and the factor that clips them,
            which the optimizer's step takes (spec_grad_norm);
* clip      the same, with the gradients scaled in place (spec_clip_grads).

A case is a dict of plain values; prepare() makes its inputs on the GPU from a
seed, run() is one pass, with `own` false in the plain form (elementary torch
operations), with `own` true through the package. exact() computes the same
outputs from the definitions in 64 bits.
"""
import itertools
import math

import torch

own = False

DEV = "cuda"
GREEDY_T = 0.05
CLIP_EPS = 1e-6          # added to the norm that a bound is divided by
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _package():
    import speculative_decoding_rejection_gb300 as sv
    return sv


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the next draft token of a few requests over a short vocabulary: latency only
        dict(name="sample-B4-V1024-f32", op="sample", B=4, k_lo=0, k_hi=0, V=1024, dtype="f32",
             filters="all", masked=0, filtered=0, draw=1),
        # the next draft token of a mixed batch over an odd vocabulary, a quarter of
        # the tokens under a grammar
        dict(name="sample-B64-V32003-bf16", op="sample", B=64, k_lo=0, k_hi=0, V=32003, dtype="bf16",
             filters="mixed", masked=4, filtered=0, draw=1),
        # f32 logits, an odd vocabulary, the law cut by its mass alone
        dict(name="sample-B48-V50257-f32", op="sample", B=48, k_lo=0, k_hi=0, V=50257, dtype="f32",
             filters="top_p", masked=0, filtered=0, draw=1),
        # the target rows of a batch with ragged drafts, cut before they are verified
        dict(name="filter-B256-K3..5-V151936-bf16", op="sample", B=256, k_lo=3, k_hi=5, V=151936,
             dtype="bf16", filters="mixed", masked=0, filtered=1, draw=0),
        # the next draft token of a full serving batch, each request with its own law
        dict(name="sample-B1024-V201088-bf16", op="sample", B=1024, k_lo=0, k_hi=0, V=201088,
             dtype="bf16", filters="mixed", masked=0, filtered=0, draw=1),
        # one token through a vocabulary projection held in 4 bits
        dict(name="head4-M1-K4096-N32000-g128", op="head4", M=1, K=4096, N=32000, group=128, zeros=0,
             act="none", bias=1, residual=0),
        # the residual block of a draft head for a batch of requests, small groups
        # with zero points
        dict(name="head4-M32-K2880-N2880-g32-silu", op="head4", M=32, K=2880, N=2880, group=32, zeros=1,
             act="silu", bias=1, residual=1),
        # five positions through a large vocabulary projection
        dict(name="head4-M5-K4096-N128256-g64", op="head4", M=5, K=4096, N=128256, group=64, zeros=0,
             act="none", bias=0, residual=0),
        # the gradients of a small draft head: few tensors of ragged sizes
        dict(name="norm-12x20000-f32", op="norm", tensors=12, numel=20000, dtype="f32", inf=0),
        # all gradients of a bf16 draft head of 480 million weights
        dict(name="norm-60x8000000-bf16", op="norm", tensors=60, numel=8000000, dtype="bf16", inf=0),
        # many small tensors, clipped in place
        dict(name="clip-150x30000-bf16", op="clip", tensors=150, numel=30000, dtype="bf16", inf=0),
        # an f32 draft head of about 200 million weights, clipped in place
        dict(name="clip-40x5000000-f32", op="clip", tensors=40, numel=5000000, dtype="f32", inf=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("sample", "sample", "sample", "head4", "head4", "norm", "clip"))
    if op == "sample":
        V = rng.choice((_log_int(rng, 500, 201088), rng.choice((32000, 128256, 151936, 201088))))
        dtype = rng.choice(("f32", "bf16", "bf16"))
        filtered = rng.choice((0, 0, 1))
        k_lo = rng.randint(0, 4) if filtered else 0
        k_hi = rng.randint(k_lo, 6) if filtered else 0
        most = (4e8 if dtype == "bf16" else 1.3e8) / (V * (k_hi + 1) * (4 if dtype == "f32" else 2))
        return dict(op=op, B=max(1, min(_log_int(rng, 1, 1024), int(most))), k_lo=k_lo, k_hi=k_hi, V=V,
                    dtype=dtype, filters=rng.choice(("none", "all", "top_k", "top_p", "min_p", "mixed", "mixed")),
                    masked=rng.choice((0, 0, 3, 50)), filtered=filtered,
                    draw=1 if not filtered else rng.randint(0, 1))
    if op == "head4":
        K = _log_int(rng, 64, 8192)
        N = min(_log_int(rng, 64, 130000), 4096 * 128256 // K)
        return dict(op=op, M=_log_int(rng, 1, 64), K=K, N=N, group=rng.choice((32, 64, 128)),
                    zeros=rng.randint(0, 1), act=rng.choice(("none", "silu", "gelu")),
                    bias=rng.randint(0, 1), residual=rng.randint(0, 1))
    tensors = _log_int(rng, 1, 200)
    numel = max(100, min(_log_int(rng, 300, 8000000), 200000000 // tensors))
    return dict(op=op, tensors=tensors, numel=numel, dtype=rng.choice(("f32", "bf16")),
                inf=rng.choice((0, 0, 0, 1)))


# ---------------------------------------------------- sizes that a case fixes
def _rows(case):
    """Rows of each request: its drafts and one more."""
    lo, hi = case["k_lo"], case["k_hi"]
    return [1 + lo + (b * 7919 + 3) % (hi - lo + 1) for b in range(case["B"])]


def _sizes(case):
    """Ragged tensor sizes about the case's, odd ones among them."""
    n = case["numel"]
    return [max(1, int(n * (0.2 + 1.6 * ((i + 1) * 0.6180339887 % 1.0)))) + i % 2
            for i in range(case["tensors"])]


def _offsets(lengths):
    return list(itertools.accumulate(lengths, initial=0))


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)
    s = {"case": case, "op": case["op"]}
    {"sample": _prepare_sample, "head4": _prepare_head4, "norm": _prepare_norm,
     "clip": _prepare_norm}[case["op"]](s, case, g)
    return s


def _uniform(n, g):
    return torch.rand(n, generator=g, device=DEV)


def _prepare_sample(s, case, g):
    """Logits with a Zipf-like tail, the order of the tokens shared by a request's
    rows, and the laws that requests ask for."""
    B, V = case["B"], case["V"]
    rows = _rows(case)
    R = sum(rows)
    s["cu_rows"] = torch.tensor(_offsets(rows), dtype=torch.int32, device=DEV)
    req = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(rows, device=DEV))
    s["logits"] = torch.empty(R, V, dtype=DTYPES[case["dtype"]], device=DEV)
    tail = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
    tail = tail[torch.randperm(V, generator=g, device=DEV)]
    shift = torch.randint(0, V, (B,), generator=g, device=DEV)
    banned = _uniform(V, g) < (1.0 / case["masked"] if case["masked"] else 0.0)
    banned[0] = False
    x = torch.arange(V, device=DEV)
    step = max(1, (1 << 27) // V)
    for a in range(0, R, step):
        e = min(R, a + step)
        z = 2.0 * torch.randn(e - a, V, generator=g, device=DEV)
        z += tail[(x[None] + shift[req[a:e], None]) % V]
        z[:, banned] = -math.inf
        s["logits"][a:e] = z
    s["uniform"] = _uniform(R, g) if case["draw"] else None
    # one request in twelve is greedy
    s["temperature"] = torch.where(torch.arange(B, device=DEV) % 12 == 7, 0.0, 0.5 + 0.8 * _uniform(B, g))
    kind = case["filters"]
    mixed = torch.arange(B, device=DEV) % 4
    top_k = torch.randint(1, 200, (B,), generator=g, device=DEV)
    top_k = torch.where((mixed == 0) | (mixed == 3), top_k, 0) if kind == "mixed" else top_k
    s["top_k"] = top_k.to(torch.int32) if kind in ("all", "top_k", "mixed") else None
    top_p = 0.5 + 0.49 * _uniform(B, g)
    top_p = torch.where(mixed < 2, top_p, 1.0) if kind == "mixed" else top_p
    s["top_p"] = top_p if kind in ("all", "top_p", "mixed") else None
    min_p = 0.005 + 0.2 * _uniform(B, g)
    min_p = torch.where(mixed == 2, min_p, 0.0) if kind == "mixed" else min_p
    s["min_p"] = min_p if kind in ("all", "min_p", "mixed") else None
    s["tokens"] = torch.empty(R, dtype=torch.int32, device=DEV) if case["draw"] else None
    s["prob"] = torch.empty(R, device=DEV) if case["draw"] else None
    s["kept"] = torch.empty(R, dtype=torch.int32, device=DEV)
    s["filtered"] = torch.empty_like(s["logits"]) if case["filtered"] else None


def _normal(shape, scale, g):
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(torch.bfloat16)


def _prepare_head4(s, case, g):
    M, K, N, group = case["M"], case["K"], case["N"], case["group"]
    G = -(-K // group)
    s["x"] = _normal((M, K), 1.0, g)
    half = -(-K // 2)
    s["codes"] = torch.empty(N, half, dtype=torch.uint8, device=DEV)   # the code of an even column in the low bits
    step = max(1, (1 << 26) // K)
    for a in range(0, N, step):
        e = min(N, a + step)
        q = (7.5 + 2.7 * torch.randn(e - a, 2 * half, generator=g, device=DEV)).round_().clamp_(0, 15)
        q = q.to(torch.uint8)
        s["codes"][a:e] = q[:, 0::2] | (q[:, 1::2] << 4)
    s["scales"] = ((0.5 + _uniform(N * G, g).view(N, G)) * (0.4 / math.sqrt(K))).to(torch.bfloat16)
    s["zeros"] = torch.randint(6, 11, (N, G), generator=g, device=DEV).to(torch.uint8) if case["zeros"] else None
    s["bias"] = _normal((N,), 0.5, g) if case["bias"] else None
    s["residual"] = _normal((M, N), 1.0, g) if case["residual"] else None
    s["y"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    # the weights as the kernel reads them, laid out once by a serving program
    s["weight"] = _package().spec_head4_pack(s["codes"], s["scales"], s["zeros"], K=K, group=group) if own else None


def _prepare_norm(s, case, g):
    sizes = _sizes(case)
    at = _offsets([-(-n // 256) * 256 for n in sizes])   # one flat buffer, padded with zeros
    dtype = DTYPES[case["dtype"]]
    s["grad"] = torch.zeros(at[-1], dtype=dtype, device=DEV)
    for i, (a, n) in enumerate(zip(at, sizes)):
        s["grad"][a:a + n] = (0.003 * (1 + i % 5)) * torch.randn(n, generator=g, device=DEV)
    s["grad_scale"] = 0.2 + 0.1 * _uniform(1, g)   # a loss scale's inverse
    # what clips at once and goes on clipping from pass to pass
    total = 0.25 * (float(s["grad"].abs().max()) if case["inf"] else
                    math.sqrt(float(s["grad"].float().square().sum(dtype=torch.float64))))
    s["bound"] = 0.5 * total
    s["out"] = torch.empty(2, device=DEV)
    if own:
        sv = _package()

        def views(t):
            return [t[a:a + n] for a, n in zip(at, sizes)]

        # the table of tensors that a training program keeps for its optimizer
        blocks = at[-1] // sv.SPEC_ADAMW_BLOCK
        codes = [torch.zeros(at[-1], dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros(blocks, device=DEV) for _ in range(2)]
        s["table"] = sv.spec_adamw_table(
            views(torch.zeros_like(s["grad"])), views(s["grad"]), views(codes[0]), views(codes[1]),
            exp_avg_scale=[scales[0][a // 256:] for a in at[:-1]],
            exp_avg_sq_scale=[scales[1][a // 256:] for a in at[:-1]])


# ---------------------------------------------------------------- the passes
def run(state):
    return {"sample": _run_sample, "head4": _run_head4, "norm": _run_norm, "clip": _run_clip}[state["op"]](state)


def _workspace(s, size):
    """The scratch that a serving program keeps from call to call."""
    if s.get("workspace") is None:
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return s["workspace"]


def _results(s):
    return {n: s[n] for n in ("tokens", "prob", "kept", "filtered") if s[n] is not None}


# ------------------------------------------------------- a token of each row
def _run_sample(s):
    if own:
        sv = _package()
        sv.spec_sample(s["logits"], s["uniform"], s["cu_rows"], temperature=s["temperature"],
                       top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                       out=(s["tokens"], s["prob"], s["kept"], s["filtered"]),
                       workspace=_workspace(s, sv.spec_sample_workspace(*s["logits"].shape)))
        return _results(s)
    # 64 bits: a token at a border of the law is inside it or outside
    R, V = s["logits"].shape
    cu = s["cu_rows"].long()
    req = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=DEV), cu[1:] - cu[:-1], output_size=R)
    T = s["temperature"].double()[req][:, None]
    greedy = T < GREEDY_T
    T = torch.where(greedy, 1.0, T)
    z, order = s["logits"].float().sort(dim=1, descending=True, stable=True)   # ties: the lower id first
    rank = torch.arange(V, device=DEV)[None]
    gap = z.double() - z[:, :1].double()
    keep = z > -math.inf
    if s["min_p"] is not None:
        keep &= gap >= T * s["min_p"].double()[req][:, None].log()
    if s["top_k"] is not None:
        k = s["top_k"].long()[req][:, None]
        keep &= (rank < k) | (k <= 0)
    weight = torch.where(keep, (gap / T).exp(), 0.0)
    mass = weight.cumsum(1)
    if s["top_p"] is not None:
        p = s["top_p"].double()[req][:, None]
        keep &= (p >= 1) | (mass - weight < p * mass[:, -1:])
    keep &= ~greedy | (rank == 0)
    count = keep.sum(1, keepdim=True)
    s["kept"].copy_(count[:, 0])
    if s["filtered"] is not None:
        s["filtered"].scatter_(1, order, torch.where(keep, z, -math.inf).to(s["filtered"].dtype))
    if s["uniform"] is not None:
        total = mass.gather(1, count - 1)
        at = ((mass <= s["uniform"].double()[:, None] * total) & keep).sum(1, keepdim=True)
        at = torch.minimum(at, count - 1)
        s["tokens"].copy_(order.gather(1, at)[:, 0])
        s["prob"].copy_((weight.gather(1, at) / total)[:, 0])
    return _results(s)


# ------------------------------------------ a product with weights of 4 bits
def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _run_head4(s):
    c = s["case"]
    if own:
        sv = _package()
        act = {"none": sv.SPEC_ACT_NONE, "silu": sv.SPEC_ACT_SILU, "gelu": sv.SPEC_ACT_GELU}[c["act"]]
        y, _ = sv.spec_head4_forward(
            s["x"], s["weight"], s["bias"], s["residual"], act=act, out=s["y"],
            workspace=_workspace(s, sv.spec_head4_forward_workspace(c["M"], c["N"], c["K"])))
        return y
    K, group = c["K"], c["group"]
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).view(c["N"], -1)[:, :K].float()
    zero = s["zeros"].float().repeat_interleave(group, 1)[:, :K] if s["zeros"] is not None else 8.0
    w = (q - zero) * s["scales"].float().repeat_interleave(group, 1)[:, :K]
    z = s["x"].float() @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------- the norm of all gradients
def _plain_norm(s, bound):
    g = s["grad"].float() * s["grad_scale"]
    norm = g.abs().max() if s["case"]["inf"] else g.square().sum(dtype=torch.float64).sqrt()
    factor = s["grad_scale"][0].double() * (bound / (norm.double() + CLIP_EPS)).clamp(max=1.0)
    return norm.float(), factor.float()


def _run_norm(s):
    if own:
        sv = _package()
        out, _ = sv.spec_grad_norm(s["table"], max_norm=s["bound"], inf=bool(s["case"]["inf"]),
                                   grad_scale=s["grad_scale"], out=s["out"],
                                   workspace=_workspace(s, sv.spec_grad_norm_workspace()))
        return out
    norm, factor = _plain_norm(s, s["bound"])
    return torch.stack((norm, factor))


def _run_clip(s):
    s["bound"] *= 0.97
    if own:
        sv = _package()
        out, _ = sv.spec_clip_grads(s["table"], max_norm=s["bound"], inf=bool(s["case"]["inf"]),
                                    grad_scale=s["grad_scale"], out=s["out"],
                                    workspace=_workspace(s, sv.spec_grad_norm_workspace()))
        s["grad_scale"].fill_(1.0)   # the gradients are unscaled now
        return out, s["grad"]
    norm, factor = _plain_norm(s, s["bound"])
    s["grad"].copy_(s["grad"].float() * factor)
    s["grad_scale"].fill_(1.0)
    return torch.stack((norm, factor)), s["grad"]


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "sample":
        R, V = sum(_rows(case)), case["V"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": R * V * size * (1 + case["filtered"]) + 16 * R, "flops": 4 * R * V}
    if op == "head4":
        M, K, N = case["M"], case["K"], case["N"]
        G = -(-K // case["group"])
        return {"bytes": N * -(-K // 2) + N * G * (2 + case["zeros"])
                + 2 * (M * K + M * N * (1 + case["residual"]) + N * case["bias"]),
                "flops": 2 * M * K * N}
    n = sum(_sizes(case))
    size = 4 if case["dtype"] == "f32" else 2
    # clipping has to know the norm before it writes: the gradients are read twice
    return {"bytes": n * size * (3 if op == "clip" else 1) + 8, "flops": 3 * n}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "head4": _exact_head4, "norm": _exact_norm, "clip": _exact_norm}[case["op"]](
        case, s)


def _exact_sample(case, s):
    R, V = s["logits"].shape
    tokens, kept = torch.empty(R, dtype=torch.int32, device=DEV), torch.empty(R, dtype=torch.int32, device=DEV)
    prob = torch.empty(R, dtype=torch.float64, device=DEV)
    filtered = torch.full((R, V), -math.inf, dtype=torch.float64, device=DEV) if case["filtered"] else None
    cu = s["cu_rows"].tolist()
    values = {n: s[n].tolist() if s[n] is not None else None for n in ("temperature", "top_k", "top_p", "min_p")}
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        T = values["temperature"][b]
        for r in range(lo, hi):
            z = s["logits"][r].double()
            if T < GREEDY_T:
                ids, law = z.argmax().view(1), torch.ones(1, dtype=torch.float64, device=DEV)
                ids = torch.nonzero(z == z[ids[0]])[0]
            else:
                law, ids = torch.sort(torch.log_softmax(z / T, 0), dim=0, descending=True, stable=True)
                # equal logits are neighbours and in the order of their ids
                law = law.exp()
                inside = z[ids] > -math.inf
                if values["min_p"] is not None and values["min_p"][b] > 0:
                    inside &= (z[ids[0]] - z[ids]) / T <= -math.log(values["min_p"][b])
                n = int(inside.sum())
                if values["top_k"] is not None and values["top_k"][b] > 0:
                    n = min(n, values["top_k"][b])
                ids, law = ids[:n], law[:n] / law[:n].sum()
                if values["top_p"] is not None and values["top_p"][b] < 1:
                    reach = torch.cumsum(law, 0) >= values["top_p"][b]
                    n = min(n, int((~reach).sum()) + 1)
                ids, law = ids[:n], law[:n] / law[:n].sum()
            kept[r] = ids.numel()
            if filtered is not None:
                filtered[r, ids] = z[ids]
            if s["uniform"] is not None:
                at = torch.searchsorted(torch.cumsum(law, 0), s["uniform"][r].double().view(1), right=True)
                at = at.clamp(max=ids.numel() - 1)
                tokens[r], prob[r] = ids[at][0], law[at][0]
    out = {"tokens": tokens, "prob": prob} if case["draw"] else {}
    out["kept"] = kept
    if filtered is not None:
        out["filtered"] = filtered
    return out


def _exact_head4(case, s):
    M, K, N, group = case["M"], case["K"], case["N"], case["group"]
    y = torch.empty(M, N, dtype=torch.float64, device=DEV)
    x = s["x"].double()
    column = torch.arange(K, device=DEV)
    for a in range(0, N, 8192):
        e = min(N, a + 8192)
        code = (s["codes"][a:e, column // 2].int() >> (4 * (column % 2)).int()) & 15
        zero = s["zeros"][a:e, column // group].double() if s["zeros"] is not None else 8.0
        y[:, a:e] = x @ ((code.double() - zero) * s["scales"][a:e, column // group].double()).t()
    if s["bias"] is not None:
        y += s["bias"].double()
    y = _act(y, case["act"])
    return y + s["residual"].double() if s["residual"] is not None else y


def _exact_norm(case, s):
    scale = float(s["grad_scale"][0])
    g = s["grad"].double()
    norm = scale * (float(g.abs().max()) if case["inf"] else math.sqrt(float((g * g).sum())))
    bound = s["bound"] * (0.97 if case["op"] == "clip" else 1.0)
    factor = scale * min(1.0, bound / (norm + CLIP_EPS))
    out = torch.tensor([norm, factor], dtype=torch.float64, device=DEV)
    return (out, g * factor) if case["op"] == "clip" else out
