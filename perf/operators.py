"""Timed cases of the draft-head operators.

One speculation round with a draft head that learns while it serves uses four
operators next to the verifier:

* rules     penalties, biases and grammar masks on the logits of a linear
            batch or a draft tree (spec_process_logits);
* distill   the weighted KL loss of the draft's logits against the target's,
            with its gradient (spec_distill_loss);
* head      a product with bias, activation and residual in its epilogue, and
            its backward pass (spec_head_forward, spec_head_backward);
* adamw     one AdamW step over many tensors at once, with states in 32 or in
            8 bits (spec_adamw_step).

A case is a dict of plain values; prepare() makes its inputs on the GPU from a
seed, run() is one pass, with `own` false in the plain form (elementary torch
operations in 32 bits), with `own` true through the package. exact() computes
the same outputs from the definitions in 64 bits.
"""
import itertools
import math

import torch

own = False

DEV = "cuda"
GREEDY_T = 0.05
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
FP8_MAX = 448.0          # largest e4m3 value
FP8_TINY = 2.0 ** -9     # smallest positive e4m3 value
BLOCK = 256              # elements that share one scale of an 8-bit state
TINY_ABSMAX = 2.0 ** -100


def _package():
    import speculative_decoding_rejection_gb300 as sv
    return sv


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a few requests with short rows: latency only
        dict(name="rules-B4-K4-V1024-f32", op="rules", B=4, k_lo=4, k_hi=4, V=1024, dtype="f32",
             hist=96, bias=8, grammar=2, tree=0, depth=0),
        # the nodes of 32 draft trees, every node with its own grammar state
        dict(name="rules-tree-B32-N64-V128256-bf16", op="rules", B=32, k_lo=63, k_hi=63, V=128256,
             dtype="bf16", hist=1500, bias=16, grammar=1, tree=1, depth=6),
        # the target rows of a full serving batch with ragged drafts, a quarter
        # of the requests under a grammar
        dict(name="rules-B1024-K1..5-V201088-bf16", op="rules", B=1024, k_lo=1, k_hi=5, V=201088,
             dtype="bf16", hist=700, bias=4, grammar=4, tree=0, depth=0),
        # ragged drafts of a mixed batch over an odd vocabulary
        dict(name="distill-B64-K1..5-V32003-bf16", op="distill", B=64, k_lo=1, k_hi=5, V=32003,
             dtype="bf16", masked=4, unused=5),
        # every draft position of a full serving batch
        dict(name="distill-B1024-K4-V201088-bf16", op="distill", B=1024, k_lo=4, k_hi=4, V=201088,
             dtype="bf16", masked=0, unused=4),
        # one token through the vocabulary projection: the weights are read once
        dict(name="head-M1-K4096-N32000", op="head", M=1, K=4096, N=32000, act="none", bias=1,
             residual=0, pre=0),
        # the residual block of a draft head over the rows of a ragged batch,
        # its pre-activation kept for the backward pass
        dict(name="head-M197-K2880-N2880-silu", op="head", M=197, K=2880, N=2880, act="silu", bias=1,
             residual=1, pre=1),
        # all rows of a large batch through the vocabulary projection
        dict(name="head-M1280-K4096-N128256", op="head", M=1280, K=4096, N=128256, act="none", bias=0,
             residual=0, pre=0),
        # the gradients of a training step through a projection with activation
        dict(name="head-backward-M1001-K2048-N32000", op="backward", M=1001, K=2048, N=32000,
             act="silu", bias=1),
        # a small draft head: few tensors of ragged sizes, states in 32 bits
        dict(name="adamw-12x20000-f32", op="adamw", tensors=12, numel=20000, dtype="f32", bits=32,
             master=0),
        # an f32 draft head of about 200 million weights
        dict(name="adamw-40x5000000-f32", op="adamw", tensors=40, numel=5000000, dtype="f32", bits=32,
             master=0),
        # bf16 weights with f32 masters, states in 8 bits
        dict(name="adamw-60x8000000-bf16-8bit", op="adamw", tensors=60, numel=8000000, dtype="bf16",
             bits=8, master=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rules", "rules", "distill", "head", "head", "backward", "adamw", "adamw"))
    if op in ("rules", "distill"):
        V = rng.choice((_log_int(rng, 500, 201088), rng.choice((32000, 128256, 151936, 201088))))
        dtype = rng.choice(("f32", "bf16", "bf16"))
        k_lo = rng.randint(0 if op == "rules" else 1, 4)
        k_hi = rng.randint(k_lo, 8)
        size = 4 if dtype == "f32" else 2
        most = 1.5e9 / (V * size * (k_hi + 1))
        B = max(1, min(_log_int(rng, 1, 1024), int(most)))
        if op == "distill":
            return dict(op=op, B=B, k_lo=k_lo, k_hi=k_hi, V=V, dtype=dtype, masked=rng.choice((0, 3, 4)),
                        unused=rng.choice((0, 3, 5)))
        tree = rng.randint(0, 2) // 2
        depth = 0
        if tree:
            k_lo = k_hi = rng.randint(7, 63)
            depth = rng.randint(2, 8)
            B = max(1, min(B, 64, int(1.5e9 / (V * size * (k_hi + 1)))))
        return dict(op=op, B=B, k_lo=k_lo, k_hi=k_hi, V=V, dtype=dtype, hist=_log_int(rng, 1, 4000),
                    bias=rng.choice((0, 5, 40)), grammar=rng.choice((0, 1, 2, 4)), tree=tree, depth=depth)
    if op in ("head", "backward"):
        M = _log_int(rng, 1, 2048)
        K = _log_int(rng, 64, 5120)
        N = _log_int(rng, 64, 60000)
        act = rng.choice(("none", "silu", "gelu"))
        bias = rng.randint(0, 1)
        if op == "backward":
            return dict(op=op, M=M, K=K, N=min(N, 32000), act=act, bias=bias)
        return dict(op=op, M=M, K=K, N=N, act=act, bias=bias, residual=rng.randint(0, 1),
                    pre=rng.randint(0, 1))
    dtype = rng.choice(("f32", "bf16"))
    bits = rng.choice((8, 32))
    tensors = _log_int(rng, 1, 200)
    numel = max(100, min(_log_int(rng, 300, 8000000), 200000000 // tensors))
    return dict(op=op, tensors=tensors, numel=numel, dtype=dtype, bits=bits,
                master=rng.randint(0, 1) if dtype == "bf16" else 0)


# ---------------------------------------------------- sizes that a case fixes
def _lengths(case):
    """Drafts of each request (or nodes less the root of each tree)."""
    lo, hi = case["k_lo"], case["k_hi"]
    return [lo + (b * 7919 + 3) % (hi - lo + 1) for b in range(case["B"])]


def _history_lengths(case):
    """Ragged histories about the case's length; one in eight requests is new."""
    h = case["hist"]
    return [0 if b % 8 == 5 else 1 + (b * 2654435761 + h) % (2 * h) for b in range(case["B"])]


def _sizes(case):
    """Ragged tensor sizes about the case's, odd ones among them."""
    n = case["numel"]
    return [max(1, int(n * (0.2 + 1.6 * ((i + 1) * 0.6180339887 % 1.0)))) + i % 2
            for i in range(case["tensors"])]


def _offsets(lengths):
    return list(itertools.accumulate(lengths, initial=0))


def _ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device=DEV)


def _zipf_tokens(n, V, g):
    """Token ids with the uneven frequencies of running text."""
    u = torch.rand(n, generator=g, device=DEV)
    rank = torch.exp(u * math.log(V)).to(torch.int64).clamp_(1, V) - 1
    return ((rank * 7919 + 11) % V).to(torch.int32)


def _rand_logits(rows, V, dtype, g):
    out = torch.empty(rows, V, dtype=DTYPES[dtype], device=DEV)
    step = max(1, (1 << 28) // V)
    for s in range(0, rows, step):
        e = min(rows, s + step)
        out[s:e] = torch.randn(e - s, V, generator=g, device=DEV) * 2.0
    return out


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    s = {"case": case, "op": case["op"]}
    {"rules": _prepare_rules, "distill": _prepare_distill, "head": _prepare_head,
     "backward": _prepare_backward, "adamw": _prepare_adamw}[case["op"]](s, case, g)
    return s


def _prepare_rules(s, case, g):
    B, V = case["B"], case["V"]
    K = _lengths(case)
    cu_rows = _offsets([k + 1 for k in K])
    R = cu_rows[-1]
    s["max_rows"] = max(K) + 1
    s["logits"] = _rand_logits(R, V, case["dtype"], g)
    s["cu_rows"] = _ints(cu_rows)
    hist = _history_lengths(case)
    cu_hist = _offsets(hist)
    s["cu_history"] = _ints(cu_hist)
    s["history"] = _zipf_tokens(cu_hist[-1], V, g)
    s["prompt_len"] = _ints(h // 3 for h in hist)
    if case["tree"]:
        n = K[0] + 1
        s["tokens"] = _zipf_tokens(R, V, g)
        s["cu_tokens"] = None
        parent, depth = [-1], [0]
        for v in range(1, n):
            at = (v - 1) // 3
            at = at if depth[at] < case["depth"] - 1 else 0
            parent.append(at)
            depth.append(depth[at] + 1)
        s["parent"] = _ints(parent * B)
    else:
        s["tokens"] = _zipf_tokens(sum(K), V, g)
        s["cu_tokens"] = _ints(_offsets(K))
        s["parent"] = None
    s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=DEV)
    s["frequency"] = 0.8 * torch.rand(B, generator=g, device=DEV) - 0.1
    s["presence"] = 0.6 * torch.rand(B, generator=g, device=DEV)
    s["bias_ids"] = s["bias_values"] = s["cu_bias"] = None
    if case["bias"]:
        n = [(b * 31 + case["bias"]) % (2 * case["bias"] + 1) for b in range(B)]
        cu = _offsets(n)
        stride = max(1, V // (2 * case["bias"] + 1))
        s["cu_bias"] = _ints(cu)
        s["bias_ids"] = _ints((i * stride + b) % V for b in range(B) for i in range(n[b]))
        s["bias_values"] = 8.0 * torch.rand(cu[-1], generator=g, device=DEV) - 5.0
    s["mask"] = s["mask_rows"] = None
    if case["grammar"]:
        rows = [b for b in range(B) for _ in range(K[b] + 1)]
        with_mask = [b % case["grammar"] == 0 for b in rows]
        index = list(itertools.accumulate(with_mask, initial=0))[:-1]
        s["mask_rows"] = _ints(i if m else -1 for i, m in zip(index, with_mask))
        M, W = sum(with_mask), -(-V // 32)
        words = torch.randint(-2 ** 31, 2 ** 31, (M, W), generator=g, device=DEV, dtype=torch.int64)
        # grammar states allow few tokens, or all but few, in runs of ids
        runs = (torch.arange(W, device=DEV)[None, :] // 16 + torch.arange(M, device=DEV)[:, None]) % 5
        words = torch.where(runs == 0, words, torch.where(runs == 1, -1, 0))
        s["mask"] = words.to(torch.int32)
    s["out"] = torch.empty_like(s["logits"])


def _prepare_distill(s, case, g):
    B, V = case["B"], case["V"]
    K = _lengths(case)
    R = sum(K)
    s["cu_draft"] = _ints(_offsets(K))
    s["target"] = _rand_logits(R + B, V, case["dtype"], g)
    t_row = torch.arange(R, device=DEV) + torch.repeat_interleave(
        torch.arange(B, device=DEV), torch.tensor(K, device=DEV))
    s["draft"] = torch.empty(R, V, dtype=DTYPES[case["dtype"]], device=DEV)
    step = max(1, (1 << 28) // V)
    for a in range(0, R, step):
        e = min(R, a + step)
        s["draft"][a:e] = s["target"][t_row[a:e]].float() + 0.7 * torch.randn(
            e - a, V, generator=g, device=DEV)
    s["temperature"] = 0.6 + 0.8 * torch.rand(B, generator=g, device=DEV)
    weight = torch.rand(R, generator=g, device=DEV) / max(R, 1)
    if case["unused"]:   # positions after a rejection, which no loss counts
        weight[torch.arange(R, device=DEV) % case["unused"] == case["unused"] - 1] = 0.0
    s["weight"] = weight
    if case["masked"]:   # tokens that a grammar forbids, in both rows of a pair
        banned = torch.rand(V, generator=g, device=DEV) < 1.0 / case["masked"]
        banned[0] = False
        s["target"][:, banned] = -math.inf
        s["draft"][:, banned] = -math.inf
    s["loss"] = torch.empty(R, dtype=torch.float32, device=DEV)
    s["grad"] = torch.empty_like(s["draft"])


def _normal(shape, scale, g):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 27):
        e = min(flat.numel(), a + (1 << 27))
        flat[a:e] = scale * torch.randn(e - a, generator=g, device=DEV)
    return out


def _prepare_head(s, case, g):
    M, K, N = case["M"], case["K"], case["N"]
    s["x"] = _normal((M, K), 1.0, g)
    s["weight"] = _normal((N, K), 1.0 / math.sqrt(K), g)
    s["bias"] = _normal((N,), 0.5, g) if case["bias"] else None
    s["residual"] = _normal((M, N), 1.0, g) if case["residual"] else None
    s["y"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    s["pre"] = torch.empty_like(s["y"]) if case["pre"] else None


def _prepare_backward(s, case, g):
    M, K, N = case["M"], case["K"], case["N"]
    s["x"] = _normal((M, K), 1.0, g)
    s["weight"] = _normal((N, K), 1.0 / math.sqrt(K), g)
    s["pre"] = _normal((M, N), 1.0, g) if case["act"] != "none" else None
    s["dy"] = _normal((M, N), 1.0 / math.sqrt(N), g)
    s["dx"] = torch.empty_like(s["x"])
    s["dw"] = torch.empty_like(s["weight"])
    s["db"] = torch.empty(N, dtype=torch.float32, device=DEV) if case["bias"] else None


def _prepare_adamw(s, case, g):
    sizes = _sizes(case)
    at = _offsets([-(-n // BLOCK) * BLOCK for n in sizes])   # one flat buffer, padded with zeros
    total = at[-1]
    dtype = DTYPES[case["dtype"]]
    valid = torch.zeros(total, dtype=torch.bool, device=DEV)
    for a, n in zip(at, sizes):
        valid[a:a + n] = True

    def values(scale):
        return (scale * torch.randn(total, generator=g, device=DEV)).mul_(valid)

    master = values(0.05)
    s["grad"] = values(0.01).to(dtype)
    m, v = values(0.003), values(0.01).square_()
    s["param"] = master.to(dtype)
    s["master"] = master if case["master"] else None
    if case["bits"] == 8:
        s["exp_avg"], s["exp_avg_scale"] = _pack_signed(m)
        s["exp_avg_sq"], s["exp_avg_sq_scale"] = _pack_root(v)
    else:
        s["exp_avg"], s["exp_avg_sq"] = m, v
        s["exp_avg_scale"] = s["exp_avg_sq_scale"] = None
    s["step"] = 10
    s["grad_scale"] = torch.tensor([0.25], device=DEV)
    s["hyper"] = dict(lr=3e-4, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01)

    def views(t, per=1):
        return None if t is None else [t[a // per:a // per + -(-n // per)] for a, n in zip(at, sizes)]

    # the table of tensors that a training program builds once
    s["table"] = _package().spec_adamw_table(
        views(s["param"]), views(s["grad"]), views(s["exp_avg"]), views(s["exp_avg_sq"]),
        exp_avg_scale=views(s["exp_avg_scale"], BLOCK), exp_avg_sq_scale=views(s["exp_avg_sq_scale"], BLOCK),
        master=views(s["master"])) if own else None


# ---------------------------------------------------------------- the passes
def run(state):
    return {"rules": _run_rules, "distill": _run_distill, "head": _run_head,
            "backward": _run_backward, "adamw": _run_adamw}[state["op"]](state)


def _workspace(s, size):
    """The scratch that a serving program keeps from call to call."""
    if s.get("workspace") is None:
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return s["workspace"]


# ----------------------------------------------------- rules on the logits
def _run_rules(s):
    if own:
        sv = _package()
        out, _ = sv.spec_process_logits(
            s["logits"], s["cu_rows"], max_rows=s["max_rows"], history=s["history"],
            cu_history=s["cu_history"], prompt_len=s["prompt_len"], tokens=s["tokens"],
            cu_tokens=s["cu_tokens"], parent=s["parent"], repetition=s["repetition"],
            frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
            bias_values=s["bias_values"], cu_bias=s["cu_bias"], mask=s["mask"],
            mask_rows=s["mask_rows"], out=s["out"],
            workspace=_workspace(s, sv.spec_process_logits_workspace()))
        return out
    z = s["logits"].float()
    R, V = z.shape
    B = s["cu_rows"].numel() - 1
    cu = s["cu_rows"].long()
    req = torch.repeat_interleave(torch.arange(B, device=DEV), cu[1:] - cu[:-1], output_size=R)
    pos = torch.arange(R, device=DEV) - cu[req]
    # counts over each request's history: all of it, and the generated part
    H = s["history"].numel()
    ch = s["cu_history"].long()
    hreq = torch.repeat_interleave(torch.arange(B, device=DEV), ch[1:] - ch[:-1], output_size=H)
    made = (torch.arange(H, device=DEV) - ch[hreq] >= s["prompt_len"].long()[hreq]).float()
    at = hreq * V + s["history"].long()
    made_count = torch.zeros(B * V, device=DEV).index_add_(0, at, made).view(B, V)
    any_count = torch.zeros(B * V, device=DEV).index_add_(0, at, torch.ones_like(made)).view(B, V)
    # the tokens between the request's history and the row
    if s["parent"] is not None:
        parent = s["parent"].long()
        depth = s["case"]["depth"]
        path = itertools.accumulate(
            range(depth - 1),
            lambda node, _: torch.where(pos.gather(0, node) > 0, cu[req] + parent[node].clamp(min=0), node),
            initial=torch.arange(R, device=DEV))
        nodes = torch.stack(list(path), 1)
        is_new = pos[nodes] > 0
        extra = s["tokens"].long()[nodes]
    else:
        ct = s["cu_tokens"].long()
        j = torch.arange(max(1, s["max_rows"] - 1), device=DEV)[None, :]
        is_new = j < torch.minimum(pos, (ct[1:] - ct[:-1])[req])[:, None]
        if s["tokens"].numel():
            extra = s["tokens"].long()[(ct[req][:, None] + j).clamp(max=s["tokens"].numel() - 1)]
        else:
            extra = torch.zeros_like(is_new, dtype=torch.int64)
    is_new = is_new.float()
    count = made_count[req].scatter_add_(1, extra, is_new)
    seen = any_count[req].scatter_add_(1, extra, is_new) > 0
    if s["bias_ids"] is not None:
        nb = s["bias_ids"].numel()
        cb = s["cu_bias"].long()
        breq = torch.repeat_interleave(torch.arange(B, device=DEV), cb[1:] - cb[:-1], output_size=nb)
        bias = torch.zeros(B * V, device=DEV).index_add_(0, breq * V + s["bias_ids"].long(),
                                                         s["bias_values"])
        z = z + bias.view(B, V)[req]
    rho = s["repetition"][req][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
    z = z - s["frequency"][req][:, None] * count - s["presence"][req][:, None] * (count > 0)
    if s["mask"] is not None:
        row = s["mask_rows"].long()
        words = s["mask"][row.clamp(min=0)].repeat_interleave(32, dim=1)[:, :V]
        allowed = ((words >> (torch.arange(V, device=DEV, dtype=torch.int32) % 32)) & 1) != 0
        z = torch.where(allowed | (row < 0)[:, None], z, -math.inf)
    return z.to(s["logits"].dtype)


# -------------------------------------------------- loss and its gradient
def _run_distill(s):
    if own:
        sv = _package()
        loss, grad, _ = sv.spec_distill_loss(
            s["target"], s["draft"], s["cu_draft"], s["temperature"], s["weight"],
            out=(s["loss"], s["grad"]),
            workspace=_workspace(s, sv.spec_distill_loss_workspace(*s["draft"].shape)))
        return loss, grad
    R = s["draft"].shape[0]
    cu = s["cu_draft"].long()
    B = cu.numel() - 1
    req = torch.repeat_interleave(torch.arange(B, device=DEV), cu[1:] - cu[:-1], output_size=R)
    T = s["temperature"][req][:, None]
    T = torch.where(T < GREEDY_T, 1.0, T)
    w = s["weight"]
    zt = s["target"][torch.arange(R, device=DEV) + req].float() / T
    zd = s["draft"].float() / T
    log_p = zt - zt.amax(1, keepdim=True)
    log_p = log_p - log_p.exp().sum(1, keepdim=True).log()
    log_q = zd - zd.amax(1, keepdim=True)
    log_q = log_q - log_q.exp().sum(1, keepdim=True).log()
    p, q = log_p.exp(), log_q.exp()
    kl = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(1, dtype=torch.float64)
    loss = torch.where(w != 0, w * kl, 0.0).float()
    grad = torch.where(w[:, None] != 0, (w[:, None] / T) * (q - p), 0.0).to(s["draft"].dtype)
    return loss, grad


# ------------------------------------------------ product with an epilogue
def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _act_code(sv, act):
    return {"none": sv.SPEC_ACT_NONE, "silu": sv.SPEC_ACT_SILU, "gelu": sv.SPEC_ACT_GELU}[act]


def _run_head(s):
    c = s["case"]
    if own:
        sv = _package()
        y, pre, _ = sv.spec_head_forward(
            s["x"], s["weight"], s["bias"], s["residual"], act=_act_code(sv, c["act"]),
            out=(s["y"], s["pre"]),
            workspace=_workspace(s, sv.spec_head_forward_workspace(c["M"], c["N"], c["K"])))
        return (y, pre) if c["pre"] else (y,)
    z = s["x"].float() @ s["weight"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(torch.bfloat16)
    return (y, z.to(torch.bfloat16)) if c["pre"] else (y,)


def _run_backward(s):
    c = s["case"]
    if own:
        sv = _package()
        dx, dw, db, _ = sv.spec_head_backward(
            s["dy"], s["x"], s["weight"], s["pre"], act=_act_code(sv, c["act"]),
            out=(s["dx"], s["dw"], s["db"]),
            workspace=_workspace(s, sv.spec_head_backward_workspace(c["M"], c["N"], c["K"])))
        return (dx, dw, db) if c["bias"] else (dx, dw)
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["pre"].float(), c["act"])
    dx = (dz @ s["weight"].float()).to(torch.bfloat16)
    dw = (dz.t() @ s["x"].float()).to(torch.bfloat16)
    return (dx, dw, dz.sum(0)) if c["bias"] else (dx, dw)


# ------------------------------------------------------------- AdamW step
def _pack_signed(m):
    """e4m3 codes of m over the largest magnitude of each block, and the scales."""
    m = m.view(-1, BLOCK)
    most = m.abs().amax(1, keepdim=True)
    flat = most < TINY_ABSMAX
    code = (m * torch.where(flat, 0.0, FP8_MAX / most)).to(torch.float8_e4m3fn)
    return code.view(-1), torch.where(flat, 0.0, most / FP8_MAX).view(-1)


def _pack_root(v):
    """The same for the square root of v, of which nothing positive becomes zero."""
    r = v.sqrt().view(-1, BLOCK)
    most = r.amax(1, keepdim=True)
    flat = most < TINY_ABSMAX
    code = r * torch.where(flat, 0.0, FP8_MAX / most)
    code = torch.where((r > 0) & ~flat, code.clamp(min=FP8_TINY), code).to(torch.float8_e4m3fn)
    return code.view(-1), torch.where(flat, 0.0, most / FP8_MAX).view(-1)


def _run_adamw(s):
    h = s["hyper"]
    s["step"] += 1
    names = [n for n in ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
             if s[n] is not None]
    if own:
        sv = _package()
        sv.spec_adamw_step(s["table"], s["step"], grad_scale=s["grad_scale"],
                           workspace=_workspace(s, 256), **h)
        return {n: s[n] for n in names}
    g = s["grad"].float() * s["grad_scale"]
    p = s["master"] if s["master"] is not None else s["param"].float()
    if s["case"]["bits"] == 8:
        m = (s["exp_avg"].float().view(-1, BLOCK) * s["exp_avg_scale"][:, None]).view(-1)
        v = (s["exp_avg_sq"].float().view(-1, BLOCK) * s["exp_avg_sq_scale"][:, None]).view(-1).square_()
    else:
        m, v = s["exp_avg"], s["exp_avg_sq"]
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * (g * g)
    c1 = 1 - h["beta1"] ** s["step"]
    c2 = math.sqrt(1 - h["beta2"] ** s["step"])
    p = p * (1 - h["lr"] * h["weight_decay"]) - (h["lr"] / c1) * m / (v.sqrt() / c2 + h["eps"])
    s["param"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if s["case"]["bits"] == 8:
        for name, (code, scale) in (("exp_avg", _pack_signed(m)), ("exp_avg_sq", _pack_root(v))):
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
    else:
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
    return {n: s[n] for n in names}


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("rules", "distill"):
        K, V = _lengths(case), case["V"]
        size = 4 if case["dtype"] == "f32" else 2
        if op == "distill":
            R = sum(K)
            used = R - (sum(1 for r in range(R) if r % case["unused"] == case["unused"] - 1)
                        if case["unused"] else 0)
            return {"bytes": 2 * used * V * size + R * V * size + 8 * R, "flops": 12 * used * V}
        R = sum(K) + case["B"]
        masked = sum(k + 1 for b, k in enumerate(K) if case["grammar"] and b % case["grammar"] == 0)
        return {"bytes": 2 * R * V * size + masked * 4 * -(-V // 32) + 4 * sum(_history_lengths(case)),
                "flops": R * V}
    if op == "head":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * (M * K + N * K + M * N * (1 + case["residual"] + case["pre"]) + N * case["bias"]),
                "flops": 2 * M * K * N}
    if op == "backward":
        M, K, N = case["M"], case["K"], case["N"]
        passes = 2 if case["act"] != "none" else 1
        return {"bytes": 2 * (M * K * 2 + N * K * 2 + M * N * passes) + 4 * N * case["bias"],
                "flops": 4 * M * K * N}
    n = sum(_sizes(case))
    size = 4 if case["dtype"] == "f32" else 2
    per = 3 * size + (4 + 16 / BLOCK if case["bits"] == 8 else 16)
    if case["master"]:
        per += 8 - size   # the f32 master is read and written, the bf16 weight only written
    return {"bytes": n * per, "flops": 20 * n}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"rules": _exact_rules, "distill": _exact_distill, "head": _exact_head,
            "backward": _exact_backward, "adamw": _exact_adamw}[case["op"]](case, s)


def _exact_rules(case, s):
    V = case["V"]
    out = s["logits"].double()
    cu, ch = s["cu_rows"].tolist(), s["cu_history"].tolist()
    ct = s["cu_tokens"].tolist() if s["cu_tokens"] is not None else None
    cb = s["cu_bias"].tolist() if s["cu_bias"] is not None else None
    parent = s["parent"].tolist() if s["parent"] is not None else None
    mask_rows = s["mask_rows"].tolist() if s["mask_rows"] is not None else None
    bit = torch.arange(32, device=DEV, dtype=torch.int32)
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        hist = s["history"][ch[b]:ch[b + 1]].long()
        made = hist[int(s["prompt_len"][b]):]
        base_any = torch.bincount(hist, minlength=V)
        base_made = torch.bincount(made, minlength=V)
        rho, freq, pres = (s[n][b].double() for n in ("repetition", "frequency", "presence"))
        for r in range(lo, hi):
            if parent is None:
                new = s["tokens"][ct[b]:min(ct[b] + r - lo, ct[b + 1])].long()
            else:
                path, node = [], r - lo
                while node > 0:
                    path.append(lo + node)
                    node = parent[lo + node]
                new = s["tokens"][torch.tensor(path, dtype=torch.int64, device=DEV)].long()
            more = torch.bincount(new, minlength=V)
            z = out[r]
            if cb is not None:
                z.index_add_(0, s["bias_ids"][cb[b]:cb[b + 1]].long(),
                             s["bias_values"][cb[b]:cb[b + 1]].double())
            at = torch.nonzero(base_any + more).view(-1)
            v = z[at]
            v = torch.where(v > 0, v / rho, v * rho)
            n = (base_made + more)[at].double()
            z[at] = v - freq * n - pres * (n > 0).double()
            if mask_rows is not None and mask_rows[r] >= 0:
                words = s["mask"][mask_rows[r]]
                z.masked_fill_((((words[:, None] >> bit) & 1) == 0).reshape(-1)[:V], -math.inf)
    return out


def _exact_distill(case, s):
    R = s["draft"].shape[0]
    loss = torch.zeros(R, dtype=torch.float64, device=DEV)
    grad = torch.zeros(s["draft"].shape, dtype=torch.float64, device=DEV)
    cu = s["cu_draft"].tolist()
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        T = s["temperature"][b].double()
        w = s["weight"][lo:hi].double()
        zt = s["target"][lo + b:hi + b].double() / T
        zd = s["draft"][lo:hi].double() / T
        lp = zt - torch.logsumexp(zt, 1, keepdim=True)
        lq = zd - torch.logsumexp(zd, 1, keepdim=True)
        term = lp.exp() * (lp - lq)
        loss[lo:hi] = w * torch.where(lp > -math.inf, term, 0.0).sum(1)
        grad[lo:hi] = (w / T)[:, None] * (lq.exp() - lp.exp())
    return loss, grad


def _exact_head(case, s):
    z = s["x"].double() @ s["weight"].double().t()
    if s["bias"] is not None:
        z += s["bias"].double()
    if case["act"] == "silu":
        y = z * torch.sigmoid(z)
    elif case["act"] == "gelu":
        y = torch.nn.functional.gelu(z, approximate="tanh")
    else:
        y = z
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return (y, z) if case["pre"] else (y,)


def _exact_backward(case, s):
    dz = s["dy"].double()
    if case["act"] != "none":
        with torch.enable_grad():
            pre = s["pre"].double().requires_grad_()
            y = (pre * torch.sigmoid(pre) if case["act"] == "silu"
                 else torch.nn.functional.gelu(pre, approximate="tanh"))
            dz, = torch.autograd.grad(y, pre, dz)
    dx = dz @ s["weight"].double()
    dw = dz.t() @ s["x"].double()
    return (dx, dw, dz.sum(0)) if case["bias"] else (dx, dw)


def _exact_adamw(case, s):
    h, t = s["hyper"], s["step"] + 1
    g = s["grad"].double() * s["grad_scale"].double()
    p = (s["master"] if case["master"] else s["param"]).double()
    m, v = s["exp_avg"].double(), s["exp_avg_sq"].double()
    if case["bits"] == 8:
        m = m * s["exp_avg_scale"].double().repeat_interleave(BLOCK)
        v = (v * s["exp_avg_sq_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = m + (1 - h["beta1"]) * (g - m)
    v = v + (1 - h["beta2"]) * (g * g - v)
    m_hat = m / (1 - math.pow(h["beta1"], t))
    v_hat = v / (1 - math.pow(h["beta2"], t))
    p = p - h["lr"] * (m_hat / (v_hat.sqrt() + h["eps"]) + h["weight_decay"] * p)
    out = {"param": p, "exp_avg": m, "exp_avg_sq": v}
    if case["master"]:
        out["master"] = p
    if case["bits"] == 8:
        for name, x in (("exp_avg", m), ("exp_avg_sq", v.sqrt())):
            most = x.abs().view(-1, BLOCK).amax(1)
            out[name + "_scale"] = most / FP8_MAX
            code = x.view(-1, BLOCK) * torch.where(most > 0, FP8_MAX / most, 0.0)[:, None]
            if name == "exp_avg_sq":
                code = torch.where(x.view(-1, BLOCK) > 0, code.clamp(min=FP8_TINY), code)
            out[name] = code.float().to(torch.float8_e4m3fn).view(-1)
    return out
