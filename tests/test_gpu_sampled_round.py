"""A round of drafting with a head in 4 bits, under each request's law, from the draws to the
head's next step: every operator's result against the 64-bit reference of what it was given,
the tokens that are committed against the target's law, and the whole round in a CUDA
graph."""
import numpy as np
import pytest
import torch

import speculative_decoding_rejection_gb300 as sv
from oracle import draft_oracle as O
from oracle import spec_oracle as V_

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, I32 = torch.bfloat16, torch.int32
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01)


def f64(t):
    return t.double().cpu().numpy()


class Round:
    """B requests, K drafts each, a head [V, H] held in bf16 to learn and in 4 bits to draft."""

    def __init__(self, B, K, H, V, group, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *n: torch.randn(*n, generator=g, device=DEV)   # noqa: E731
        self.B, self.K, self.H, self.V, self.group = B, K, H, V, group
        self.states = rand(B, K, H).to(BF16)
        self.w = (3 * H ** -0.5 * rand(V, H)).to(BF16)
        self.bias = (0.1 * rand(V)).to(BF16)
        self.target_raw = (2 * rand(B * (K + 1), V)).to(BF16)
        self.target_raw[:, ::17] = -1e30                      # tokens that no request may have
        self.u = torch.rand(K, B, generator=g, device=DEV)
        self.law = dict(temperature=torch.rand(B, generator=g, device=DEV) + 0.4,
                        top_k=torch.arange(B, device=DEV, dtype=I32) * 7,
                        top_p=1 - 0.4 * torch.rand(B, generator=g, device=DEV),
                        min_p=torch.where(torch.arange(B, device=DEV) % 2 == 0, 0.0, 0.01))
        self.cu_draft = torch.arange(0, B * K + 1, K, dtype=I32, device=DEV)
        self.cu_target = torch.arange(0, B * (K + 1) + 1, K + 1, dtype=I32, device=DEV)
        self.packed, _ = sv.spec_head4_quantize(self.w, group=group)
        self.first_packed = self.packed.packed.clone()
        self.dw = torch.zeros_like(self.w)
        self.db = torch.zeros(V, device=DEV)
        self.db16 = torch.zeros_like(self.bias)
        params, grads = [self.w, self.bias], [self.dw, self.db16]
        codes = [[torch.zeros(p.numel(), dtype=torch.uint8, device=DEV) for p in params] for _ in range(2)]
        scales = [[torch.zeros(-(-p.numel() // sv.SPEC_ADAMW_BLOCK), device=DEV) for p in params] for _ in range(2)]
        self.master = [p.float() for p in params]
        self.states8 = codes + scales
        self.table = sv.spec_adamw_table(params, grads, *codes, exp_avg_scale=scales[0], exp_avg_sq_scale=scales[1],
                                         master=self.master)
        self.start = [t.clone() for t in params + self.master]

    def restart(self):
        for t, s in zip([self.w, self.bias] + self.master, self.start):
            t.copy_(s)
        for t in [t for group in self.states8 for t in group]:
            t.zero_()
        self.packed.packed.copy_(self.first_packed)

    def draft(self):
        """(logits, tokens, prob, kept, filtered) of each step, by rows [B]."""
        steps = []
        for i in range(self.K):
            logits, _ = sv.spec_head4_forward(self.states[:, i].contiguous(), self.packed, self.bias)
            steps.append((logits,) + sv.spec_sample(logits, self.u[i], want_kept=True, want_filtered=True, **self.law))
        return steps

    def verify(self, steps):
        tokens = torch.stack([s[1] for s in steps], 1).reshape(-1)
        draft = torch.stack([s[4] for s in steps], 1).reshape(self.B * self.K, self.V)
        target = sv.spec_sample(self.target_raw, None, self.cu_target, want_filtered=True, **self.law)[3]
        out = sv.spec_verify_linear(target, draft, tokens, self.cu_draft, self.law["temperature"], 77, max_k=self.K)
        return tokens, draft, target, out

    def learn(self):
        x = self.states.reshape(-1, self.H)
        logits, _, _ = sv.spec_head_forward(x, self.w, self.bias)
        loss, grad, _ = sv.spec_distill_loss(self.target_raw, logits, self.cu_draft, self.law["temperature"])
        sv.spec_head_backward(grad, x, self.w, out=(None, self.dw, self.db))
        self.db16.copy_(self.db)
        norm, _ = sv.spec_grad_norm(self.table, max_norm=0.5)
        sv.spec_adamw_step(self.table, 1, grad_scale=norm[1:], **HYPER)
        sv.spec_head4_quantize(self.w, group=self.group, out=self.packed)
        return logits, grad, norm

    def all(self):
        steps = self.draft()
        return steps, self.verify(steps), self.learn()


SIZES = [(5, 3, 160, 1003, 32), (1, 1, 128, 515, 128), (12, 4, 200, 32000, 64)]


@pytest.mark.parametrize("B,K,H,V,group", SIZES)
def test_a_round(B, K, H, V, group):
    r = Round(B, K, H, V, group, B + V)
    codes, scales = O.quantize4(f64(r.w), group)
    w4 = O.dequantize4(codes, scales, None, group)
    steps, (tokens, draft, target, verified), (logits, grad, norm) = r.all()
    law = {k: f64(v) for k, v in r.law.items()}

    def laws(z, b, u=None):
        return O.sample_row(z, u, law["temperature"][b], int(law["top_k"][b]), law["top_p"][b], law["min_p"][b])

    for i, (z, tok, prob, kept, rows, ws) in enumerate(steps):
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        # the head's products: 32-bit sums, a step of 2^-22 of the magnitudes for each 16 columns and
        # what joins them, one rounding to bf16
        x, b16 = f64(r.states[:, i]), f64(r.start[1])
        want, size = x @ w4.T + b16, np.abs(x) @ np.abs(w4).T + np.abs(b16)
        err = (H // 16 + 40) * 2.0 ** -22 * size
        assert np.all(np.abs(f64(z) - want) <= err + 2.0 ** -8 * (np.abs(want) + err))
        for b in range(B):
            ref = laws(f64(z[b]), b, float(r.u[i, b]))
            assert ref["edge"] > 2.0 ** -36 and ref["edge_u"] > 2.0 ** -36
            assert int(tok[b]) == ref["token"] and int(kept[b]) == len(ref["order"])
            assert abs(float(prob[b]) - ref["prob"]) <= 2.0 ** -23 * ref["prob"]
            on = np.zeros(V, bool)
            on[ref["order"]] = True
            assert torch.equal(rows[b], torch.where(torch.tensor(on, device=DEV), z[b], -np.inf))
    # the target's rows of a request under its law, and what the verifier makes of both
    out, accepted, _, ws = verified
    assert sv.spec_get_status(ws) == sv.SPEC_OK
    ref = V_.verify_linear(target.cpu(), draft.cpu(), tokens.cpu().numpy(), r.cu_draft.cpu().numpy(),
                           r.law["temperature"].cpu().numpy(), 77, max_k=K)
    for b in range(B):
        kept_at = []
        for i in range(K + 1):
            on = laws(f64(r.target_raw[b * (K + 1) + i]), b)
            assert on["edge"] > 2.0 ** -36
            kept_at.append(set(on["order"].tolist()))
            assert set(torch.nonzero(target[b * (K + 1) + i] > -np.inf).flatten().tolist()) == kept_at[-1]
        n = int(accepted[b])
        assert all(int(t) in kept_at[i] for i, t in enumerate(out[b, :n + 1]))
        flag = int(ref["flag_slot"][b])
        end = K + 1 if flag < 0 else flag
        assert out[b, :end].tolist() == ref["tokens"][b, :end].tolist()
    # the gradients' norm (sums of squares in two words: within 2^-22), and the step by its factor
    grads = [f64(r.dw), f64(r.db16)]
    want, factor = O.grad_norm(grads, 0.5)
    assert abs(float(norm[0]) - want) <= 2.0 ** -22 * want and abs(float(norm[1]) - factor) <= 2.0 ** -21 * factor
    for p, m, start, g in zip((r.w, r.bias), r.master, r.start[2:], grads):
        ref_w, _, _ = O.adamw(f64(start), g, 0.0, 0.0, 1, grad_scale=float(norm[1]), **HYPER)
        assert torch.equal(p, m.to(BF16))
        # weights of magnitude 1 and steps of lr in 32 bits, a few roundings each
        assert np.all(np.abs(f64(m) - ref_w) <= 8 * 2.0 ** -24 * (np.abs(ref_w) + 2 * HYPER["lr"]))
    codes, scales = O.quantize4(f64(r.w), group)
    assert np.array_equal(f64(sv.spec_head4_unpack(r.packed)),
                          O.to_bf16(O.dequantize4(codes, scales, None, group)))


def test_a_round_in_a_graph():
    r = Round(6, 2, 144, 4001, 64, 5)
    flat = lambda x: [t for y in x for t in (flat(y) if isinstance(y, (tuple, list)) else [y]) if t is not None]  # noqa: E731
    eager = [t.clone() for t in flat(r.all()) if t.dtype != torch.uint8]
    after = [t.clone() for t in (r.w, r.master[0], r.packed.packed)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.restart()
    with torch.cuda.stream(side):
        r.all()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = r.all()
    for _ in range(2):
        r.restart()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, [t for t in flat(got) if t.dtype != torch.uint8]):
            assert torch.equal(a, b)
        for a, b in zip(after, (r.w, r.master[0], r.packed.packed)):
            assert torch.equal(a, b)
