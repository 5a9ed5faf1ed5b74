"""A draft head that learns while it serves, on a toy target.

Every round drafts K tokens per request with a small head, applies the
requests' rules and laws (top-k, top-p, min-p) to the draft's and the target's
logits, verifies the drafts, commits what was accepted, and takes one
distillation step of the head on the target's logits ("Test-Time Speculation",
§2). All of it runs in the package's kernels: the head's products
(spec_head_forward, spec_head_backward; the drafts' from a copy of the
vocabulary's weights in 4 bits, spec_head4_forward, rounded anew after every
step), the rules (spec_process_logits), the draws and the laws' rows
(spec_sample), the verification (spec_verify_linear), the loss with its gradient
(spec_distill_loss), the gradients' norm (spec_grad_norm) and the update
(spec_adamw_step, bf16 weights with f32 masters and 8-bit states).

The target is a fixed random head over token embeddings, so its next-token law
depends on the last token; the draft head starts from other weights and has to
find it.

    python examples/online_draft_head.py [--rounds 200]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_rejection_gb300 as sv  # noqa: E402

DEV = "cuda"
BF16, I32 = torch.bfloat16, torch.int32


class DraftHead:
    """logits = (h + silu(h W1^T + b1)) Wv^T, with its AdamW states."""

    def __init__(self, hidden, vocab, g):
        def rand(*shape, scale):
            return (scale * torch.randn(*shape, generator=g, device=DEV)).to(BF16)

        self.w1, self.b1 = rand(hidden, hidden, scale=hidden ** -0.5), rand(hidden, scale=0.01)
        self.wv = rand(vocab, hidden, scale=hidden ** -0.5)
        self.params = [self.w1, self.b1, self.wv]
        self.grads = [torch.zeros_like(p) for p in self.params]
        blocks = [-(-p.numel() // sv.SPEC_ADAMW_BLOCK) for p in self.params]
        codes = [[torch.zeros(p.numel(), dtype=torch.float8_e4m3fn, device=DEV) for p in self.params]
                 for _ in range(2)]
        scales = [[torch.zeros(n, device=DEV) for n in blocks] for _ in range(2)]
        self.table = sv.spec_adamw_table(self.params, self.grads, *codes, exp_avg_scale=scales[0],
                                         exp_avg_sq_scale=scales[1],
                                         master=[p.float() for p in self.params])
        self.steps = 0
        self.wv4, _ = sv.spec_head4_quantize(self.wv, group=64)

    def draft(self, h):
        """The logits from the 4-bit weights, for at most SPEC_HEAD4_MAX_ROWS rows."""
        y, _, _ = sv.spec_head_forward(h, self.w1, self.b1, residual=h, act=sv.SPEC_ACT_SILU)
        return sv.spec_head4_forward(y, self.wv4)[0]

    def forward(self, h):
        y, pre, _ = sv.spec_head_forward(h, self.w1, self.b1, residual=h, act=sv.SPEC_ACT_SILU, want_pre=True)
        logits, _, _ = sv.spec_head_forward(y, self.wv)
        return logits, (h, y, pre)

    def step(self, saved, dlogits, lr):
        h, y, pre = saved
        g1, gb, gv = self.grads
        dy, _, _, _ = sv.spec_head_backward(dlogits, y, self.wv, out=(torch.empty_like(y), gv, None))
        _, _, db, _ = sv.spec_head_backward(dy, h, self.w1, pre, act=sv.SPEC_ACT_SILU,
                                            out=(None, g1, torch.empty(gb.numel(), device=DEV)))
        gb.copy_(db)
        self.steps += 1
        norm, _ = sv.spec_grad_norm(self.table, max_norm=1.0)
        ws = sv.spec_adamw_step(self.table, self.steps, lr=lr, weight_decay=0.0, grad_scale=norm[1:])
        sv.spec_head4_quantize(self.wv, group=64, out=self.wv4)
        return ws


def run(rounds=200, B=64, K=4, vocab=2048, hidden=256, lr=2e-3, seed=1, report=print):
    """Returns the mean accepted drafts of the first and of the last tenth of
    the rounds, and the losses."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    embed = torch.randn(vocab, hidden, generator=g, device=DEV).to(BF16)
    target_w = (6.0 * hidden ** -0.5 * torch.randn(vocab, hidden, generator=g, device=DEV)).to(BF16)
    head = DraftHead(hidden, vocab, g)
    temperature = torch.full((B,), 0.8, device=DEV)
    cu_draft = torch.arange(0, B * K + 1, K, dtype=I32, device=DEV)
    cu_target = torch.arange(0, B * (K + 1) + 1, K + 1, dtype=I32, device=DEV)
    cu_one = torch.arange(B + 1, dtype=I32, device=DEV)
    # the rules: every request forbids a run of tokens and penalises repetition
    word = torch.arange((vocab + 31) // 32, device=DEV)
    mask = torch.where((word[None] + torch.arange(B, device=DEV)[:, None]) % 16 == 0, 0, -1).to(I32)
    requests = torch.arange(B, dtype=I32, device=DEV)
    rules = dict(repetition=torch.full((B,), 1.05, device=DEV), presence=torch.full((B,), 0.1, device=DEV),
                 mask=mask)
    # and has a law of its own
    law = dict(temperature=temperature, top_k=torch.where(requests % 2 == 0, 0, 200).to(I32),
               top_p=torch.where(requests % 3 == 0, 1.0, 0.98), min_p=torch.where(requests % 4 == 0, 1e-4, 0.0))
    last = torch.randint(0, vocab, (B,), generator=g, device=DEV)
    history = [[int(t)] for t in last]
    accepted_mean, losses = [], []
    for n in range(rounds):
        seen = torch.tensor([t for h in history for t in h[-32:]], dtype=I32, device=DEV)
        cu_seen = torch.tensor([0] + [min(len(h), 32) for h in history], device=DEV).cumsum(0).to(I32)
        context = dict(history=seen, cu_history=cu_seen)
        # draft K tokens, each from the rules' view of the head's logits
        tokens = torch.empty(B, K, dtype=I32, device=DEV)
        hidden_rows = [embed[last]]
        draft_rows = []
        for i in range(K):
            raw = head.draft(hidden_rows[-1])
            # the row's context: the history, then the drafts so far, which
            # lie between it and the row as in a batch of i + 1 rows
            so_far = tokens[:, :i].contiguous()
            row, _ = sv.spec_process_logits(
                raw, cu_one, max_rows=1, mask_rows=requests,
                history=torch.cat([torch.cat([seen[a:b], so_far[r]]) for r, (a, b) in enumerate(
                    zip(cu_seen[:-1].tolist(), cu_seen[1:].tolist()))]) if i else seen,
                cu_history=(cu_seen + i * cu_one).to(I32), **rules)
            u = torch.rand(B, generator=g, device=DEV)
            drawn, _, _, row, ws = sv.spec_sample(row, u, want_filtered=True, **law)
            assert sv.spec_get_status(ws) == sv.SPEC_OK
            draft_rows.append(row)
            tokens[:, i] = drawn
            hidden_rows.append(embed[tokens[:, i].long()])
        states = torch.stack(hidden_rows, 1)                       # [B, K + 1, hidden]
        target_raw, _, _ = sv.spec_head_forward(states.reshape(-1, hidden), target_w)
        flat = tokens.reshape(-1)
        target, ws = sv.spec_process_logits(target_raw, cu_target, max_rows=K + 1, tokens=flat,
                                            cu_tokens=cu_draft, **context,
                                            mask_rows=requests.repeat_interleave(K + 1), **rules)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        target = sv.spec_sample(target, None, cu_target, want_filtered=True, **law)[3]
        draft = torch.stack(draft_rows, 1).reshape(B * K, vocab)
        out, accepted, _, ws = sv.spec_verify_linear(target, draft, flat, cu_draft, temperature, seed + n, max_k=K)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        for h, row, a in zip(history, out.tolist(), accepted.tolist()):
            h += row[:a + 1]
        last = torch.tensor([h[-1] for h in history], device=DEV)
        accepted_mean.append(float(accepted.float().mean()))
        # one step on the positions that count: up to the first rejection
        pos = torch.arange(K, device=DEV)[None]
        used = (pos <= accepted[:, None]).float()
        logits, saved = head.forward(states[:, :K].reshape(-1, hidden))
        loss, grad, ws = sv.spec_distill_loss(target_raw, logits, cu_draft, temperature,
                                              (used / used.sum()).reshape(-1))
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        losses.append(float(loss.sum()))
        ws = head.step(saved, grad, lr)
        assert sv.spec_get_status(ws) == sv.SPEC_OK
        if n % max(1, rounds // 10) == 0:
            report(f"round {n:4d}: accepted {accepted_mean[-1]:.2f} of {K}, KL {losses[-1]:.3f}")
    tenth = max(1, rounds // 10)
    return sum(accepted_mean[:tenth]) / tenth, sum(accepted_mean[-tenth:]) / tenth, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rounds", type=int, default=200)
    first, final, _ = run(ap.parse_args().rounds)
    print(f"accepted drafts per round: {first:.2f} at the start, {final:.2f} at the end")
