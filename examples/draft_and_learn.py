"""A draft that learns from what verification leaves of its target.

Two small next-token models of random weights: the target (bfloat16, fixed) and the draft
(float32 weights, trained).  Every round the draft proposes a chain of tokens, each drawn
under the request's filters with the distribution it came from kept as q (specdec_sample);
the target scores the chain, its rows go under the same filters (specdec_sample with
SPECDEC_SAMPLE_LOGITS) and through specdec_verify_linear, so that the emitted tokens follow
the filtered target; its unfiltered rows are kept as their largest logits and log-sum-exp
(specdec_top_logits), and the draft takes a gradient step towards them (specdec_distill).

    python examples/draft_and_learn.py [--rounds 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_64_gb300 import binding as sd  # noqa: E402


class Bigram:
    """Logits of the next token from the last one."""

    def __init__(self, V, hidden, seed, scale, dtype, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.embed = torch.randn(V, hidden, generator=g, device=device).to(dtype)
        self.head = (torch.randn(hidden, V, generator=g, device=device) * scale * hidden ** -0.5).to(dtype)

    def __call__(self, tokens):
        return self.embed[tokens] @ self.head


def propose(draft, last, gamma, temperature, uniforms, filters):
    """A drafted chain int32 [B, gamma] after tokens `last` [B] and its q [B, gamma, V]."""
    B, V = last.shape[0], draft.head.shape[1]
    q = torch.empty((B, gamma, V), dtype=torch.bfloat16, device=last.device)
    tokens = torch.empty((B, gamma), dtype=torch.int32, device=last.device)
    kept = torch.empty((B, 1), dtype=torch.int32, device=last.device)
    status = torch.empty_like(kept)
    with torch.no_grad():
        for i in range(gamma):
            x = draft(last.long())[:, None].to(torch.bfloat16)
            step = sd.SampleOut(torch.empty((B, 1, 1), dtype=torch.int32, device=last.device),
                                q[:, i:i + 1], kept, status)
            sd.sample(x, temperature, uniforms[:, i:i + 1, None].contiguous(), out=step, **filters)
            last = tokens[:, i] = step.tokens[:, 0, 0]
    return tokens, q


def run(rounds=20, B=16, V=500, gamma=4, k=32, lr=2.0, seed=0, trace=None):
    """Returns the mean number of accepted tokens of every round."""
    device = "cuda"
    target = Bigram(V, 64, seed, 3.0, torch.bfloat16, device)
    draft = Bigram(V, 64, seed + 1, 0.5, torch.float32, device)
    weights = [draft.embed.requires_grad_(True), draft.head.requires_grad_(True)]
    g = torch.Generator(device=device)
    g.manual_seed(seed + 2)
    temperature = torch.full((B,), 0.8, device=device)
    filters = dict(top_k=torch.full((B,), 50, dtype=torch.int32, device=device),
                   top_p=torch.full((B,), 0.95, device=device))
    last = torch.randint(0, V, (B,), generator=g, device=device).int()
    accepted = []
    for _ in range(rounds):
        u = torch.rand((B, 2 * gamma + 1), generator=g, device=device).clamp(1e-6, 1 - 1e-6)
        tokens, q = propose(draft, last, gamma, temperature, u[:, gamma + 1:], filters)
        path = torch.cat((last[:, None], tokens), 1).long()
        logits = target(path)                                             # [B, gamma + 1, V]
        rows = sd.filter_logits(logits, temperature, **filters).rows
        r = sd.verify_linear(rows, q, tokens, temperature, u[:, :gamma + 1].contiguous())
        # positions that the path reached teach; those behind the first rejection do not
        record = sd.top_logits(logits, k)
        reached = torch.arange(gamma + 1, device=device) <= r.n_accepted[:, None]
        weight = reached.float() / reached.sum()
        loss = sd.distill_loss(draft(path), record.ids, record.values, record.lse, weight).sum()
        loss.backward()
        if trace is not None:
            trace.append(dict(path=path, logits=logits, rows=rows, q=q, out=r, record=record, weight=weight,
                              loss=loss.detach(), grads=[w.grad.clone() for w in weights],
                              weights=[w.detach().clone() for w in weights]))
        with torch.no_grad():
            for w in weights:
                w -= lr * w.grad
                w.grad = None
        accepted.append(float(r.n_accepted.float().mean()))
        last = r.final_token
    return accepted


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rounds", type=int, default=20)
    a = ap.parse_args()
    for i, n in enumerate(run(a.rounds)):
        print(f"round {i}: {n:.2f} drafted tokens accepted")


if __name__ == "__main__":
    main()
