"""The draft side's calls together, as examples/draft_and_learn.py uses them: the emitted tokens are
possible under the filters, each step's gradient is the one of a float64 composition."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    from speculative_decoding_verification_64_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import draft_and_learn
    return draft_and_learn


def test_rounds(example):
    trace = []
    accepted = example.run(rounds=6, trace=trace)
    assert len(accepted) == 6 and all(0 <= a <= 4 for a in accepted)
    for t in trace:
        r, q, rows = t["out"], t["q"].float(), t["rows"]
        B, gamma, V = q.shape
        assert (r.row_status == 0).all() and (t["record"].row_status == 0).all()
        # a drafted token has probability, at most 50 tokens have, and they add up to one
        drafted = t["path"][:, 1:]
        assert (q.gather(2, drafted[..., None]) > 0).all() and ((q > 0).sum(2) <= 50).all()
        assert (q.sum(2) - 1).abs().max() <= 2.0 ** -8
        # what is emitted was kept by the filter of its row
        for b in range(B):
            for i in range(int(r.n_accepted[b]) + 1):
                assert rows[b, i, int(r.out_tokens[b, i])] > -float("inf")
        # the step's gradient in float64
        embed, head = (w.double().requires_grad_(True) for w in t["weights"])
        s = torch.log_softmax(embed[t["path"]] @ head, -1)
        ids, z, lse = t["record"].ids.long(), t["record"].values.double(), t["record"].lse.double()
        p = torch.exp(z - lse[..., None])
        left = 1 - p.sum(-1)
        rest = torch.ones_like(s).scatter(-1, ids, 0.0)
        of = (torch.exp(s) * rest).sum(-1)
        loss = (p * (z - lse[..., None] - s.gather(-1, ids))).sum(-1) + left * (torch.log(left) - torch.log(of))
        loss = (loss * t["weight"].double()).sum()
        assert abs(loss.item() - t["loss"].item()) <= 1e-4 * abs(loss.item())
        loss.backward()
        # float32 products of 64 terms before and of up to 80 rows behind the kernel: 2^-24 * (64 + 80)
        # of sizes up to a few times the result's largest, and the kernel's own 2^-16 of it
        for g, want in zip(t["grads"], (embed.grad, head.grad)):
            assert (g.double() - want).abs().max() <= 1e-4 * want.abs().max()
