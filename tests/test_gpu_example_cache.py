"""The cached verify example: its lengths follow the accepted counts, and a step's logits are those
of a pass over the whole text without a cache, up to what 8 bits cost."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from speculative_decoding_verification_64_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location(
        "verify_with_cache", os.path.join(ROOT, "examples", "verify_with_cache.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_lengths_and_tokens(example):
    trace = []
    emitted = example.run(steps=3, B=3, prompt=37, trace=trace)
    held = torch.full((3,), 36)
    for logits, r, lengths in trace:
        assert (r.row_status == 0).all() and torch.isfinite(logits.float()).all()
        held = held + r.n_accepted.cpu() + 1
        for n in lengths:
            assert torch.equal(n.cpu().long(), held)
    assert [len(e) for e in emitted] == [int(held[b]) - 36 for b in range(3)]
    assert example.run(steps=3, B=3, prompt=37) == emitted


def test_cached_pass_agrees_with_one_without_a_cache(example):
    """Logits of the last 9 tokens of a text, over a cache of the first 60 and in one chain of 69.
    A code is off by 2^-4 of its value at most, at random: the logits of the two passes differ by
    a few per cent of their size; 0.1 is allowed, where a misplaced token or block gives 1."""
    B, V = 2, 1000
    model = example.Decoder(V=V)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    tokens = torch.randint(0, V, (B, 69), generator=g, device="cuda")
    whole, _ = model.forward(tokens, example.make_caches(model, B, 80))
    caches = example.make_caches(model, B, 80)
    for a, b in ((0, 33), (33, 34), (34, 60)):
        _, new = model.forward(tokens[:, a:b], caches)
        example.append(caches, new)
    last, _ = model.forward(tokens[:, 60:], caches)
    want = whole[:, 60:].float()
    assert (last.float() - want).norm() <= 0.1 * want.norm()
