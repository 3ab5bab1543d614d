"""The draft side's calls on a stream other than the current one make their outputs and workspaces
on that stream, so that nobody else is given that memory while their kernels run."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

B, R, V, K = 2, 3, 16, 4


class Library:
    """Every entry point, doing nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


def calls(sd):
    x, T, u = torch.zeros(B, R, V), torch.ones(B), torch.zeros(B, R, 1)
    ids, z = torch.zeros(B, R, K, dtype=torch.int32), torch.zeros(B, R, K)
    y = x.clone().requires_grad_(True)
    return {
        "sample": lambda s: sd.sample(x, T, u, stream=s),
        "filter_logits": lambda s: sd.filter_logits(x, T, stream=s),
        "top_logits": lambda s: sd.top_logits(x, K, stream=s),
        "distill": lambda s: sd.distill(x, ids, z, stream=s),
        "distill_loss": lambda s: sd.distill_loss(x, ids, z, stream=s),
        "distill_loss, with a gradient": lambda s: sd.distill_loss(y, ids, z, stream=s),
    }


NAMES = sorted(calls(types.SimpleNamespace()))


@pytest.mark.parametrize("name", NAMES)
def test_a_call_makes_its_tensors_on_its_stream(monkeypatch, name):
    from speculative_decoding_verification_64_gb300 import binding as sd
    current, made, empty = [], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    call = calls(sd)[name]
    monkeypatch.setattr(sd, "load_library", Library)
    monkeypatch.setattr(sd, "_here", lambda *args: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)

    def make(*args, **kw):
        made.append(current[-1] if current else None)
        return empty(*args, **kw)

    monkeypatch.setattr(torch, "empty", make)
    s = types.SimpleNamespace(cuda_stream=0)
    call(s)
    assert made and all(on is s for on in made)
    assert not current
