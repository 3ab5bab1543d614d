"""distill_loss: what autograd may and may not ask of it (a library that does nothing, no GPU)."""
import pytest

torch = pytest.importorskip("torch")

B, R, V, K = 2, 3, 16, 4


class Library:
    """Every entry point, doing nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def sd(monkeypatch):
    from speculative_decoding_verification_64_gb300 import binding
    monkeypatch.setattr(binding, "load_library", Library)
    monkeypatch.setattr(binding, "_here", lambda *args: 0)
    return binding


def inputs():
    return dict(logits=torch.zeros(B, R, V), ids=torch.zeros(B, R, K, dtype=torch.int32),
                teacher=torch.zeros(B, R, K), lse=torch.zeros(B, R), weight=torch.ones(B, R))


@pytest.mark.parametrize("name", ["teacher", "lse"])
@pytest.mark.parametrize("learn", [True, False])
def test_the_teacher_has_no_gradient(sd, name, learn):
    v = inputs()
    v["logits"].requires_grad_(learn)
    v[name].requires_grad_(True)
    with pytest.raises(ValueError, match=f"{name}.detach"):
        sd.distill_loss(**v)
    with torch.no_grad():
        assert not sd.distill_loss(**v).requires_grad
    v[name] = v[name].detach()
    assert sd.distill_loss(**v).requires_grad == learn
