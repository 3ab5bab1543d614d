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


@pytest.mark.parametrize("name", ["logits", "teacher", "lse", "weight"])
@pytest.mark.parametrize("learn", [True, False])
def test_tangents_are_refused(sd, name, learn):
    import torch.autograd.forward_ad as forward_ad
    v = inputs()
    v["logits"].requires_grad_(learn)
    with forward_ad.dual_level():
        v[name] = forward_ad.make_dual(v[name], torch.ones_like(v[name]))
        with pytest.raises(NotImplementedError, match="forward mode"):
            sd.distill_loss(**v)
        v[name] = forward_ad.unpack_dual(v[name]).primal
        sd.distill_loss(**v)


def test_functional_transforms_are_refused(sd):
    v = inputs()
    x = v.pop("logits")
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: sd.distill_loss(x, **v), (x,), (torch.ones_like(x),))
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda x: sd.distill_loss(x, **v).sum())(x)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_made_for_nobody(sd, monkeypatch, mode):
    """No gradient where none is recorded, whatever requires one."""
    v = inputs()
    v["logits"].requires_grad_(True)
    v["weight"].requires_grad_(True)
    made = []
    call = sd.distill
    monkeypatch.setattr(sd, "distill", lambda *a, **kw: made.append(kw["grad"]) or call(*a, **kw))
    with mode():
        loss = sd.distill_loss(**v)
    assert made == [False] and not loss.requires_grad


def test_hooks_on_saved_tensors_have_the_gradient(sd):
    """Whatever is as large as the logits goes through them, and is gone with the graph."""
    import gc
    import weakref
    v = inputs()
    v["logits"].requires_grad_(True)
    packed, held = [], []

    def pack(t):
        packed.append(tuple(t.shape))
        t = t.detach().clone()
        held.append(weakref.ref(t))
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        loss = sd.distill_loss(**v).sum()
    assert packed.count((B, R, V)) == 2  # the logits, their gradient
    node = loss.grad_fn.next_functions[0][0]
    large = [k for k, t in vars(node).items() if torch.is_tensor(t)]
    assert not large
    g, = torch.autograd.grad(loss, v["logits"])
    assert g.shape == (B, R, V)
    del g, loss, node
    gc.collect()
    assert all(r() is None for r in held)


def test_what_becomes_of_a_gradient_is_the_callers(sd):
    """Changed in place, as clipping does, it does not stand in a retained graph's way."""
    v = inputs()
    x = v["logits"].requires_grad_(True)
    loss = sd.distill_loss(**v).sum()
    for _ in range(3):
        g, = torch.autograd.grad(loss, x, retain_graph=True)
        g.mul_(2.0)
    for _ in range(3):
        loss.backward(retain_graph=True)
        x.grad.mul_(2.0)
    with torch.no_grad():
        v["weight"].add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
