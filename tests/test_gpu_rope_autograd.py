"""The gradient of rope through autograd: what the explicit call with `backward` gives, and the
formula's by differences.  The map is linear, so a difference over a step of 1 carries rounding only:
128 products of float32 of size |x| |dy| <= 25, 128 * 25 * 2^-22 < 8e-4 at most."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def case(dtype, seed=1, B=2, N=3, Hq=4, Hk=2, D=64):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(dtype)
    return make(B, N, Hq + Hk, D), make(B, N, Hq, D), make(B, N, Hk, D)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_gradients_of_slices_of_a_projection(sd, dtype, interleaved, backward):
    x, dq, dk = case(dtype)
    how = dict(base=torch.tensor([5, 70000], dtype=torch.int32).cuda(), interleaved=interleaved,
               magnitude=1.25)
    freq = sd.rope_frequencies(48)
    x.requires_grad_(True)
    q, k = sd.rope(x[:, :, :4], x[:, :, 4:], freq, backward=backward, **how)
    assert q.requires_grad and k.requires_grad
    with torch.no_grad():
        plain = sd.rope(x[:, :, :4], x[:, :, 4:], freq, backward=backward, **how)
        assert not plain[0].requires_grad
        assert torch.equal(plain[0], q) and torch.equal(plain[1], k)
    gx, = torch.autograd.grad((q, k), x, (dq, dk))
    want = sd.rope(dq, dk, freq, backward=not backward, **how)
    assert torch.equal(gx, torch.cat(want, 2))


def test_gradients_by_differences(sd):
    x, dq, dk = case(torch.float32, seed=2)
    freq = sd.rope_frequencies(64)
    parent = torch.tensor([[-1, 0, 0], [-1, 0, 1]], dtype=torch.int32).cuda()
    run = lambda t: sd.rope(t[:, :, :4], t[:, :, 4:], freq, parent=parent, magnitude=0.75)
    x.requires_grad_(True)
    loss = lambda t: sum((a.double() * b.double()).sum() for a, b in zip(run(t), (dq, dk)))
    gx, = torch.autograd.grad(loss(x), x)
    rng = np.random.default_rng(3)
    with torch.no_grad():
        for _ in range(20):
            e = torch.zeros_like(x)
            i = tuple(int(rng.integers(0, n)) for n in e.shape)
            e[i] = 1.0
            assert abs(float((loss(x + e) - loss(x - e)) / 2) - float(gx[i])) <= 8e-4


def test_one_of_the_two_another_stream_and_twice(sd):
    x, dq, dk = case(torch.float32, seed=4)
    freq = sd.rope_frequencies(64)
    q, k = x[:, :, :4].contiguous(), x[:, :, 4:].contiguous()
    want_q, want_k = sd.rope(dq, dk, freq, backward=True)
    k.requires_grad_(True)
    a, b = sd.rope(q, k, freq)
    assert torch.equal(torch.autograd.grad(b, k, dk)[0], want_k)
    k.requires_grad_(False)
    q.requires_grad_(True)
    a, none = sd.rope(q, None, freq)
    assert none is None and torch.equal(torch.autograd.grad(a, q, dq)[0], want_q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = sd.rope(q, k, freq, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(torch.autograd.grad((a, b), q, (dq, dk))[0], want_q)
    # the gradient's own gradient
    dq.requires_grad_(True)
    a, _ = sd.rope(q, None, freq)
    g, = torch.autograd.grad(a, q, dq, create_graph=True)
    assert torch.equal(torch.autograd.grad(g, dq, q.detach())[0], sd.rope(q.detach(), None, freq)[0])


def test_outputs_of_the_caller_are_refused(sd):
    x, _, _ = case(torch.float32)
    x = x[:, :, :4].contiguous().requires_grad_(True)
    freq = sd.rope_frequencies(64)
    with pytest.raises(ValueError):
        sd.rope(x, None, freq, q_out=torch.empty_like(x))
    with torch.no_grad():
        sd.rope(x, None, freq, q_out=torch.empty_like(x))
