"""distill_loss under autograd: the gradients of the logits and of the weights, of one or of both."""
import pytest

import draft_oracle as ref
from test_gpu_distill import UNSURE, cuda, teacher
from test_gpu_sample import floats, normal, on_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

W = [[0.5, 0.0, 1.0], [2.0, -0.25, 0.0]]


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def case(seed=31, V=700, K=20):
    x = normal(seed, 2, 3, V)
    return x, teacher(seed, x, K, 1.0, True)


@pytest.mark.parametrize("of_logits", [True, False])
def test_gradient_of_the_weights(sd, of_logits):
    """d (w loss) / d w is the loss, at a weight of 0 too, whatever else requires a gradient."""
    x, record = case()
    ids, z, lse = (cuda(a) for a in record)
    t, w = on_gpu(x, "f32"), floats(W)
    d = floats([[1.0, 3.0, 0.0], [0.5, 1.0, -2.0]])
    plain = sd.distill(t, ids, z, lse)
    want = sd.distill_loss(t, ids, z, lse, w)
    t.requires_grad_(of_logits)
    w.requires_grad_(True)
    loss = sd.distill_loss(t, ids, z, lse, w)
    assert torch.equal(loss, want)
    both = (t, w) if of_logits else (w,)
    first = torch.autograd.grad(loss, both, d, retain_graph=True)
    again = torch.autograd.grad(loss, both, d)
    for g in (first, again):
        assert torch.equal(g[-1], d * plain.loss)
        if of_logits:
            assert torch.equal(g[0], sd.distill(t.detach(), ids, z, lse, w.detach() * d).grad)
    # and that loss is the divergence
    for b in range(2):
        for r in range(3):
            loss = ref.distill(x[b, r].astype("float32").astype("float64"), record[0][b, r], record[1][b, r],
                               record[2][b, r])[0]
            assert abs(float(plain.loss[b, r]) - loss) <= 2 * UNSURE + 2.0 ** -21 * 20 + 2.0 ** -23 * abs(loss)


def test_one_of_two_gradients(sd):
    """Asked for by itself, each is what it is beside the other."""
    x, record = case(32)
    ids, z, lse = (cuda(a) for a in record)
    t, w = on_gpu(x, "bf16").requires_grad_(True), floats(W).requires_grad_(True)
    plain = sd.distill(t.detach(), ids, z, lse, w.detach())
    alone = sd.distill(t.detach(), ids, z, lse, grad=False).loss
    for order in ((t, w), (w, t)):
        loss = sd.distill_loss(t, ids, z, lse, w).sum()
        for leaf in order:
            g, = torch.autograd.grad(loss, leaf, retain_graph=True)
            assert torch.equal(g, plain.grad if leaf is t else alone)


def test_rows_of_weight_0_that_hold_anything(sd):
    """Their loss and the logits' gradient are 0 whatever they hold; the weight's gradient is their
    divergence: NaN for a malformed row, 0 for one without entries."""
    x, (ids, z, lse) = case(33)
    x[0, 1, 5] = float("nan")
    ids[1, 2] = -1
    ids, z, lse = cuda(ids), cuda(z), cuda(lse)
    t, w = on_gpu(x, "f32").requires_grad_(True), floats(W).requires_grad_(True)
    loss = sd.distill_loss(t, ids, z, lse, w)
    assert torch.isfinite(loss).all()
    g, dw = torch.autograd.grad(loss.sum(), (t, w))
    assert torch.isfinite(g).all() and (g[0, 1] == 0).all() and (g[1, 2] == 0).all()
    assert dw[0, 1].isnan() and dw[1, 2] == 0
    dw[0, 1] = 0.0
    assert torch.isfinite(dw).all()


def test_learned_weights(sd):
    """Weights out of other weights, as a program has them: a row's mean, and scaled after the fact."""
    x, record = case(34)
    ids, z, lse = (cuda(a) for a in record)
    t, a = on_gpu(x, "f32").requires_grad_(True), floats(W).requires_grad_(True)
    loss = (sd.distill_loss(t, ids, z, lse, torch.softmax(a, 1)) * 0.5).mean()
    loss.backward()
    alone = sd.distill(t.detach(), ids, z, lse)
    b = floats(W).requires_grad_(True)
    (torch.softmax(b, 1) * alone.loss * 0.5).mean().backward()
    # float32 products of three, in any order
    assert (a.grad - b.grad).abs().max() <= 2.0 ** -21 * alone.loss.abs().max()
    want = sd.distill(t.detach(), ids, z, lse, torch.softmax(b.detach(), 1) * (0.5 / 6)).grad
    assert (t.grad - want).abs().max() <= 2.0 ** -21 * want.abs().max()


def test_rows_of_weight_0_under_any_gradient(sd):
    """Nothing comes of them, the first time and over a retained graph, whatever comes in."""
    x, record = case(35)
    ids, z, lse = (cuda(a) for a in record)
    t, w = on_gpu(x, "f32").requires_grad_(True), floats(W)
    loss = sd.distill_loss(t, ids, z, lse, w)
    d = floats([[1.0, float("inf"), 1.0], [1.0, 1.0, float("nan")]])
    want = sd.distill(t.detach(), ids, z, lse, w).grad
    for _ in range(3):
        g, = torch.autograd.grad(loss, t, d, retain_graph=True)
        assert torch.equal(g, want) and (g[0, 1] == 0).all() and (g[1, 2] == 0).all()


@pytest.mark.parametrize("of_weights", [False, True])
def test_offloaded_and_checkpointed(sd, of_weights):
    """Saved tensors that go to the host and back, or are made again, give the same gradients."""
    from torch.utils.checkpoint import checkpoint
    x, record = case(36)
    ids, z, lse = (cuda(a) for a in record)
    d = floats([[1.0, 3.0, 0.0], [0.5, 1.0, -2.0]])

    def leaves():
        a = on_gpu(x, "f32").requires_grad_(True)
        return (a, floats(W).requires_grad_(of_weights))

    def step(a, w):
        return sd.distill_loss(a * 1.5, ids, z, lse, w)

    def gradients(loss, of, times=2):
        of = of if of_weights else of[:1]
        return [torch.autograd.grad(loss, of, d, retain_graph=i + 1 < times) for i in range(times)]

    of = leaves()
    want = gradients(step(*of), of)
    of = leaves()
    with torch.autograd.graph.save_on_cpu(pin_memory=True):
        loss = step(*of)
    off = gradients(loss, of)
    of = leaves()
    made = gradients(checkpoint(step, *of, use_reentrant=False), of, 1)
    for got in (off, made):
        for g, v in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, v))


def test_gradients_that_are_changed_in_place(sd):
    x, record = case(37)
    ids, z, lse = (cuda(a) for a in record)
    t = on_gpu(x, "f32").requires_grad_(True)
    plain = sd.distill(t.detach(), ids, z, lse)
    loss = sd.distill_loss(t, ids, z, lse).sum()
    for _ in range(3):
        g, = torch.autograd.grad(loss, t, retain_graph=True)
        assert torch.equal(g, plain.grad)
        g.zero_()
    loss.backward(retain_graph=True)
    t.grad.mul_(0.5)
    loss.backward()
    assert torch.equal(t.grad, plain.grad * 0.5 + plain.grad)
