"""specdec_distill on records whose shares add up to more than 1 (a log-sum-exp of another
temperature, or of other logits): the gradient is that of the loss."""
import numpy as np
import pytest

import draft_oracle as ref
from test_gpu_distill import cuda
from test_gpu_distill_records import check, whole
from test_gpu_sample import floats, normal, on_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def record(seed, B, R, V, K, T, mass):
    """Records of all masses in `mass` [R], in turn."""
    rng = np.random.default_rng(seed)
    x = normal(seed, B, R, V)
    ids = np.stack([[rng.permutation(V)[:K] for _ in range(R)] for _ in range(B)]).astype(np.int32)
    z = (rng.standard_normal((B, R, K)) * 2).astype(np.float32)
    return x, ids, z, (whole(z, T) - np.log(np.array(mass))).astype(np.float32)


MASS = [0.3, 1.0, 1.5, 2.27, 40.0, 3000.0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 1.3])
@pytest.mark.parametrize("V,K", [(9, 3), (1000, 64), (70000, 300), (64, 64)])
def test_gradient_of_shares_of_any_sum(sd, V, K, T, dtype):
    x, ids, z, lse = record(V, 2, len(MASS), V, K, float(np.float32(T)), MASS)
    if V == K:
        x, ids, z, lse = (a[:, 1:] for a in (x, ids, z, lse))  # (0.3 has nowhere to go)
        ids, z, lse = (np.ascontiguousarray(a) for a in (ids, z, lse))
    check(sd, x, ids, z, lse, T, dtype)


def test_by_differences(sd):
    """Of the float32 loss, steps of 2^-5: they leave 2^-10 / 6 of the third derivative, below the shares'
    sum, and twice the losses' own error over 2^-4: 4e-5 of the sum and 2^-24 of a loss below 100."""
    x, ids, z, lse = record(21, 1, 3, 40, 7, 1.0, [1.5, 2.27, 9.0])
    t, ids, z, lse = on_gpu(x, "f32"), cuda(ids), cuda(z), cuda(lse)
    g = sd.distill(t, ids, z, lse).grad
    for v in range(0, 40, 3):
        e = torch.zeros_like(t)
        e[:, :, v] = 2.0 ** -5
        up, down = (sd.distill(y, ids, z, lse, grad=False).loss for y in (t + e, t - e))
        for r, mass in enumerate((1.5, 2.27, 9.0)):
            tol = mass * (2.0 ** -10 / 6 + 32 * 4e-5) + 32 * 100 * 2.0 ** -24
            assert abs(float(up[0, r] - down[0, r]) * 16 - float(g[0, r, v])) <= tol


def test_under_autograd(sd):
    x, ids, z, lse = record(22, 2, 3, 500, 20, 1.0, [1.5, 2.27, 9.0])
    ids, z, lse = cuda(ids), cuda(z), cuda(lse)
    t = on_gpu(x, "f32").requires_grad_(True)
    d = floats([[1.0, 3.0, 0.0], [0.5, 1.0, -2.0]])
    g, = torch.autograd.grad(sd.distill_loss(t, ids, z, lse), t, d)
    assert torch.equal(g, sd.distill(t.detach(), ids, z, lse, d).grad)
