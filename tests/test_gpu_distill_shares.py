"""specdec_distill on records whose shares add up to more than 1 (a log-sum-exp of another
temperature, or of other logits): the gradient is that of the loss, shares beyond the sums are refused."""
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [500, 70000])
def test_shares_beyond_the_sums_are_refused(sd, V, dtype):
    """A share of more than 2^12: SPECDEC_ROW_NONFINITE, up to it the loss and the gradient."""
    x = normal(23, 1, 5, V)
    ids = np.broadcast_to(np.array([V - 1, 2], dtype=np.int32), (1, 5, 2)).copy()
    z = np.broadcast_to(np.array([0.0, -1.0], dtype=np.float32), (1, 5, 2)).copy()
    lse = np.array([[-8.31, -8.33, -50.0, -1e3, -1e30]], dtype=np.float32)  # e^8.318 = 2^12
    r = sd.distill(on_gpu(x, dtype), cuda(ids), cuda(z), cuda(lse))
    assert r.row_status[0].tolist() == [0] + [sd.ROW_NONFINITE] * 4
    assert r.loss[0, 1:].isnan().all() and r.grad[0, 1:].isnan().all()
    check(sd, x[:, :1], ids[:, :1].copy(), z[:, :1].copy(), lse[:, :1].copy(), dtype=dtype)
    # an absent entry's, and one of no probability, are not looked at
    ids[0, :, 0], z[0, :, 1] = -1, -np.inf
    r = sd.distill(on_gpu(x, dtype), cuda(ids), cuda(z), cuda(lse))
    assert (r.row_status == 0).all()
