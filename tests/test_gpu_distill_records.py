"""specdec_distill on records whose shares do not add up to 1: what a float32 log-sum-exp's rounding
leaves over of a record that names every token the draft has, and shares of more than 1."""
import numpy as np
import pytest

import draft_oracle as ref
from test_gpu_distill import UNSURE, cuda
from test_gpu_sample import on_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def whole(z, T):
    """Log-sum-exps of all of z [B, R, K] at T, in float32."""
    z = z.astype(np.float64) / T
    top = z.max(-1)
    return (top + np.log(np.exp(z - top[..., None]).sum(-1))).astype(np.float32)


def check(sd, x, ids, z, lse, T=1.0, dtype="f32", gradient=True):
    """All rows against the float64 form; returns the result."""
    t = on_gpu(x, dtype)
    got = sd.distill(t, cuda(ids), cuda(z), cuda(lse), None, T)
    alone = sd.distill(t, cuda(ids), cuda(z), cuda(lse), None, T, grad=False)
    assert torch.equal(alone.loss, got.loss) and (got.row_status == 0).all()
    T = float(np.float32(T))
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for b in range(x.shape[0]):
        for r in range(x.shape[1]):
            y, at, w = t[b, r].double().cpu().numpy(), ids[b, r], float(lse[b, r])
            with np.errstate(divide="ignore", invalid="ignore"):
                loss, g = ref.distill(y, at, z[b, r], lse[b, r], T)
            zt, top = z[b, r].astype(np.float64) / T, y.max() / T
            p = np.exp(zt - w)
            s = np.exp(y / T - top)
            ln_s = np.log(s.sum())
            s /= s.sum()
            mass, of = p.sum(), s.sum() - s[at].sum()
            left = max(0.0, 1.0 - mass)
            # The shares are good to 2^-22; they count times their entry's difference and, all
            # together, times what is subtracted from it.  ln S is off by UNSURE.  Shares of 2 and more
            # in all are summed up in float32: the parts' sizes times 2^-22.  r is off by as much as the
            # shares, which counts times its own logarithm and that of what it stands against.
            tol = 2.0 ** -21 * float((p * np.abs(zt - y[at] / T)).sum() + mass * abs(top + ln_s - w))
            tol += mass * (UNSURE + 2.0 ** -22 * (abs(top) + abs(w)))
            if left > 0 and of > 2.0 ** -100:
                tol += 2.0 ** -21 * (abs(np.log(left / of)) + 1.0) + left * UNSURE
            if np.isinf(loss):
                assert float(got.loss[b, r]) == loss
                continue
            assert abs(float(got.loss[b, r]) - loss) <= tol + 2.0 ** -23 * abs(loss), (b, r, loss, got.loss[b, r])
            if not gradient:
                continue
            # s_v, times the shares' sum, is off by UNSURE and 2^-22; the share by 2^-22 of itself
            off = max(1.0, mass) * s * (UNSURE + 2.0 ** -22)
            off[at] += 2.0 ** -22 * p
            if left > 0 and of > 2.0 ** -100:
                other = np.ones(len(y), dtype=bool)
                other[at] = False
                off[other] += s[other] / of * (2.0 ** -21 + 2 * UNSURE * left)
            d = np.abs(got.grad[b, r].double().cpu().numpy() - g)
            tol = step * np.abs(g) + (1 + step) * 1.01 / T * off + 2.0 ** -110
            assert (d <= tol).all(), (b, r, np.max(d / tol))
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("offset", [0.0, 40.0, 100.0, -100.0, 300.0, 5000.0])
def test_records_of_all_that_is_left(sd, offset, T, dtype):
    """A record of every token that the draft has left, its log-sum-exp rounded to float32: up to
    2^-24 |lse| of the mass is over, and there is no token for it."""
    rng = np.random.default_rng(int(abs(offset)) + 1)
    for V, K in ((200, 10), (64, 64), (1000, 1000)):
        x = np.full((1, 32, V), -np.inf)
        ids = np.stack([rng.permutation(V)[:K] for _ in range(32)])[None].astype(np.int32)
        y = rng.standard_normal((1, 32, K)) * 2 + offset
        np.put_along_axis(x, ids.astype(np.int64), y, -1)
        z = (y + rng.standard_normal(y.shape)).astype(np.float32)
        lse = whole(z, float(np.float32(T)))
        r = check(sd, x, ids, z, lse, T, dtype)
        assert torch.isfinite(r.loss).all() and torch.isfinite(r.grad).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_records_of_our_own(sd, dtype):
    """The log-sum-exps of specdec_top_logits, of rows under one mask."""
    rng = np.random.default_rng(3)
    for V, K, offset in ((3000, 50, 60.0), (1024, 1024, 200.0), (40000, 1000, 90.0)):
        x = np.full((1, 40, V), -np.inf)
        at = np.sort(rng.permutation(V)[:K])
        x[:, :, at] = rng.standard_normal((1, 40, K)) * 2 + offset
        rec = sd.top_logits(on_gpu(x + rng.standard_normal(x.shape), "f32"), K)
        ids, z, lse = (a.cpu().numpy() for a in (rec.ids, rec.values, rec.lse))
        assert all(set(i.tolist()) == set(at.tolist()) for i in ids[0])
        r = check(sd, x, ids, z, lse, dtype=dtype)
        assert torch.isfinite(r.loss).all()


def test_a_rest_that_float32_does_not_hold(sd):
    """Tokens outside the record of less than 2^-126 of the mass count as none, in whichever CTA they
    stand and whatever else stands there."""
    rng = np.random.default_rng(5)
    for V, last in ((100, 99), (60000, 59990)):
        ids = np.broadcast_to(np.array([3, 4, 5, 6, 7, last - 1], dtype=np.int32), (1, 60, 6)).copy()
        x = np.full((1, 60, V), -np.inf)
        x[:, :, 3:8] = rng.standard_normal((1, 60, 5)) + 100.0
        x[:, :, last - 1] = 100.0 - np.linspace(70.0, 90.0, 60)
        x[:, :, last] = 100.0 - np.linspace(91.0, 112.0, 60)
        z = np.take_along_axis(x, ids.astype(np.int64), -1).astype(np.float32)
        r = check(sd, x, ids, z, whole(z, 1.0))
        assert torch.isfinite(r.loss).all() and torch.isfinite(r.grad).all()


def test_a_rest_that_the_draft_rules_out(sd):
    """What the teacher gives to tokens that the draft has not is infinitely far, where it is more
    than rounding."""
    x = np.full((1, 3, 50), -np.inf)
    x[:, :, :4] = 0.5
    ids = np.broadcast_to(np.arange(4, dtype=np.int32), (1, 3, 4)).copy()
    z = np.zeros((1, 3, 4), dtype=np.float32)
    lse = whole(z, 1.0) + np.array([[1e-6, 1e-4, 1.0]], dtype=np.float32)
    r = check(sd, x, ids, z, lse, gradient=False)
    assert torch.isfinite(r.loss[0, 0]) and torch.isinf(r.loss[0, 1:]).all()
    assert torch.isfinite(r.grad).all()
