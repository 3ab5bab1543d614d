"""specdec_distill against float64, its refusals, and its gradient through autograd."""
import numpy as np
import pytest

import draft_oracle as ref
from test_gpu_sample import DT, floats, normal, on_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def teacher(seed, x, K, T, lse):
    """Records of noisy copies of the rows (float32), their entries in no order."""
    rng = np.random.default_rng(seed)
    y = np.where(np.isfinite(x), x, -30.0) + rng.standard_normal(x.shape)
    ids = np.argsort(-y, axis=-1)[:, :, :K]
    ids = np.take_along_axis(ids, rng.permuted(np.broadcast_to(np.arange(K), ids.shape), axis=-1), -1)
    z = np.take_along_axis(y, ids, -1).astype(np.float32)
    top = y.max(-1)
    whole = (top / T + np.log(np.exp((y - top[..., None]) / T).sum(-1))).astype(np.float32)
    return ids.astype(np.int32), z, whole if lse else None


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


# A weight 2^y, |y| <= 64 where it counts, is off by 3 * 2^-24 |y| ln 2 (difference, c and product
# rounded), ex2 by 2^-22 and a sum of them by 64 additions: of themselves, all in all
UNSURE = 3 * 64 * 0.7 * 2.0 ** -24 + 2.0 ** -22 + 64 * 2.0 ** -24


def check(sd, x, K, T=1.0, lse=True, w=None, dtype="f32", pad=0, shift=0, rows=None, record=None):
    B, R, V = x.shape
    t = on_gpu(x, dtype, pad, shift)
    if record is None:
        record = teacher(V + K, t.double().cpu().numpy(), K, T, lse)
    ids, z, whole = record
    weights = None if w is None else floats(w).view(B, R)
    got = sd.distill(t, cuda(ids), cuda(z), cuda(whole), weights, T)
    alone = sd.distill(t, cuda(ids), cuda(z), cuda(whole), weights, T, grad=False)
    assert alone.grad is None
    T = float(np.float32(T))
    for b in range(B):
        for r in range(R):
            if rows is not None and (b, r) not in rows:
                continue
            assert alone.loss[b, r] == got.loss[b, r]
            y = t[b, r].double().cpu().numpy()
            loss, g = ref.distill(y, ids[b, r], z[b, r], None if whole is None else whole[b, r], T)
            weight = 1.0 if w is None else float(np.float32(np.reshape(w, (B, R))[b, r]))
            if weight == 0:
                loss = 0.0
            assert got.row_status[b, r] == 0
            # ln s is off by UNSURE, p by 2^-22, r by 2^-21 (its rounded lse): |ln r / s_rest| < 20
            # times that, and the shares' logarithms
            assert abs(float(got.loss[b, r]) - loss) <= 2 * UNSURE + 2.0 ** -21 * 20 + 2.0 ** -23 * abs(loss)
            if not np.isfinite(y).any():
                continue
            some = ids[b, r] >= 0
            at = ids[b, r][some]
            s = np.exp((y - y.max()) / T)
            s /= s.sum()
            off = s * UNSURE                       # of s_v / T, from which p_v is taken
            off[at] += 2.0 ** -22                  # p_v <= 1
            if whole is not None and some.any():
                other = np.ones(V, dtype=bool)
                other[at] = False
                left = max(0.0, 1 - np.exp(z[b, r][some].astype(np.float64) / T - float(whole[b, r])).sum())
                of = s[other].sum()
                if of > 0:                         # s_v r / s_rest: r off by 2^-21, s_rest by UNSURE
                    off[other] += s[other] / of * (2.0 ** -21 + 2 * UNSURE * left)
            step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
            g = g * weight
            d = np.abs(got.grad[b, r].double().cpu().numpy() - g)
            tol = step * np.abs(g) + (1 + step) * 1.01 * abs(weight) / T * off + 2.0 ** -110
            assert (d <= tol).all(), (b, r, np.max(d / tol))
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lse", [True, False])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 1), (7, 7), (64, 5), (1000, 64), (5003, 300), (2000, 1024)])
def test_sizes(sd, dtype, lse, V, K):
    check(sd, normal(V, 2, 3, V), K, T=1.5, lse=lse, w=[[1.0, 0.25, 0.0], [2.0, -1.0, 1e-3]], dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (5, 7), (8, 2)])
def test_rows_that_start_anywhere(sd, dtype, pad, shift):
    check(sd, normal(9, 2, 3, 1501), 20, dtype=dtype, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype,V,B", [("bf16", 128256, 1), ("f32", 128256, 1), ("bf16", 40001, 120),
                                       ("f32", 3001, 500), ("f32", 1 << 19, 1), ("bf16", 1 << 19, 2)])
def test_clusters_of_every_size(sd, dtype, V, B):
    x = np.random.default_rng(V).standard_normal((B, 1, V)).astype(np.float32)
    check(sd, x, 64, dtype=dtype, rows={(0, 0), (B // 2, 0), (B - 1, 0)})


@pytest.mark.parametrize("V,B", [(50001, 80), (80000, 50), (100003, 40), (115000, 34), (130002, 30), (160001, 20),
                                 (200000, 16), (240005, 13), (300000, 11)])
def test_clusters_of_other_sizes(sd, V, B):
    """3, 5, 6, 7, 8, 10, 12, 14 and 16 CTAs a float32 row."""
    x = np.random.default_rng(V).standard_normal((B, 1, V)).astype(np.float32)
    check(sd, x, 300, rows={(0, 0), (B - 1, 0)})


@pytest.mark.parametrize("T", [0.01, 0.5, 4.0, 1000.0])
@pytest.mark.parametrize("offset", [0.0, 300.0])
def test_temperatures_and_offsets(sd, T, offset):
    check(sd, normal(8, 2, 2, 2000, scale=min(2.0, 20 * T)) + offset, 30, T=T, lse=False)


def test_absent_entries_and_rows_without_any(sd):
    x = normal(10, 1, 4, 900)
    ids, z, lse = teacher(1, x, 12, 1.0, True)
    x[0, 2] = np.nan                       # not looked at: nothing to learn there
    ids[0, 0, 3:7] = -1
    z[0, 0, 3:7] = np.nan                  # not read
    ids[0, 1, 1:] = -1
    ids[0, 2], ids[0, 3] = -1, -1
    for whole in (lse, None):
        r = check(sd, x, 12, record=(ids, z, whole), rows={(0, 0), (0, 1), (0, 3)})
        assert (r.loss[0, 2:] == 0).all() and (r.grad[0, 2:] == 0).all() and (r.row_status == 0).all()


@pytest.mark.parametrize("lse", [True, False])
@pytest.mark.parametrize("T", [1.0, 0.7, 2.0])
@pytest.mark.parametrize("V,K", [(200, 200), (1000, 1000), (32000, 64), (128256, 512)])
def test_small_losses(sd, V, K, T, lse):
    # A draft next to its teacher: a loss of some 1e-5 out of terms of some units.  The entries'
    # weights are good to 2^-27, three logarithms to 2^-28, the rest of the sums to less: 2^-25
    # in all.  The shares are off by 2^-22, which counts times |ln p / s|.  The other tokens' weights
    # O are off by UNSURE of themselves; ln S goes with them by O / S, and with a log-sum-exp
    # -r ln s_rest by -r more.
    rng = np.random.default_rng(V + K)
    T32 = float(np.float32(T))
    y = 3.0 * rng.standard_normal((1, 3, V))
    x = (y + 0.01 * rng.standard_normal(y.shape)).astype(np.float32)
    ids = np.argsort(-y, axis=-1)[:, :, :K].astype(np.int32)
    z = np.take_along_axis(y, ids, -1).astype(np.float32)
    top = y.max(-1)
    whole = (top / T32 + np.log(np.exp((y - top[..., None]) / T32).sum(-1))).astype(np.float32)
    whole = whole if lse else None
    got = sd.distill(cuda(x), cuda(ids), cuda(z), cuda(whole), None, T, grad=False)
    for r in range(3):
        row = x[0, r].astype(np.float64)
        with np.errstate(divide="ignore"):
            loss, _ = ref.distill(row, ids[0, r], z[0, r], None if whole is None else whole[0, r], T32)
        if np.isinf(loss):  # (a rounded log-sum-exp leaves 2^-20 to tokens that do not exist)
            assert float(got.loss[0, r]) == loss
            continue
        s = np.exp((row - row.max()) / T32)
        s /= s.sum()
        of = 1.0 - s[ids[0, r]].sum() if K < V else 0.0
        p = np.exp(z[0, r].astype(np.float64) / T32 - (0.0 if whole is None else whole[0, r]))
        p = p if lse else p / p.sum()
        left = max(0.0, 1.0 - p.sum()) if lse else 0.0
        ratio = np.abs(np.log(p / s[ids[0, r]]))
        some = 2.0 ** -25 + 2.0 ** -22 * float((p * ratio).sum()) + abs(of - left) * UNSURE
        assert abs(float(got.loss[0, r]) - loss) <= some + 2.0 ** -23 * abs(loss)


def test_masked_tokens_and_certain_teachers(sd):
    x = normal(11, 1, 4, 700)
    x[0, :, 50:600] = -np.inf
    ids, z, lse = teacher(2, x, 10, 1.0, True)
    z[0, 1, 4:] = -np.inf                   # entries of no probability
    for whole in (lse, None):
        check(sd, x, 10, record=(ids, z, whole))
    # the entries are all that is left of the draft: nothing is asked of the rest
    x[0, :, 10:] = -np.inf
    ids = np.broadcast_to(np.arange(10, dtype=np.int32), (1, 4, 10)).copy()
    z = np.random.default_rng(3).standard_normal((1, 4, 10)).astype(np.float32)
    lse = np.log(np.exp(z.astype(np.float64)).sum(-1)).astype(np.float32)
    r = check(sd, x, 10, record=(ids, z, lse))
    assert torch.isfinite(r.loss).all()
    # a token that the teacher wants and the draft rules out
    x[0, 0, 3] = -np.inf
    r = sd.distill(on_gpu(x, "f32"), cuda(ids), cuda(z))
    assert r.loss[0, 0] == np.inf and torch.isfinite(r.grad).all() and r.row_status[0, 0] == 0


def test_bad_rows(sd):
    x = normal(12, 9, 1, 500)
    ids, z, lse = teacher(4, x, 6, 1.0, True)
    x[0, 0, 499] = np.nan
    x[1, 0, 0] = np.inf
    x[2] = -np.inf
    ids[3, 0, 2], ids[4, 0, 5] = 500, -2
    ids[5, 0, 4] = ids[5, 0, 1]
    z[6, 0, 0] = np.nan
    z[7, 0, 0] = np.inf
    lse[8, 0] = np.inf
    want = [sd.ROW_NONFINITE] * 3 + [sd.ROW_BAD_TOKEN] * 3 + [sd.ROW_NONFINITE] * 3
    for dtype in ("f32", "bf16"):
        r = sd.distill(on_gpu(x, dtype), cuda(ids), cuda(z), cuda(lse))
        assert r.row_status[:, 0].tolist() == want
        assert r.loss.isnan().all() and r.grad.isnan().all()
        # without weight none of it is looked at
        r = sd.distill(on_gpu(x, dtype), cuda(ids), cuda(z), cuda(lse), torch.zeros(9, 1).cuda())
        assert (r.row_status == 0).all() and (r.loss == 0).all() and (r.grad == 0).all()
    fine = np.tile(np.arange(6, dtype=np.int32), (2, 1, 1))
    zero = np.zeros((2, 1, 6), dtype=np.float32)
    w = torch.tensor([[float("inf")], [float("nan")]]).cuda()
    r = sd.distill(on_gpu(x[3:5], "f32"), cuda(fine), cuda(zero), None, w)
    assert (r.row_status == sd.ROW_NONFINITE).all() and r.grad.isnan().all()
    r = sd.distill(on_gpu(x[3:5], "f32"), cuda(fine), cuda(zero - np.inf))
    assert (r.row_status == sd.ROW_NONFINITE).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_over_the_logits_and_into_slices(sd, dtype):
    x = normal(13, 2, 3, 1003)
    ids, z, lse = (cuda(a) for a in teacher(5, x, 40, 1.0, True))
    t = on_gpu(x, dtype, pad=5, shift=3)
    want = sd.distill(t, ids, z, lse)
    y = on_gpu(x, dtype, pad=5, shift=3)
    whole = y._base.clone()
    r = sd.distill(y, ids, z, lse, out=sd.DistillOut(want.loss.clone(), y, want.row_status.clone()))
    assert torch.equal(y, want.grad) and torch.equal(r.loss, want.loss)
    y.copy_(t)
    assert torch.equal(y._base, whole)   # nothing beside the rows
    big = torch.full((2, 7, 1003), 3.0, dtype=DT[dtype], device="cuda")
    sd.distill(t, ids, z, lse, out=sd.DistillOut(want.loss, big[:, 1:7:2], want.row_status))
    assert torch.equal(big[:, 1:7:2], want.grad) and (big[:, ::2] == 3).all()
    with pytest.raises(sd.SpecdecError):
        buf = torch.zeros(2 * 3 * 1003 + 8, dtype=DT[dtype], device="cuda")
        a, b = buf[:-8].view(2, 3, 1003), buf[8:].view(2, 3, 1003)
        sd.distill(a, ids, z, lse, out=sd.DistillOut(want.loss, b, want.row_status))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_autograd(sd, dtype):
    x = normal(14, 2, 3, 800)
    ids, z, lse = (cuda(a) for a in teacher(6, x, 25, 1.0, True))
    w = floats([[0.5, 0.0, 1.0], [2.0, 0.25, 1.5]])
    t = on_gpu(x, dtype).requires_grad_(True)
    plain = sd.distill(t.detach(), ids, z, lse, w)
    loss = sd.distill_loss(t, ids, z, lse, w)
    assert torch.equal(loss, plain.loss * w)
    with torch.no_grad():
        assert torch.equal(sd.distill_loss(t, ids, z, lse, w), loss)
    assert torch.equal(sd.distill_loss(t.detach(), ids, z, lse, w), loss)
    g, = torch.autograd.grad(loss.sum(), t, retain_graph=True)
    assert torch.equal(g, plain.grad)
    # again over the retained graph, and with other incoming gradients
    h, = torch.autograd.grad(loss.sum(), t, retain_graph=True)
    assert torch.equal(h, plain.grad) and torch.equal(g, plain.grad)
    d = floats([[1.0, 3.0, 0.0], [0.5, 1.0, -2.0]])
    scaled = sd.distill(t.detach(), ids, z, lse, w * d).grad
    g, = torch.autograd.grad(loss, t, d)
    assert torch.equal(g, scaled)
    g, = torch.autograd.grad(sd.distill_loss(t, ids, z, lse, w), t, d)   # in place of the forward's
    assert torch.equal(g, scaled)
    g, = torch.autograd.grad(sd.distill_loss(t, ids, z, lse).sum() * 0.5, t)
    assert torch.equal(g, sd.distill(t.detach(), ids, z, lse, torch.full_like(w, 0.5)).grad)


def test_gradient_by_differences(sd):
    """Of the float32 loss: a step of 2^-5 leaves 2^-10 / 6 of the third derivative (below 1) and a
    rounding of the losses (4e-5, as above) over 2^-4: 2e-4 + 7e-4."""
    x = normal(15, 1, 1, 50)
    ids, z, lse = (cuda(a) for a in teacher(7, x, 8, 1.0, True))
    t = on_gpu(x, "f32")
    for whole in (lse, None):
        g = sd.distill(t, ids, z, whole).grad
        for v in range(0, 50, 3):
            e = torch.zeros_like(t)
            e[0, 0, v] = 2.0 ** -5
            f = lambda y: float(sd.distill(y, ids, z, whole, grad=False).loss)
            assert abs((f(t + e) - f(t - e)) * 16 - float(g[0, 0, v])) <= 1e-3


def test_empty_batch(sd):
    r = sd.distill(torch.zeros(0, 2, 5).cuda(), torch.zeros(0, 2, 1, dtype=torch.int32).cuda(),
                   torch.zeros(0, 2, 1).cuda())
    assert r.loss.shape == (0, 2) and r.grad.shape == (0, 2, 5)
