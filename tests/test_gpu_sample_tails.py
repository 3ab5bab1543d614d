"""specdec_sample on rows of one large token and a long tail of equal ones far below: cuts and draws are
those of sums that are off by V * 2^-43 of the largest weight and 2^-34 of themselves at most."""
import numpy as np
import pytest

from test_gpu_sample import floats, on_gpu, tolerance

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


U = np.array([2.0 ** -40, 2.0 ** -30, 1e-9, 6e-8, 0.5, 1 - 2.0 ** -20, 1 - 2.0 ** -23, 1 - 2.0 ** -24],
             dtype=np.float32)
P = np.array([0.25, 0.999, 1 - 2.0 ** -22, 1 - 2.0 ** -24, 1.0], dtype=np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5000, 128256, 1 << 19])
@pytest.mark.parametrize("down", [20.0, 28.0, 29.75, 30.0, 35.0])
@pytest.mark.parametrize("peak", ["first", "last"])
def test_far_tails(sd, V, down, peak, dtype):
    at = 0 if peak == "first" else V - 1
    x = np.full((len(P), 1, V), 1.5 - down)  # (exact in both types)
    x[:, 0, at] = 1.5
    t, T = on_gpu(x, dtype), floats([1.0] * len(P))
    u = torch.from_numpy(np.broadcast_to(U, (len(P), 1, len(U))).copy()).cuda()
    got = sd.sample(t, T, u, top_p=floats(P))
    flt = sd.filter_logits(t, T, top_p=floats(P))
    assert (got.row_status == 0).all() and torch.equal(got.kept, flt.kept)
    w = np.exp(-down)
    Z = 1 + (V - 1) * w
    off = V * 2.0 ** -43 + 2.0 ** -34 * Z
    for b, p in enumerate(P.astype(np.float64)):
        kept = int(got.kept[b, 0])
        mass = 1 + (kept - 1) * w
        # the cut: two sums are compared, each off by `off`
        if p < 1:
            assert mass >= p * Z - 2 * off
            assert kept == 1 or mass - w <= p * Z + 2 * off
        else:
            assert kept == V
        # the kept are the peak and the first of the others
        mask = np.zeros(V, dtype=bool)
        mask[at] = True
        mask[np.flatnonzero(~mask)[:kept - 1]] = True
        y = x[b, 0]
        assert np.array_equal(flt.rows[b, 0].double().cpu().numpy(), np.where(mask, y, -np.inf))
        q = np.where(mask, np.exp(y - 1.5), 0.0) / mass
        g = got.rows[b, 0].double().cpu().numpy()
        assert not g[~mask].any()
        assert (np.abs(g - q) <= tolerance(y, 1.0, q, dtype) + 2 * off * q).all()
        # the draws
        run = np.cumsum(np.where(mask, np.exp(y - 1.5), 0.0))
        for v, token in zip(U.astype(np.float64), got.tokens[b, 0].tolist()):
            assert mask[token]
            assert run[token] >= v * mass - 2 * off
            assert token == 0 or run[token - 1] <= v * mass + 2 * off
            if w < 2.0 ** -43:
                assert token == at
