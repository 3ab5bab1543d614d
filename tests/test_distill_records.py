"""The float64 form of distillation that the GPU tests compare with, on records whose shares do not add
up to 1 (no GPU)."""
import numpy as np
import pytest

import draft_oracle as ref


@pytest.mark.parametrize("mass", [0.2, 0.9999, 1.0001, 1.5, 2.27, 40.0])
@pytest.mark.parametrize("ids", [[7, -1, 2], [0, 1, 2]])
def test_gradient_by_differences(mass, ids):
    rng = np.random.default_rng(1)
    x, z = rng.standard_normal(9) * 2, rng.standard_normal(3)
    some = np.array(ids) >= 0
    lse = np.log(np.exp(z[some] / 1.3).sum() / mass)
    loss, g = ref.distill(x, ids, z, lse, T=1.3)
    for v in range(9):
        e = np.zeros(9)
        e[v] = 1e-5
        d = (ref.distill(x + e, ids, z, lse, T=1.3)[0] - ref.distill(x - e, ids, z, lse, T=1.3)[0]) / 2e-5
        # third derivatives of up to the shares' sum over T^3; a loss below 200 rounded to 2^-53 of itself
        assert abs(d - g[v]) < mass * 1e-10 + 200 * 2.0 ** -53 / 1e-5
    assert abs(g.sum()) < 1e-12 * max(1.0, mass)


def test_records_of_all_tokens_are_finite():
    """A float32 log-sum-exp leaves up to 2^-24 of itself over, for which there is no token."""
    for offset in (0.0, 20.0, 40.0, 100.0, 300.0, 5000.0):
        rng = np.random.default_rng(int(offset))
        over = 0.0
        for _ in range(50):
            x = np.full(64, -np.inf)
            x[:10] = rng.standard_normal(10) * 2 + offset
            z = (x[:10] + rng.standard_normal(10)).astype(np.float32)
            y = z.astype(np.float64)
            lse = np.float32(y.max() + np.log(np.exp(y - y.max()).sum()))
            over = max(over, 1.0 - np.exp(y - float(lse)).sum())
            loss, g = ref.distill(x, np.arange(10), z, lse)
            assert np.isfinite(loss) and np.isfinite(g).all()
        assert over <= offset * 2.0 ** -24 + 2.0 ** -20
    # what is more than that has nowhere to go
    x[10:] = -np.inf
    with np.errstate(divide="ignore", invalid="ignore"):
        assert ref.distill(x, np.arange(10), z, float(lse) + 0.01)[0] == np.inf
