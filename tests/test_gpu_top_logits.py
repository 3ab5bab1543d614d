"""specdec_top_logits against float64: values and tokens exactly, the log-sum-exp to what float32
carries."""
import numpy as np
import pytest

import draft_oracle as ref
from test_gpu_sample import normal, on_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def check(sd, x, K, T=1.0, dtype="f32", pad=0, shift=0, rows=None):
    B, R, V = x.shape
    t = on_gpu(x, dtype, pad, shift)
    got = sd.top_logits(t, K, T)
    T = float(np.float32(T))
    for b in range(B):
        for r in range(R):
            if rows is not None and (b, r) not in rows:
                continue
            values, ids, lse = ref.record(t[b, r].double().cpu().numpy(), K, T)
            assert got.row_status[b, r] == 0
            assert got.ids[b, r].tolist() == ids.tolist(), (b, r)
            assert np.array_equal(got.values[b, r].double().cpu().numpy(), values)
            # the sum: arguments off by 3 * 2^-24 |y| ln 2, |y| <= 64 (smaller weights are less of the
            # sum than that), ex2 by 2^-22, 64 float32 additions; then one rounding of the result
            tol = 3 * 64 * 0.7 * 2.0 ** -24 + 2.0 ** -22 + 64 * 2.0 ** -24 + 2.0 ** -24 * abs(lse)
            assert abs(float(got.lse[b, r]) - lse) <= tol
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,K", [(1, 1), (5, 3), (5, 5), (64, 17), (1000, 1), (1000, 64), (1000, 1000),
                                 (1024, 1024), (5003, 256), (8191, 1024)])
def test_sizes(sd, dtype, V, K):
    check(sd, normal(V + K, 2, 3, V), K, T=0.7, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (5, 7)])
def test_rows_that_start_anywhere(sd, dtype, pad, shift):
    check(sd, normal(3, 2, 3, 9001), 50, dtype=dtype, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype,V", [("bf16", 128256), ("f32", 128256), ("bf16", 1 << 21), ("f32", 1 << 21)])
@pytest.mark.parametrize("K", [1, 64, 1024])
def test_large_vocabularies(sd, dtype, V, K):
    check(sd, np.random.default_rng(V).standard_normal((1, 2, V)).astype(np.float32), K, dtype=dtype,
          rows={(0, 1)})


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 100, 1024])
def test_equal_logits_rank_by_index(sd, dtype, K):
    check(sd, np.full((1, 1, 20000), -3.25), K, dtype=dtype)
    x = np.full((1, 2, 9001), 1.5)
    x[0, 0, ::7] = 2.0
    x[0, 1, -3:] = 2.0
    check(sd, x, K, dtype=dtype)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("K", [64, 1024])
def test_sorted_rows(sd, order, K):
    for dtype in ("f32", "bf16"):
        check(sd, np.sort(normal(5, 1, 1, 60000))[:, :, ::order], K, dtype=dtype)


def test_minus_infinity_and_signs_of_zero(sd):
    x = normal(6, 3, 1, 5000)
    x[0, 0, 100:] = -np.inf
    x[1, 0, 1:] = -np.inf
    x[2] = 0.0
    x[2, 0, ::3] = -0.0
    for dtype in ("f32", "bf16"):
        check(sd, x, 300, dtype=dtype)


def test_bad_rows(sd):
    x = normal(7, 5, 1, 4000)
    x[0, 0, 3999] = np.nan
    x[1, 0, 0] = np.inf
    x[2] = -np.inf
    x[3, 0, 7] = 2.0 ** 101
    for dtype in ("f32", "bf16"):
        r = sd.top_logits(on_gpu(x, dtype), 9)
        assert r.row_status[:, 0].tolist() == [sd.ROW_NONFINITE] * 4 + [0]
        assert r.values[:4].isnan().all() and (r.ids[:4] == -1).all() and r.lse[:4].isnan().all()
        assert (r.ids[4] >= 0).all()


def test_workspace_and_outputs_of_the_caller(sd):
    x = on_gpu(normal(8, 2, 3, 3000), "bf16")
    want = sd.top_logits(x, 10)
    n = sd.top_logits_workspace_size(2, 3, 3000, sd.BF16)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    out = sd.TopOut(*[torch.empty_like(v) for v in vars(want).values()])
    assert sd.top_logits(x, 10, out=out, workspace=ws) is out
    for name, v in vars(want).items():
        assert torch.equal(v, getattr(out, name)), name
    with pytest.raises(sd.SpecdecError):
        sd.top_logits(x, 10, workspace=ws[:n - 16].clone())
    assert sd.top_logits(torch.zeros(0, 2, 5).cuda(), 2).ids.shape == (0, 2, 2)


@pytest.mark.parametrize("K", [5, 64, 300])
def test_many_rows(sd, K):
    """More rows than the GPU holds at once, some with runs of equal logits."""
    x = np.random.default_rng(K).standard_normal((700, 3, 600)).astype(np.float32)
    x[5], x[699, :, ::2] = 0.5, 3.0
    check(sd, x, K, rows={(0, 0), (5, 1), (300, 2), (699, 0), (699, 2)})
    t = on_gpu(x, "bf16")
    got = sd.top_logits(t, K)
    want = torch.sort(t.float(), dim=-1, descending=True, stable=True)
    assert torch.equal(got.ids, want.indices[..., :K].int())
    assert torch.equal(got.values, want.values[..., :K])
