"""specdec_sample against float64: tokens, kept counts and cuts exactly, distributions to what
float32 carries."""
import numpy as np
import pytest

import draft_oracle as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def uniforms(rng, shape):
    return ((rng.integers(0, 2 ** 23, shape) + 0.5) * 2.0 ** -23).astype(np.float32)


def on_gpu(x, dtype, pad=0, shift=0):
    """x [B, R, V] as rows `pad` elements apart that begin `shift` elements into a buffer."""
    B, R, V = x.shape
    buf = torch.full((B * R * (V + pad) + shift,), 1e9, dtype=DT[dtype], device="cuda")
    t = buf[shift:].view(B, R, V + pad)[:, :, :V]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return t


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32).cuda()


def floats(v):
    return None if v is None else torch.tensor(v, dtype=torch.float32).cuda()


def tolerance(x, T, q, dtype):
    """A weight is 2^y, y = (l - max) c: each of the difference, c and the product is rounded
    (3 * 2^-24 |y| ln 2 of the weight), ex2 is good to 2^-22 and the factor and its product to
    2^-24 each; then the stored type's half step.  Below 2^-120 a weight may be flushed."""
    y = np.abs(np.where(np.isfinite(x), x - np.max(x), 0.0)) / max(T, 1e-30) * 1.4427
    rel = 3 * 2.0 ** -24 * 0.7 * y + 2.0 ** -22 + 2.0 ** -23 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
    return q * rel * 1.0001 + 2.0 ** -120


def check(sd, x, T, S=2, k=None, p=None, m=None, dtype="f32", pad=0, shift=0, seed=0, rows=None):
    """x [B, R, V]; T, k, p, m lists of B; rows: those that are looked at (all)."""
    B, R, V = x.shape
    u = uniforms(np.random.default_rng(seed + 77), (B, R, S))
    t = on_gpu(x, dtype, pad, shift)
    got = sd.sample(t, floats(T), torch.from_numpy(u).cuda(), ints(k), floats(p), floats(m))
    flt = sd.filter_logits(t, floats(T), ints(k), floats(p), floats(m))
    f32 = lambda v, b, d: d if v is None else float(np.float32(v[b]))
    for b in range(B):
        Tb, kb, pb, mb = f32(T, b, 0), 0 if k is None else k[b], f32(p, b, 1.0), f32(m, b, 0.0)
        for r in range(R):
            if rows is not None and (b, r) not in rows:
                continue
            y = t[b, r].double().cpu().numpy()  # as stored
            tokens, q, mask = ref.sample(y, Tb, u[b, r], kb, pb, mb)
            assert got.row_status[b, r] == 0
            assert int(got.kept[b, r]) == mask.sum() == int(flt.kept[b, r]), (b, r)
            assert got.tokens[b, r].tolist() == tokens, (b, r)
            g = got.rows[b, r].double().cpu().numpy()
            assert not g[~mask].any()
            assert (np.abs(g - q) <= tolerance(y, Tb, q, dtype)).all(), (b, r, np.abs(g - q).max())
            f = flt.rows[b, r].double().cpu().numpy()
            assert np.array_equal(f, np.where(mask, y, -np.inf)), (b, r)
    return got


def normal(seed, B, R, V, scale=2.0):
    return np.random.default_rng(seed).standard_normal((B, R, V)) * scale


FILTERS = [dict(), dict(k=[5, 40, 1]), dict(p=[0.9, 0.3, 0.999]), dict(m=[0.02, 0.5, 0.0001]),
           dict(k=[50, 0, 20], p=[0.8, 0.95, 1.0]), dict(k=[0, 7, 100], p=[0.7, 1.0, 0.5], m=[0.2, 0.1, 0.0]),
           dict(p=[0.9, 0.6, 0.0], m=[0.05, 0.0, 1.0])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 1000, 5003])
@pytest.mark.parametrize("f", range(len(FILTERS)))
def test_small_vocabularies(sd, dtype, V, f):
    check(sd, normal(V + f, 3, 2, V), [0.7, 0.0, 1.3], dtype=dtype, seed=V, **FILTERS[f])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (5, 7), (8, 2)])
def test_rows_that_start_anywhere(sd, dtype, pad, shift):
    check(sd, normal(9, 2, 3, 1501), [1.0, 0.6], dtype=dtype, pad=pad, shift=shift, p=[0.8, 1.0], k=[0, 30])


@pytest.mark.parametrize("dtype,V,B", [("bf16", 128256, 1), ("f32", 128256, 1), ("f32", 32000, 1),
                                       ("bf16", 20000, 12), ("bf16", 40001, 120), ("f32", 3001, 300)])
@pytest.mark.parametrize("f", [0, 1, 2, 4])
def test_clusters_of_every_size(sd, dtype, V, B, f):
    """From one row (16 CTAs) to as many as fill the GPU with one or two CTAs each."""
    flt = {n: [v[b % 3] for b in range(B)] for n, v in FILTERS[f].items()}
    x = np.random.default_rng(V + f).standard_normal((B, 1, V)).astype(np.float32)
    look = {(b, 0) for b in (0, 1, 2, B // 2, B - 1)}
    check(sd, x, [0.9] * B, dtype=dtype, rows=look, **flt)


# float32 rows that take 3, 5, 6, 7, 8, 10, 12, 14 and 16 CTAs, the smaller numbers of them by
# as many rows as leave no SM idle
WIDE = [(50001, 80), (80000, 50), (100003, 40), (115000, 34), (130002, 30), (160001, 20), (200000, 16),
        (240005, 13), (300000, 11)]


@pytest.mark.parametrize("V,B", WIDE)
@pytest.mark.parametrize("k", [1, 128, 129, 1024])
def test_top_k_in_clusters_of_every_size(sd, V, B, k):
    """The bound from groups of several lanes (up to 128) and of one thread's part."""
    x = np.random.default_rng(V + k).standard_normal((B, 1, V)).astype(np.float32)
    check(sd, x, [0.9] * B, rows={(0, 0), (B - 1, 0)}, k=[k] * B, p=[0.97] * B)


@pytest.mark.parametrize("V,B", WIDE)
def test_top_p_in_clusters_of_every_size(sd, V, B):
    x = np.random.default_rng(V).standard_normal((B, 1, V)).astype(np.float32)
    check(sd, x, [0.9] * B, rows={(0, 0), (B - 1, 0)}, p=[0.9, 0.5] * (B // 2) + [0.99] * (B % 2))


def test_the_largest_vocabulary(sd):
    V = 1 << 19
    for dtype in ("f32", "bf16"):
        check(sd, normal(3, 1, 2, V), [1.0], dtype=dtype, p=[0.9], rows={(0, 1)}, S=1)
        check(sd, normal(4, 1, 1, V), [1.0], dtype=dtype, k=[1000], S=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("flt", [dict(), dict(k=[300]), dict(k=[1024]), dict(p=[0.5]), dict(p=[0.25], m=[0.9]),
                                 dict(k=[1000], p=[0.75])])
def test_equal_logits_rank_by_index(sd, dtype, flt):
    """More equal tokens than any list holds, and shares that fall on a token's border."""
    check(sd, np.full((1, 1, 20000), -3.25), [0.7], dtype=dtype, S=3, **flt)
    x = np.full((1, 1, 9000), 1.5)
    x[0, 0, ::7] = 2.0
    check(sd, x, [1.0], dtype=dtype, S=3, **flt)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("flt", [dict(k=[1024]), dict(k=[64], p=[0.9]), dict(p=[0.9])])
def test_sorted_rows(sd, order, flt):
    x = np.sort(normal(5, 1, 1, 30000))[:, :, ::order]
    for dtype in ("f32", "bf16"):
        check(sd, x, [1.0], dtype=dtype, **flt)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_at_minus_infinity(sd, dtype):
    x = normal(6, 4, 1, 3000)
    x[:, :, 100:] = -np.inf
    x[1, 0, 1:] = -np.inf          # one token left
    x[2, 0, :] = -np.inf
    x[2, 0, 2999] = -50.0          # the last one
    x[3, 0, 5:] = -np.inf          # fewer than top-k asks for
    x[3, 0, 2] = np.finfo(np.float32).min if dtype == "f32" else -3.3e38
    for f in (dict(), dict(k=[40] * 4), dict(p=[0.9] * 4), dict(k=[40] * 4, p=[0.9] * 4, m=[0.01] * 4)):
        check(sd, x, [0.8] * 4, dtype=dtype, **f)


@pytest.mark.parametrize("T", [2.0 ** -20, 1e-3, 0.05, 30.0, 2.0 ** 20])
@pytest.mark.parametrize("offset", [0.0, 1000.0, -30000.0, 1e30])
def test_temperatures_and_offsets(sd, T, offset):
    for dtype in ("f32", "bf16"):
        x = normal(8, 3, 1, 2000) + offset
        check(sd, x, [T] * 3, dtype=dtype, k=[0, 50, 0], p=[1.0, 0.9, 0.9])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_flat_rows_and_rows_of_few_values(sd, dtype):
    """Borders among thousands of near equal tokens, heavy heads, logits coarser than any bin."""
    rng = np.random.default_rng(21)
    V = 40000
    x = np.stack([rng.standard_normal(V) * 0.01, rng.standard_normal(V) * 3, rng.integers(-3, 4, V) * 1.0,
                  np.where(np.arange(V) < 3, 12.0, rng.standard_normal(V)), np.linspace(-1, 1, V),
                  1000 + rng.integers(0, 3, V) * 8.0])[:, None]
    T = [1.0, 0.7, 0.5, 1.0, 2.0, 2.0 ** -20]
    for p, m in ((0.9, 0.0), (0.5, 0.0), (0.999, 0.0), (0.95, 0.001), (0.3, 0.9), (0.9, 0.5), (1e-6, 0.0)):
        check(sd, x, T, dtype=dtype, p=[p] * 6, m=[m] * 6)


@pytest.mark.parametrize("V", [900, 30000, 128256])
@pytest.mark.parametrize("kind", ["tiny", "low", "mixed", "few", "one", "high"])
def test_values_that_are_counted_and_others(sd, V, kind):
    """bfloat16 rows whose cut is at a value near 0, far below it, between those, at a value of
    thousands of tokens, or above what is counted."""
    rng = np.random.default_rng(V)
    T = 1.0
    if kind == "tiny":
        x = rng.standard_normal((1, 1, V)) * 2.0 ** -16
    elif kind == "low":
        x, T = -64.0 - 400.0 * rng.random((1, 1, V)), 200.0
        x[0, 0, rng.integers(0, V, 20)] = 1.0
    elif kind == "mixed":
        x = rng.choice([1.5, 2.0 ** -17, -2.0 ** -20, 0.0, -0.75, -3.0, -200.0], size=(1, 1, V))
        T = 50.0
    elif kind == "few":
        x = rng.choice([0.5, 0.25, -0.125, -2.0], size=(1, 1, V))
    elif kind == "one":
        x = np.full((1, 1, V), -1.25)
    else:
        x, T = 30.0 + 60.0 * rng.random((1, 1, V)), 40.0
    ps = [0.01, 0.15, 0.29, 0.43, 0.5, 0.57, 0.72, 0.86, 0.97, 0.99999]
    n = len(ps)
    check(sd, np.broadcast_to(x, (n, 1, V)), [T] * n, dtype="bf16", p=ps, seed=V)
    check(sd, np.broadcast_to(x, (n, 1, V)), [T] * n, dtype="bf16", p=ps, m=[0.0, 0.9] * (n // 2), S=0)


def test_zeros_of_both_signs_and_denormals(sd):
    x = np.zeros((1, 1, 6000))
    x[0, 0, ::2] = -0.0
    x[0, 0, 1::3] = -1e-40
    x[0, 0, 2::5] = 1e-40
    for f in (dict(k=[700]), dict(p=[0.4]), dict(p=[0.7]), dict(), dict(m=[1.0])):
        check(sd, x, [1.0], S=4, **f)
    x[0, 0, 1::2] = -1.0     # the largest is a zero
    for f in (dict(k=[2000]), dict(p=[0.4]), dict(m=[1.0]), dict(m=[0.9], p=[0.5])):
        f = {n: [min(v[0], 1000)] for n, v in f.items()}
        for dtype in ("f32", "bf16"):
            check(sd, x, [1.0], S=4, dtype=dtype, **f)


@pytest.mark.parametrize("S", [0, 1, 63, 64])
def test_numbers_of_draws(sd, S):
    check(sd, normal(10, 2, 2, 3000), [1.0, 0.8], S=S, p=[0.9, 1.0], k=[0, 100])


def test_law_of_the_draws(sd):
    """A grid of uniforms meets every token as often as its probability says, to one either way."""
    V, n = 37, 64 * 40
    x = torch.randn(1, 1, V, generator=torch.Generator().manual_seed(1)).cuda()
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float().cuda()
    r = sd.sample(x.expand(1, 40, V).contiguous(), floats([1.0]), u.view(1, 40, 64).contiguous())
    seen = torch.bincount(r.tokens.flatten().long().cpu(), minlength=V).double()
    assert (seen - n * torch.softmax(x[0, 0].double().cpu(), 0)).abs().max() <= 1.001


def test_bad_rows_and_parameters(sd):
    V = 300
    x = normal(11, 9, 1, V)
    x[0, 0, 5] = np.nan
    x[1, 0, 299] = np.inf
    x[2] = -np.inf
    x[3, 0, 0] = 2.0 ** 101
    nan = float("nan")
    T = [1.0, 1.0, 1.0, 1.0, -1.0, 1.0, 1.0, 1.0, nan]
    k = [0, 5, 5, 0, 0, -1, 1025, 0, 0]
    p = [0.5, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.5, 1.0]
    want = [sd.ROW_NONFINITE] * 4 + [sd.ROW_BAD_TEMP] + [sd.ROW_BAD_FILTER] * 3 + [sd.ROW_BAD_TEMP]
    u = torch.full((9, 1, 2), 0.5).cuda()
    for dtype in ("f32", "bf16"):
        r = sd.sample(on_gpu(x, dtype), floats(T), u, ints(k), floats(p))
        assert r.row_status[:, 0].tolist() == want
        assert (r.tokens == -1).all() and (r.kept == 0).all() and r.rows.isnan().all()
    for flt in (dict(top_p=floats([nan])), dict(min_p=floats([nan])), dict(min_p=floats([-0.1])),
                dict(top_p=floats([-1e-9])), dict(min_p=floats([1.1]))):
        r = sd.sample(torch.zeros(1, 1, 8).cuda(), floats([1.0]), torch.full((1, 1, 1), 0.5).cuda(), **flt)
        assert r.row_status.item() == sd.ROW_BAD_FILTER
    # uniforms outside (0, 1) draw the first or the last kept token
    r = sd.sample(torch.zeros(1, 1, 8).cuda(), floats([1.0]), floats([[[0.0, 1.0, -3.0, 2.0, nan]]]))
    assert r.tokens[0, 0].tolist() == [0, 7, 0, 7, 0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_into_slices_and_in_place(sd, dtype):
    """A draft loop writes q[:, i]; a filter may work on the logits themselves."""
    V, gamma = 1003, 3
    q = torch.full((2, gamma, V), 9.0, dtype=DT[dtype], device="cuda")
    keep = q.clone()
    x = on_gpu(normal(12, 2, 1, V), dtype)
    u = torch.full((2, 1, 1), 0.4).cuda()
    T, p = floats([1.0, 0.5]), floats([0.9, 0.8])
    want = sd.sample(x, T, u, top_p=p)
    for i in range(gamma):
        out = sd.SampleOut(torch.empty(2, 1, 1, dtype=torch.int32, device="cuda"), q[:, i:i + 1],
                           torch.empty(2, 1, dtype=torch.int32, device="cuda"),
                           torch.empty(2, 1, dtype=torch.int32, device="cuda"))
        sd.sample(x, T, u, top_p=p, out=out)
        assert torch.equal(q[:, i], want.rows[:, 0]) and torch.equal(q[:, i + 1:], keep[:, i + 1:])
        assert torch.equal(out.tokens, want.tokens)
    flt = sd.filter_logits(x, T, top_p=p)
    y = on_gpu(x.double().cpu().numpy(), dtype, pad=5, shift=3)
    whole = y._base.clone()
    sd.filter_logits(y, T, top_p=p, out=sd.SampleOut(None, y, flt.kept, flt.row_status))
    assert torch.equal(y, flt.rows)
    y.copy_(x)
    assert torch.equal(y._base, whole)   # nothing beside the rows
    with pytest.raises(sd.SpecdecError):
        buf = torch.zeros(2 * V + 8, dtype=DT[dtype], device="cuda")
        a, b = buf[:2 * V].view(2, 1, V), buf[8:].view(2, 1, V)
        sd.filter_logits(a, T, out=sd.SampleOut(None, b, flt.kept, flt.row_status))


def test_requests_in_another_order(sd):
    """[R, B, V] logits: a request's rows far apart, the requests side by side."""
    x = on_gpu(normal(13, 3, 2, 700), "f32")
    u = torch.from_numpy(uniforms(np.random.default_rng(1), (2, 3, 1))).cuda()
    T, p = floats([1.0, 0.6]), floats([0.9, 0.7])
    a = sd.sample(x.transpose(0, 1), T, u, top_p=p)
    b = sd.sample(x.transpose(0, 1).contiguous(), T, u, top_p=p)
    for n, v in vars(a).items():
        assert torch.equal(v, getattr(b, n)), n


def test_the_same_call_gives_the_same(sd):
    x = on_gpu(normal(14, 5, 2, 30011), "bf16")
    u = torch.rand(5, 2, 3, generator=torch.Generator().manual_seed(2)).cuda()
    a = [sd.sample(x, floats([0.8] * 5), u, ints([0, 64, 0, 1, 900]), floats([0.9, 0.9, 1.0, 1.0, 0.5]))
         for _ in range(3)]
    for n, v in vars(a[0]).items():
        assert torch.equal(v, getattr(a[1], n)) and torch.equal(v, getattr(a[2], n)), n


def test_empty_batch(sd):
    r = sd.sample(torch.zeros(0, 2, 5).cuda(), floats([]), torch.zeros(0, 2, 1).cuda())
    assert r.tokens.shape == (0, 2, 1)
