"""Attention of drafted tokens over the 8-bit cache against the formula in 64 bits.

Tolerance, with A = sum p |v| / sum p of the element and S the largest scale * sum |q| |k| of
its row: a score is off by at most 2^-16 (1 + S) for bfloat16 activations (q is carried to 2^-19
of its row's largest element, the rest is float32) and 2^-19 (1 + S) for float32 ones (two fp16
terms an operand, 2^-22, and float32 sums), with the cap's 2^-21 softcap more; the weights of the
products carry 2^-11 or 2^-21; both sides of the quotient are affected:
    |out error| <= A (2 ds + 2 dw) (+ 2^-8 |out| for a bfloat16 result and its reduction)
    |lse error| <= ds + 2^-20 (1 + |lse|)
"""
import math

import numpy as np
import pytest

import attention_oracle as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def tokens(rng, B, N, Hq, Hkv, D, dtype, pad=0):
    """q, k, v as slices of one fused projection, `pad` elements between tokens."""
    H = Hq + 2 * Hkv
    x = torch.from_numpy(rng.standard_normal((B, N, H * D + pad)) * 1.5).to(dtype).cuda()
    y = x[..., :H * D].unflatten(2, (H, D))
    return y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:]


def check(r, q, k, v, cache, block, parents, nodes, scale, softcap=0.0, slopes=None, window=0,
          skip=()):
    B, N, Hq, D = q.shape
    f32 = q.dtype == torch.float32
    out, lse = r.out.double().cpu(), r.lse.double().cpu()
    for b in range(B):
        if b in skip:
            continue
        kc, vc = (ref.cached_values(cache, n, b, block) for n in ("k", "v"))
        want, wl, A, S = ref.attend(q[b].double().cpu(), k[b].double().cpu(), v[b].double().cpu(),
                                    None if parents is None else parents[b], nodes[b], kc, vc,
                                    int(cache["length"][b]), scale, softcap, slopes, window)
        ds = 2.0 ** (-19 if f32 else -16) * (1 + S) + 2.0 ** -21 * softcap
        dw = 2.0 ** (-21 if f32 else -11)
        tol = A * (2 * ds + 2 * dw)[..., None]
        if not f32:
            tol = tol + want.abs() * 2.0 ** -8
        empty = wl == -math.inf
        assert (out[b][empty] == 0).all() and (lse[b][empty] == -math.inf).all(), b
        bad = ~torch.isfinite(want)
        assert torch.equal(torch.isfinite(out[b]), ~bad), b
        err = torch.where(bad, 0.0, (out[b] - want).abs())
        assert (err <= torch.where(bad, 1.0, tol)).all(), \
            (b, float((err - tol).nan_to_num(-1).max()), float(err.max()))
        ok = torch.isfinite(wl)
        assert ((lse[b] - wl).abs()[ok] <= (ds + 2.0 ** -20 * (1 + wl.abs()))[ok]).all(), b
    keep = [b for b in range(B) if b not in skip]
    assert (r.row_status.cpu()[keep] == 0).all()


SHAPES = [
    # B lens, N, Hq, Hkv, D, block, pad
    ([0], 1, 1, 1, 16, 16, 0),
    ([1, 15, 16, 17], 1, 4, 4, 64, 16, 0),
    ([63, 64, 65, 0, 200], 3, 6, 2, 128, 64, 0),
    ([300, 5], 9, 32, 8, 128, 64, 8),
    ([129, 255], 5, 10, 2, 96, 32, 0),
    ([100, 0, 33], 17, 4, 1, 80, 16, 1),
    ([70, 513], 4, 8, 2, 256, 128, 0),
    ([31], 33, 5, 1, 48, 16, 0),
    ([40], 2, 3, 1, 208, 16, 0),
    ([1030], 6, 8, 1, 128, 1024, 0),
    ([2500, 3], 1, 16, 2, 128, 64, 0),
    ([700, 90], 16, 64, 4, 64, 32, 0),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,N,Hq,Hkv,D,block,pad", SHAPES)
def test_chains(sd, dtype, lens, N, Hq, Hkv, D, block, pad):
    rng = np.random.default_rng(sum(lens) + D)
    q, k, v = tokens(rng, len(lens), N, Hq, Hkv, D, dtype, pad)
    cache = ref.make_cache(rng, lens, [0] * len(lens), block, Hkv, D, scales="any")
    r = sd.attend(q, k, v, ref.on_gpu(cache))
    check(r, q, k, v, cache, block, None, [N] * len(lens), D ** -0.5)
    again = sd.attend(q, k, v, ref.on_gpu(cache))
    assert torch.equal(r.out, again.out) and torch.equal(r.lse, again.lse)


@pytest.mark.parametrize("B,N,Hq,Hkv,most,window", [(100, 3, 16, 8, 900, 0), (48, 17, 32, 8, 600, 0),
                                                    (90, 2, 8, 8, 700, 300), (300, 1, 2, 2, 400, 0)])
def test_many_requests(sd, B, N, Hq, Hkv, most, window):
    """More requests and heads than the device has SMs, of every length: a CTA works through
    several of them, whole and in part, and tiles of cached and of drafted tokens alternate."""
    rng = np.random.default_rng(B)
    D, block = 64, 32
    lens = [int(n) for n in rng.integers(0, most, B)]
    lens[::7] = [0] * len(lens[::7])
    nodes = [int(n) for n in rng.integers(0, N + 1, B)]
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, torch.bfloat16)
    cache = ref.make_cache(rng, lens, [0] * B, block, Hkv, D)
    n_nodes = torch.tensor(nodes, dtype=torch.int32).cuda()
    r = sd.attend(q, k, v, ref.on_gpu(cache), n_nodes=n_nodes, window=window)
    check(r, q, k, v, cache, block, None, nodes, D ** -0.5, window=window)
    again = sd.attend(q, k, v, ref.on_gpu(cache), n_nodes=n_nodes, window=window)
    assert torch.equal(r.out, again.out) and torch.equal(r.lse, again.lse)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("softcap,bias,window", [(0.0, False, 0), (30.0, False, 0), (0.0, True, 0),
                                                 (0.0, False, 50), (20.0, True, 7), (0.0, True, 1)])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(64, 8, 2, 128), (23, 3, 3, 64), (130, 2, 1, 96)])
def test_trees(sd, dtype, softcap, bias, window, N, Hq, Hkv, D):
    rng = np.random.default_rng(N + window)
    lens, block = [0, 1, 47, 48, 130], 16
    B = len(lens)
    nodes = [N, N - 1, 1, 0, N // 2]
    parents = [ref.random_tree(rng, N) for _ in lens]
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, dtype)
    cache = ref.make_cache(rng, lens, [0] * B, block, Hkv, D)
    slopes = torch.linspace(0.01, 0.5, Hq) if bias else None
    for ragged in (False, True):
        n = nodes if ragged else [N] * B
        if ragged:   # what stands past a request's nodes is not read
            for t in (q, k, v):
                for b in range(B):
                    t[b, n[b]:] = float("nan")
        parent = torch.tensor(parents, dtype=torch.int32)
        if ragged:
            for b in range(B):
                parent[b, n[b]:] = 2 ** 31 - 1
        r = sd.attend(q, k, v, ref.on_gpu(cache), parent=parent.cuda(),
                      n_nodes=torch.tensor(n, dtype=torch.int32).cuda() if ragged else None,
                      scale=0.1, softcap=softcap, slopes=slopes.cuda() if bias else None,
                      window=window)
        check(r, q, k, v, cache, block, parents, n, 0.1, softcap, slopes, window)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (128, 1)])
def test_non_finite_values_reach_only_the_rows_that_see_them(sd, dtype, D, G):
    rng = np.random.default_rng(9)
    lens, N, Hkv, block = [60, 61], 31, 2, 16
    parents = [ref.random_tree(rng, N) for _ in lens]
    q, k, v = tokens(rng, 2, N, Hkv * G, Hkv, D, dtype)
    v[0, 4, 0, 3], v[0, 9, 1, 5], v[1, 30, 0, 0] = float("nan"), float("inf"), float("-inf")
    k[1, 7, 1, 2] = float("nan")
    cache = ref.make_cache(rng, lens, [0, 0], block, Hkv, D)
    # NaN codes in tokens that a window of 40 hides from some nodes, and from all
    window = 40
    for b, j in ((0, 23), (1, 24), (0, 2), (1, 5)):
        cache["v"][cache["block_table"][b, j // block], 1, j % block, 7] = 0xFF
        cache["k"][cache["block_table"][b, j // block], 0, j % block, 7] = 0x7F
    r = sd.attend(q, k, v, ref.on_gpu(cache), parent=torch.tensor(parents).int().cuda(),
                  window=window)
    check(r, q, k, v, cache, block, parents, [N, N], D ** -0.5, window=window)
    # a NaN that everybody sees reaches everybody
    r = sd.attend(q, k, v, ref.on_gpu(cache), parent=torch.tensor(parents).int().cuda())
    check(r, q, k, v, cache, block, parents, [N, N], D ** -0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_ranges(sd, dtype):
    """Block scales and token sizes that differ by powers of ten, scores far apart, a sink that
    takes most of the weight, rows of zeros."""
    rng = np.random.default_rng(10)
    lens, N, Hq, Hkv, D, block = [400, 1000], 7, 8, 2, 128, 16
    q, k, v = tokens(rng, 2, N, Hq, Hkv, D, dtype)
    q *= 10.0 ** torch.linspace(-4, 1, N, device="cuda")[None, :, None, None].to(dtype)
    v *= 10.0 ** torch.linspace(-6, 6, N, device="cuda")[None, :, None, None].to(dtype)
    q[0, 2] = 0
    k[1, 3] = 0
    v[1, 4] = 0
    cache = ref.make_cache(rng, lens, [0, 0], block, Hkv, D)
    nb = cache["k"].shape[0]
    cache["v_scale"] = torch.from_numpy(10.0 ** rng.uniform(-6, 2, (nb, Hkv))).float()
    cache["k_scale"] = torch.from_numpy(2.0 ** rng.integers(-9, -3, (nb, Hkv))).float()
    cache["v_scale"][cache["block_table"][0, 2]] = 0.0
    r = sd.attend(q, k, v, ref.on_gpu(cache))
    check(r, q, k, v, cache, block, None, [N, N], D ** -0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,G", [(1, 1), (6, 4), (40, 4)])
def test_a_flat_tail_under_a_sink(sd, dtype, N, G):
    """One token with half of the weight and thousands that share the rest: no weight is lost."""
    rng = np.random.default_rng(11)
    n, Hkv, D, block = 5000, 1, 128, 64
    q, k, v = tokens(rng, 1, N, G * Hkv, Hkv, D, dtype)
    q[:] = 1.0
    k[:] = 0.0
    cache = ref.make_cache(rng, [n], [0], block, Hkv, D)
    cache["k"].zero_()
    cache["k_scale"][:] = 2.0 ** -6
    cache["v_scale"][:] = 2.0 ** -6
    cache["k"][cache["block_table"][0, 0], 0, 0] = \
        torch.tensor([48.0]).to(ref.E4M3).view(torch.uint8)   # 0.75 * 128 / sqrt(128) = 8.5
    r = sd.attend(q, k, v, ref.on_gpu(cache))
    check(r, q, k, v, cache, block, None, [N], D ** -0.5)


def test_scores_of_minus_infinity_and_plus_infinity(sd):
    rng = np.random.default_rng(12)
    q, k, v = tokens(rng, 1, 2, 2, 1, 64, torch.bfloat16)
    q[:] = 1.0
    k[0, 0] = float("-inf")      # node 0 sees only a score of -infinity, node 1 itself too
    cache = ref.make_cache(rng, [0], [1], 16, 1, 64)
    r = sd.attend(q, k, v, ref.on_gpu(cache))
    assert (r.out[0, 0] == 0).all() and (r.lse[0, 0] == -math.inf).all()
    assert torch.equal(r.out[0, 1, 0], v[0, 1, 0])
    k[0, 0] = float("inf")
    r = sd.attend(q, k, v, ref.on_gpu(cache))
    assert torch.isnan(r.out[0]).all()


def test_requests_with_errors_give_zeros(sd):
    rng = np.random.default_rng(13)
    lens, N, Hq, Hkv, D, block = [40] * 7, 20, 4, 1, 128, 16
    for dtype in (torch.float32, torch.bfloat16):
        q, k, v = tokens(rng, 7, N, Hq, Hkv, D, dtype)
        parents = torch.tensor([ref.random_tree(rng, N) for _ in lens]).int()
        cache = ref.make_cache(rng, lens, [0] * 7, block, Hkv, D)
        good = {n: t.clone() for n, t in cache.items()}
        cache["block_table"][0, 2] = -1
        cache["block_table"][1, 0] = cache["k"].shape[0]
        cache["length"][2] = -1
        cache["length"][3] = cache["block_table"].shape[1] * block + 1
        parents[4, 5] = 5
        nodes = torch.full((7,), N, dtype=torch.int32)
        nodes[5] = N + 1
        r = sd.attend(q, k, v, ref.on_gpu(cache), parent=parents.cuda(), n_nodes=nodes.cuda())
        assert r.row_status.tolist() == [sd.ROW_BAD_CACHE] * 4 + [sd.ROW_BAD_TREE] * 2 + [0]
        assert (r.out[:6] == 0).all() and (r.lse[:6] == -math.inf).all()
        check(r, q, k, v, good, block, parents.tolist(), [N] * 7, D ** -0.5, skip=range(6))
        r = sd.attend(q, k, v, ref.on_gpu(cache), parent=parents.cuda(), window=4)
        # a bad id outside of every window is not read
        assert r.row_status.tolist()[1] == 0


def test_misaligned_activations_and_outputs(sd):
    """Activations that start on an odd element, and outputs given by the caller."""
    rng = np.random.default_rng(14)
    for dtype in (torch.float32, torch.bfloat16):
        for N, Hq, Hkv, D in ((3, 4, 2, 64), (20, 4, 1, 128)):
            q, k, v = tokens(rng, 2, N, Hq, Hkv, D, dtype, pad=3)
            shift = [torch.empty(t.numel() + 1, dtype=dtype, device="cuda")[1:].view(t.shape).copy_(t)
                     for t in (q, k, v)]
            cache = ref.make_cache(rng, [33, 80], [0, 0], 16, Hkv, D)
            out = sd.AttendOut(torch.empty(q.numel() + 1, dtype=dtype, device="cuda")[1:].view(q.shape),
                               None, torch.empty(2, dtype=torch.int32, device="cuda"))
            want = sd.attend(q, k, v, ref.on_gpu(cache))
            got = sd.attend(*shift, ref.on_gpu(cache), out=out)
            assert got is out and torch.equal(out.out, want.out)
            check(want, q, k, v, cache, 16, None, [N, N], D ** -0.5)


@pytest.mark.parametrize("N,G", [(1, 4), (9, 4), (40, 8)])
def test_pool_past_32_bits(sd, N, G):
    block, Hkv, D = 64, 8, 128
    per = Hkv * block * D
    nb = 2 ** 32 // per + 6
    rng = np.random.default_rng(15)
    small = ref.make_cache(rng, [200], [0], block, Hkv, D, spare=0)
    n = small["k"].shape[0]
    f8 = torch.float8_e4m3fn
    pools = {}
    for name in ("k", "v"):
        pool = torch.zeros(nb, Hkv, block, D, dtype=torch.uint8, device="cuda")
        pool[nb - n:] = small[name].cuda()
        scale = torch.ones(nb, Hkv, device="cuda")
        scale[nb - n:] = small[name + "_scale"].cuda()
        pools[name] = (pool, scale)
    big = sd.KVCache(pools["k"][0].view(f8), pools["v"][0].view(f8), pools["k"][1], pools["v"][1],
                     torch.where(small["block_table"] >= 0, small["block_table"] + nb - n,
                                 -1).int().cuda(), small["length"].cuda())
    q, k, v = tokens(rng, 1, N, Hkv * G, Hkv, D, torch.bfloat16)
    a, b = sd.attend(q, k, v, big), sd.attend(q, k, v, ref.on_gpu(small))
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    check(b, q, k, v, small, block, None, [N], D ** -0.5)


def test_streams_and_graphs(sd):
    """On a side stream with workspaces of its own, and replayed from a graph with new contents."""
    rng = np.random.default_rng(16)
    B, N, Hq, Hkv, D, block = 3, 5, 8, 2, 128, 16
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, torch.bfloat16)
    cache = ref.make_cache(rng, [900, 31, 0], [8] * B, block, Hkv, D)
    gpu = ref.on_gpu(cache)
    want = sd.attend(q, k, v, gpu)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(sd.attend(q, k, v, gpu))
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)
    out, ws = sd.attend(q, k, v, gpu), sd.alloc_attend_workspace(q, gpu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.attend(q, k, v, gpu, out=out, workspace=ws)
    q.mul_(-0.5)
    gpu.length.copy_(torch.tensor([850, 7, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    fresh = sd.attend(q, k, v, gpu)
    assert torch.equal(out.out, fresh.out) and torch.equal(out.lse, fresh.lse)


def test_empty_calls_and_refusals(sd):
    rng = np.random.default_rng(17)
    q, k, v = tokens(rng, 2, 3, 4, 2, 64, torch.float32)
    cache = ref.on_gpu(ref.make_cache(rng, [5, 6], [0, 0], 16, 2, 64))
    assert sd.attend(q[:, :0], k[:, :0], v[:, :0], cache).out.shape == (2, 0, 4, 64)
    with pytest.raises(TypeError):
        sd.attend(q.half(), k.half(), v.half(), cache)
    with pytest.raises(TypeError):
        sd.attend(q, k.bfloat16(), v, cache)
    with pytest.raises(ValueError):
        sd.attend(q, k[:, :, :1], v, cache)
    with pytest.raises(ValueError):
        sd.attend(q, k[:, :2], v[:, :2], cache)
    with pytest.raises(ValueError):
        sd.attend(q[..., :32].contiguous(), k, v, cache)
    with pytest.raises(ValueError):
        sd.attend(q.cpu(), k.cpu(), v.cpu(), cache)
    with pytest.raises(ValueError):
        sd.attend(q, k, v, cache, slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        sd.attend(q, k, v, cache, parent=torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    for bad in (dict(window=-1), dict(softcap=-1.0), dict(softcap=math.nan), dict(scale=math.inf),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(sd.SpecdecError):
            sd.attend(q, k, v, cache, **bad)
    with pytest.raises(sd.SpecdecError):   # three query heads for two of the cache
        sd.attend(q[:, :, :3], k, v, cache)
