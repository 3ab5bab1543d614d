"""Attention of drafted tokens where its inputs are unusual: against the formula in 64 bits, on each
way that a call can take (the streaming kernel with its splits joined in a cluster and through the
workspace, and the tensor-core kernel).

Tolerance, with p the weights of a row, S the largest scale * sum |q| |k| of it and Q the largest
scale * (max |q| sum |k| + max |k| sum |q|):
  * a score is off by at most 2^-19 (1 + S) for float32 activations (two fp16 terms an operand);
    for bfloat16 ones by 2^-16 (1 + S) + 2^-17 Q: q and the drafted k are two e4m3 terms in units of
    their largest element, in [2^7, 2^8), so what they leave is at most half of e4m3's smallest
    step, 2^-10, which is 2^-17 of that element;
  * a cap adds no more than 2^-20 of the score itself;
  * weights carry 2^-11 of themselves (2^-21 in two terms), and as fp16 numbers at least 2^-25 where
    the row's largest contribution stands at 2^5 or above: with U the largest size that a token's
    unit can carry (448 scales, twice a drafted token's largest element), n 2^-30 max(p U) in all.
    |out error| <= (sum p |v| (2 ds + 2 dw) + n 2^-30 max(p U)) / sum p  (+ 2^-8 |out| in bfloat16)
    |lse error| <= ds + 2^-20 (1 + |lse|)
"""
import math

import numpy as np
import pytest

import attention_oracle as ref
from test_gpu_attend import tokens
from test_gpu_attend_tiles import Large

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

F32, BF16 = torch.float32, torch.bfloat16
WAYS = [pytest.param(d, w, id=f"{n}-{i}") for d, n in ((F32, "f32"), (BF16, "bf16"))
        for w, i in ((False, "small"), (True, "large"))]
ways = pytest.mark.parametrize("dtype,large", WAYS)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def on(lib, large):
    """The binding, or the binding with the call made large (see test_gpu_attend_tiles.py)."""
    return Large(lib) if large else lib


def expected(q, k_new, v_new, parent, k, v, v_unit, length, scale, softcap=0.0, window=0):
    """One request in float64; v_unit [length, Hkv]: 448 times the scale of each cached token.
    Returns out, lse, sum p |v| / sum p, S, Q and n max(p U) / sum p."""
    N, Hq, D = q.shape
    G = Hq // k_new.shape[1]
    out, mag, floor = (torch.zeros(N, Hq, D, dtype=torch.float64) for _ in range(3))
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64)
    S, Q = torch.zeros(N, Hq, dtype=torch.float64), torch.zeros(N, Hq, dtype=torch.float64)
    for n in range(N):
        up = ref.ancestors(parent, n)
        where = length + len(up) - 1
        dist = [where - j for j in range(length)] + list(range(len(up)))
        keep = [i for i, d in enumerate(dist) if window == 0 or d < window]
        keys = torch.cat((k, k_new[up]))[keep]
        vals = torch.cat((v, v_new[up]))[keep]
        units = torch.cat((v_unit, 2 * v_new[up].abs().amax(-1)))[keep]
        for h in range(Hq):
            kk, vv, uu = keys[:, h // G], vals[:, h // G], units[:, h // G]
            a, b = kk.abs().nan_to_num(0, 0, 0), q[n, h].abs().nan_to_num(0, 0, 0)
            S[n, h] = (a @ b).max() * abs(scale)
            Q[n, h] = (a.sum(-1) * b.max() + a.amax(-1) * b.sum()).max() * abs(scale)
            s = kk @ q[n, h] * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if float(s.max()) == -math.inf:
                continue
            p = torch.exp(s - s.max())
            lse[n, h] = torch.log(p.sum()) + s.max()
            out[n, h] = (p / p.sum()) @ vv
            mag[n, h] = (p / p.sum()) @ vv.abs()
            floor[n, h] = len(keep) * float((p / p.sum() * uu).max())
    return out, lse, mag, S, Q, floor


def check(r, q, k, v, cache, block, parents, scale, **how):
    f32 = q.dtype == F32
    got, lse = r.out.double().cpu(), r.lse.double().cpu()
    for b in range(q.shape[0]):
        kc, vc = (ref.cached_values(cache, n, b, block) for n in ("k", "v"))
        n = int(cache["length"][b])
        ids = cache["block_table"][b, :-(-n // block)].long()
        unit = 448 * cache["v_scale"][ids].double().repeat_interleave(block, 0)[:n]
        want, wl, A, S, Q, floor = expected(
            q[b].double().cpu(), k[b].double().cpu(), v[b].double().cpu(),
            None if parents is None else parents[b], kc, vc, unit, n, scale, **how)
        ds = 2.0 ** (-19 if f32 else -16) * (1 + S) + (0 if f32 else 2.0 ** -17) * Q + \
            (2.0 ** -20 * S if how.get("softcap") else 0)
        dw = 2.0 ** (-21 if f32 else -11)
        tol = A * (2 * ds + 2 * dw)[..., None] + 2.0 ** -30 * floor
        if not f32:
            tol = tol + want.abs() * 2.0 ** -8
        assert torch.equal(torch.isnan(lse[b]), torch.isnan(wl)), b
        empty = wl == -math.inf
        assert (got[b][empty] == 0).all() and (lse[b][empty] == -math.inf).all(), b
        bad = ~torch.isfinite(want)
        assert torch.equal(torch.isfinite(got[b]), ~bad), b
        err = torch.where(bad, 0.0, (got[b] - want).abs())
        assert (err <= torch.where(bad, 1.0, tol)).all(), \
            (b, float((err - tol).nan_to_num(-1).max()), float(err.max()))
        ok = torch.isfinite(wl)
        assert ((lse[b] - wl).abs()[ok] <= (ds + 2.0 ** -20 * (1 + wl.abs()))[ok]).all(), b
    assert (r.row_status.cpu() == 0).all()


# ---- scores that are not a number ----

@ways
@pytest.mark.parametrize("Hkv,D", [(2, 128), (1, 64)])
def test_a_query_that_is_not_a_number(lib, dtype, large, Hkv, D):
    """Its row is NaN, in out and in lse, and no other row."""
    rng = np.random.default_rng(1)
    lens, N, Hq, block = [40, 0, 17], 3, 4 * Hkv, 16
    q, k, v = tokens(rng, 3, N, Hq, Hkv, D, dtype)
    q[0, 1, 2, 5] = q[1, 0, 0, 0] = q[2, 2, 3, D - 1] = float("nan")
    cache = ref.make_cache(rng, lens, [0] * 3, block, Hkv, D)
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache))
    check(r, q, k, v, cache, block, None, D ** -0.5)
    assert torch.isnan(r.out[0, 1, 2]).all() and torch.isnan(r.lse[1, 0, 0])


@ways
@pytest.mark.parametrize("lens", [[64, 0, 33], [1, 16, 500]])
def test_a_lone_drafted_key_that_is_not_a_number(lib, dtype, large, lens):
    rng = np.random.default_rng(2)
    q, k, v = tokens(rng, 3, 1, 4, 2, 128, dtype)
    k[:, 0, 1, 7] = float("nan")
    cache = ref.make_cache(rng, lens, [0] * 3, 16, 2, 128)
    check(on(lib, large).attend(q, k, v, ref.on_gpu(cache)), q, k, v, cache, 16, None, 128 ** -0.5)


@ways
@pytest.mark.parametrize("scale", [0.0884, 4.0])
@pytest.mark.parametrize("at", ["last", "first"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_cached_key_that_is_not_a_number(lib, dtype, large, scale, at, D):
    """Alone in its granule of 16 tokens, also where all other scores are far above or below 0, so
    that its part of the sums comes under a factor of 0."""
    rng = np.random.default_rng(3)
    lens, N, block = [33, 17, 1, 65, 529], 2, 16
    q, k, v = tokens(rng, len(lens), N, 2, 1, D, dtype)
    cache = ref.make_cache(rng, lens, [0] * len(lens), block, 1, D)
    for b, n in enumerate(lens):
        j = n - 1 if at == "last" else 0
        cache["k"][cache["block_table"][b, j // block], 0, j % block, 11] = 0x7F
    check(on(lib, large).attend(q, k, v, ref.on_gpu(cache), scale=scale), q, k, v, cache, block,
          None, scale)


@ways
@pytest.mark.parametrize("scale", [0.0884, -0.0884, 0.0])
@pytest.mark.parametrize("N,D", [(1, 128), (7, 64), (7, 128), (40, 128)])
def test_infinite_drafted_keys(lib, dtype, large, scale, N, D):
    """By the formula: scores of infinity, which make NaN, or of -infinity, which leave their token
    out, or NaN where the query's element is 0."""
    rng = np.random.default_rng(10)
    lens, Hq, Hkv, block = [0, 17, 33], 4, 2, 16
    parents = [ref.random_tree(rng, N) for _ in lens]
    q, k, v = tokens(rng, 3, N, Hq, Hkv, D, dtype)
    k[0, 0, 0, 3], k[1, N - 1, 1, 5], k[2, N // 2, 0, D - 1] = math.inf, -math.inf, math.inf
    k[2, 0, 1, 0], k[2, 0, 1, 1], q[2, 0, 3, 0] = math.inf, -math.inf, 0
    q[0, :, :2, 3] = -q[0, :, :2, 3].abs()     # all see node 0: -infinity there, or infinity
    cache = ref.make_cache(rng, lens, [0] * 3, block, Hkv, D)
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache), parent=torch.tensor(parents).int().cuda(),
                              scale=scale)
    check(r, q, k, v, cache, block, parents, scale)


@ways
@pytest.mark.parametrize("size", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_a_query_that_is_not_finite_makes_its_row_nan(lib, dtype, large, size, softcap):
    """Whatever its scores would be; a row that sees nothing stays empty."""
    rng = np.random.default_rng(11)
    B, N, Hq, Hkv, D, block = 3, 6, 4, 2, 128, 16
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, dtype)
    q[0, 0, 1, 7] = q[1, 5, 3, 0] = q[2, 4, 2, 100] = size
    cache = ref.make_cache(rng, [0, 40, 0], [0] * B, block, Hkv, D)
    nodes = torch.tensor([6, 6, 4], dtype=torch.int32).cuda()
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache), n_nodes=nodes, softcap=softcap)
    for bad in ((0, 0, 1), (1, 5, 3)):
        assert torch.isnan(r.out[bad]).all() and torch.isnan(r.lse[bad])
    assert (r.out[2, 4:] == 0).all() and (r.lse[2, 4:] == -math.inf).all()
    nan = torch.isnan(r.lse).cpu()
    assert int(nan.sum()) == 2 and torch.isfinite(r.out[~nan]).all()


@ways
@pytest.mark.parametrize("N,D", [(1, 128), (6, 64), (40, 128)])
def test_a_score_of_minus_infinity_leaves_its_token_out(lib, dtype, large, N, D):
    """Also where its v is not finite: the result is that of a token with any other v."""
    rng = np.random.default_rng(13)
    lens, Hq, Hkv, block = [17, 40], 4, 2, 16
    q, k, v = tokens(rng, 2, N, Hq, Hkv, D, dtype)
    parents = [ref.random_tree(rng, N) for _ in lens]
    cache = ref.make_cache(rng, lens, [0] * 2, block, Hkv, D)
    q[:, :, :, 1] = q[:, :, :, 1].abs() + 0.5
    k[0, 0, 0, 1] = k[1, N - 1, 1, 1] = -math.inf
    how = dict(parent=torch.tensor(parents).int().cuda())
    want = on(lib, large).attend(q, k, v, ref.on_gpu(cache), **how)
    check(want, q, k, v, cache, block, parents, D ** -0.5)
    v[0, 0, 0, 3], v[0, 0, 0, 4], v[1, N - 1, 1, D - 1] = math.inf, math.nan, -math.inf
    got = on(lib, large).attend(q, k, v, ref.on_gpu(cache), **how)
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


# ---- heads of any size ----

@ways
@pytest.mark.parametrize("D", [16, 32, 48, 112, 128, 144, 160, 240, 256])
@pytest.mark.parametrize("N", [1, 9])
def test_heads_of_every_width_over_many_splits(lib, dtype, large, D, N):
    """The join of splits takes 128 elements at a time, of which the last may be 16 only."""
    rng = np.random.default_rng(12)
    lens, Hq, Hkv, block = [897, 17, 400], 2, 1, 48
    q, k, v = tokens(rng, 3, N, Hq, Hkv, D, dtype)
    cache = ref.make_cache(rng, lens, [0] * 3, block, Hkv, D)
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache))
    check(r, q, k, v, cache, block, None, D ** -0.5)


# ---- windows of any size ----

@ways
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 17, 2 ** 30])
def test_a_window_past_every_length_changes_nothing(lib, dtype, large, window):
    rng = np.random.default_rng(9)
    lens, N, Hq, Hkv, D, block = [3000, 700], 5, 8, 2, 128, 16
    q, k, v = tokens(rng, 2, N, Hq, Hkv, D, dtype)
    cache = ref.make_cache(rng, lens, [0] * 2, block, Hkv, D)
    if large:   # room for many more tokens
        cache["block_table"] = torch.cat([cache["block_table"],
                                          torch.full((2, 2500), -1, dtype=torch.int32)], 1)
    a, b = (lib.attend(q, k, v, ref.on_gpu(cache), window=w) for w in (0, window))
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    check(b, q, k, v, cache, block, None, D ** -0.5)


# ---- caps of any size ----

@ways
@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 0.5, 12.0, 30.0, 50.0, 1e4, 1e6, 1e7, 1e8, 1e20,
                                     3e38])
def test_caps_of_any_size(lib, dtype, large, softcap):
    rng = np.random.default_rng(4)
    lens, N, Hq, Hkv, D, block = [50, 0, 131], 5, 4, 2, 128, 16
    q, k, v = tokens(rng, 3, N, Hq, Hkv, D, dtype)
    q[0, 0] = 0
    cache = ref.make_cache(rng, lens, [0] * 3, block, Hkv, D)
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache), softcap=softcap)
    check(r, q, k, v, cache, block, None, D ** -0.5, softcap=softcap)


# ---- values of any size, seen or not ----

@ways
@pytest.mark.parametrize("size", [1e6, 1e9, 1e12, 1e30, 1e38, 1e-30])
@pytest.mark.parametrize("N,Hkv,D", [(24, 2, 128), (9, 1, 64)])
def test_a_drafted_value_of_any_size(lib, dtype, large, size, N, Hkv, D):
    """Leaves of a tree whose v is huge, or tiny, do nothing to the rows that do not see them."""
    rng = np.random.default_rng(5)
    lens, block = [0, 47, 300], 16
    parents = [ref.random_tree(rng, N) for _ in lens]
    q, k, v = tokens(rng, 3, N, 4 * Hkv, Hkv, D, dtype)
    for b in range(3):
        leaves = [n for n in range(N) if n not in parents[b]]
        v[b, leaves[0]] *= size
        v[b, leaves[-1]] *= size / 1e3
        v[b, parents[b][leaves[1]]] *= size ** 0.25
    cache = ref.make_cache(rng, lens, [0] * 3, block, Hkv, D)
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache), parent=torch.tensor(parents).int().cuda())
    check(r, q, k, v, cache, block, parents, D ** -0.5)


@ways
@pytest.mark.parametrize("fall", [0.0, 20.0, 60.0, 80.0])
@pytest.mark.parametrize("size", [1e30, 1e-30])
@pytest.mark.parametrize("D", [64, 128])
def test_a_visible_block_of_any_size(lib, dtype, large, fall, size, D):
    """A cached block whose v are 1e30 times the others', under scores `fall` below theirs: it takes
    part by its weight times its size, be that nothing or all."""
    rng = np.random.default_rng(6)
    lens, N, block = [160, 700], 3, 32
    q, k, v = tokens(rng, 2, N, 2, 1, D, dtype)
    q[:] = 1.0
    k *= 0.125
    cache = ref.make_cache(rng, lens, [0] * 2, block, 1, D)
    cache["k_scale"][:] = 2.0 ** -9
    for b, n in enumerate(lens):
        for i in (1, n // block - 1):
            at = cache["block_table"][b, i]
            cache["v_scale"][at] *= size
            code = torch.tensor([-fall / D / 0.125 * 2.0 ** 4]).to(ref.E4M3).view(torch.uint8)
            cache["k"][at] = code
            cache["k_scale"][at] = 2.0 ** -4
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache), scale=0.125)
    check(r, q, k, v, cache, block, None, 0.125)


@ways
@pytest.mark.parametrize("window", [20, 60])
def test_a_block_of_any_size_outside_of_windows(lib, dtype, large, window):
    """Huge blocks that a window hides from some nodes of a long chain, or from all."""
    rng = np.random.default_rng(7)
    lens, N, D, block = [100, 131], 40, 64, 16
    q, k, v = tokens(rng, 2, N, 2, 1, D, dtype)
    cache = ref.make_cache(rng, lens, [0] * 2, block, 1, D)
    for b, n in enumerate(lens):
        cache["v_scale"][cache["block_table"][b, (n - window + 20) // block]] *= 1e25
        cache["v_scale"][cache["block_table"][b, (n - window) // block]] *= 1e12
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache), window=window)
    check(r, q, k, v, cache, block, None, D ** -0.5, window=window)


@ways
def test_block_scales_of_every_size(lib, dtype, large):
    rng = np.random.default_rng(8)
    lens, N, Hq, Hkv, D, block = [333, 1000], 4, 4, 2, 128, 16
    q, k, v = tokens(rng, 2, N, Hq, Hkv, D, dtype)
    cache = ref.make_cache(rng, lens, [0] * 2, block, Hkv, D)
    nb = cache["k"].shape[0]
    cache["v_scale"] = torch.from_numpy(10.0 ** rng.uniform(-36, 35, (nb, Hkv))).float()
    cache["v_scale"][::9] = 0.0
    r = on(lib, large).attend(q, k, v, ref.on_gpu(cache))
    check(r, q, k, v, cache, block, None, D ** -0.5)
