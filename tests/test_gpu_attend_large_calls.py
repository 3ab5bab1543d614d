"""The kernel that large bfloat16 attention calls take: requests with errors, other streams and
graphs.  Contexts are long enough that a request's tiles are cut into parts of several CTAs, which a
second kernel joins, flags among them."""
import math

import numpy as np
import pytest

import attention_oracle as ref
from test_gpu_attend import check, tokens

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("N,Hq,Hkv,D", [(20, 8, 2, 128), (3, 8, 2, 64), (9, 8, 2, 128), (70, 4, 2, 96)])
@pytest.mark.parametrize("window", [0, 2500])
def test_requests_with_errors_give_zeros(sd, N, Hq, Hkv, D, window):
    rng = np.random.default_rng(N)
    lens, block = [5000, 4000, 300, 40, 4500, 3000, 4800, 5000, 17, 0], 16
    B = len(lens)
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, torch.bfloat16)
    parents = torch.tensor([ref.random_tree(rng, N) for _ in lens]).int()
    cache = ref.make_cache(rng, lens, [0] * B, block, Hkv, D)
    good = {n: t.clone() for n, t in cache.items()}
    cache["block_table"][0, 270] = -1                             # late in the request
    cache["block_table"][1, 249] = cache["k"].shape[0]            # its last block
    cache["length"][2] = -1
    cache["length"][3] = cache["block_table"].shape[1] * block + 1
    parents[4, N - 1] = N - 1
    nodes = torch.full((B,), N, dtype=torch.int32)
    nodes[5] = N + 1
    cache["block_table"][6, 299] = 2 ** 31 - 1                    # two errors, in one part and
    cache["block_table"][6, 150] = -2 ** 31                       # in several
    parents[6, 1] = -1
    r = sd.attend(q, k, v, ref.on_gpu(cache), parent=parents.cuda(), n_nodes=nodes.cuda(), window=window)
    assert r.row_status.tolist() == [sd.ROW_BAD_CACHE] * 4 + [sd.ROW_BAD_TREE] * 2 + \
        [sd.ROW_BAD_CACHE | sd.ROW_BAD_TREE] + [0] * 3
    assert (r.out[:7] == 0).all() and (r.lse[:7] == -math.inf).all()
    check(r, q, k, v, good, block, parents.tolist(), [N] * B, D ** -0.5, window=window, skip=range(7))


def test_block_ids_before_every_window_are_not_read(sd):
    rng = np.random.default_rng(1)
    B, N, Hq, Hkv, D, block = 20, 3, 8, 8, 64, 16
    lens = [int(n) for n in rng.integers(1500, 4000, B)]
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, torch.bfloat16)
    cache = ref.make_cache(rng, lens, [0] * B, block, Hkv, D)
    good = {n: t.clone() for n, t in cache.items()}
    window = 700
    for b, n in enumerate(lens):
        cache["block_table"][b, :(n - window + 1) // block] = -1
    r = sd.attend(q, k, v, ref.on_gpu(cache), window=window)
    check(r, q, k, v, good, block, None, [N] * B, D ** -0.5, window=window)
    for b, n in enumerate(lens):   # one more block is read
        cache["block_table"][b, (n - window + 1) // block] = -1
    r = sd.attend(q, k, v, ref.on_gpu(cache), window=window)
    assert (r.row_status == sd.ROW_BAD_CACHE).all() and (r.out == 0).all()


def test_streams_and_graphs(sd):
    rng = np.random.default_rng(2)
    B, N, Hq, Hkv, D, block = 4, 5, 8, 2, 128, 16
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, torch.bfloat16)
    cache = ref.make_cache(rng, [9000, 310, 0, 2500], [8] * B, block, Hkv, D)
    gpu = ref.on_gpu(cache)
    want = sd.attend(q, k, v, gpu)
    check(want, q, k, v, cache, block, None, [N] * B, D ** -0.5)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        s.wait_stream(torch.cuda.current_stream())
        got += [sd.attend(q, k, v, gpu, stream=s) for _ in range(4)]
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)
    # one workspace for calls in a row and for a graph, whatever stands in it
    out, ws = sd.attend(q, k, v, gpu), sd.alloc_attend_workspace(q, gpu)
    ws.fill_(255)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.attend(q, k, v, gpu, out=out, workspace=ws)
    for lens in ([8500, 7, 0, 2300], [0, 1, 0, 0], [9000, 310, 0, 2500]):
        q.mul_(-0.5)
        gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        fresh = sd.attend(q, k, v, gpu)
        assert torch.equal(out.out, fresh.out) and torch.equal(out.lse, fresh.lse)
        assert (out.row_status == 0).all()
        cache["length"] = torch.tensor(lens, dtype=torch.int32)
        check(fresh, q, k, v, cache, block, None, [N] * B, D ** -0.5)


def chain(q, k_new, v_new, k, v, scale, window):
    """One request's chain in float64, all rows at once: out and the largest scale * sum |q| |k|."""
    (N, Hq, D), G = q.shape, q.shape[1] // k_new.shape[1]
    keys, vals = (torch.cat(x).double().repeat_interleave(G, 1) for x in ((k, k_new), (v, v_new)))
    n = k.shape[0]
    dist = n + torch.arange(N, device=q.device)[:, None] - torch.arange(n + N, device=q.device)
    seen = (dist >= 0) & ((dist < window) if window else True)
    s = torch.einsum("nhd,jhd->hnj", q.double(), keys) * scale
    S = (torch.einsum("nhd,jhd->hnj", q.double().abs(), keys.abs()) * scale).amax()
    p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
    # (a hidden value has no part, finite or not)
    out = torch.einsum("hnj,jhd->nhd", p, vals.nan_to_num(0.0))
    bad = torch.einsum("nj,jhd->nhd", seen.double(), (~torch.isfinite(vals)).double()) > 0
    return torch.where(bad, math.nan, out), torch.einsum("hnj,jhd->nhd", p, vals.abs().nan_to_num(0.0)), S


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window,nan", [(0, False), (700, False), (700, True)])
def test_the_longest_chunk_of_a_prompt(sd, dtype, window, nan):
    """1024 nodes.  With v that is not finite in a drafted node and in tokens that the window hides
    from some: each result looks for them one by one, which takes its time but is no error."""
    rng = np.random.default_rng(3)
    N, Hq, Hkv, D, block, n = 1024, 4, 2, 64, 16, 1500
    q, k, v = tokens(rng, 1, N, Hq, Hkv, D, dtype)
    cache = ref.make_cache(rng, [n], [0], block, Hkv, D)
    if nan:
        v[0, 300, 1, 7] = math.inf
        for j in (n - 650, n - 100):
            cache["v"][cache["block_table"][0, j // block], 0, j % block, 3] = 0x7F
    kc, vc = (ref.cached_values(cache, x, 0, block).cuda() for x in ("k", "v"))
    gpu = ref.on_gpu(cache)
    more = torch.full((1, 2500), -1, dtype=torch.int32, device="cuda")
    gpu.block_table = torch.cat([gpu.block_table, more], 1)   # room for a large call
    r = sd.attend(q, k, v, gpu, window=window)
    assert r.row_status.tolist() == [0]
    want, A, S = chain(q[0], k[0], v[0], kc, vc, D ** -0.5, window)
    # (the tolerance of test_gpu_attend.py with the largest S for all rows)
    tol = A * (2 * 2.0 ** (-19 if dtype == torch.float32 else -16) * (1 + S) +
               2 * 2.0 ** (-21 if dtype == torch.float32 else -11))
    if dtype == torch.bfloat16:
        tol = tol + want.abs().nan_to_num(0.0) * 2.0 ** -8
    got, fine = r.out[0].double(), torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine)
    assert ((got - want).abs()[fine] <= tol[fine]).all()
