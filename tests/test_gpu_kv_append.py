"""Append to the 8-bit paged cache against the definition in 64 bits: codes, scales, lengths and
statuses are equal (a power-of-two scale makes each code one rounding of its value)."""
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


def make(rng, lens, more, block, Hkv, D, N, dtype, spread=1.0, pad=0):
    cache = ref.make_cache(rng, lens, more, block, Hkv, D)
    x = rng.standard_normal((2, len(lens), N, Hkv * D + pad)) * \
        np.exp2(spread * rng.standard_normal((2, len(lens), N, 1)) * 4)
    x = torch.from_numpy(x).to(dtype).cuda()
    k, v = (t[..., :Hkv * D].unflatten(2, (Hkv, D)) for t in x)
    return cache, k, v


def expect(cache, k, v, nodes, block):
    """The state after request b appended nodes[b] (None: nothing)."""
    want = {}
    for name, x in (("k", k), ("v", v)):
        values = cache[name].view(ref.E4M3).double().numpy().copy()
        scale = cache[name + "_scale"].double().numpy().copy()
        for b, ns in enumerate(nodes):
            if ns:
                ref.append(values, scale, x[b].double().cpu().numpy(), ns, int(cache["length"][b]),
                           cache["block_table"][b].tolist(), block)
        want[name], want[name + "_scale"] = values, scale
    return want


def same(gpu, want):
    for name in ("k", "v"):
        got = getattr(gpu, name).double().cpu().numpy()
        assert np.array_equal(got, want[name], equal_nan=True), name
        s = getattr(gpu, name + "_scale").double().cpu().numpy()
        assert np.array_equal(s, want[name + "_scale"]), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block,Hkv,D,N,lens,pad", [
    (16, 1, 16, 1, [0, 1, 15, 16, 17], 0), (16, 3, 48, 9, [0, 7, 8, 31, 100], 0),
    (64, 2, 128, 33, [0, 63, 64, 65, 40], 8), (32, 2, 80, 65, [0, 1, 31, 33, 64], 1),
    (128, 1, 256, 200, [5, 0, 127], 0), (16, 2, 64, 130, [0, 3, 16], 0),
    (1024, 1, 32, 70, [1000, 3], 0)])
def test_append_whole_prompts(sd, dtype, block, Hkv, D, N, lens, pad):
    rng = np.random.default_rng(block + D + N)
    cache, k, v = make(rng, lens, [N] * len(lens), block, Hkv, D, N, dtype, pad=pad)
    gpu = ref.on_gpu(cache)
    want = expect(cache, k, v, [list(range(N))] * len(lens), block)
    for _ in range(2):   # twice on the same state: the same result
        r = sd.kv_append(k, v, gpu)
        same(gpu, want)
        assert r.length.tolist() == [n + N for n in lens] and r.row_status.tolist() == [0] * len(lens)
    assert gpu.length.tolist() == lens


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_counts_and_paths(sd, dtype):
    rng = np.random.default_rng(1)
    N, block, Hkv, D = 64, 16, 2, 64
    lens = [0, 15, 16, 30, 100, 7]
    acc = [0, 5, 3, -1, 2, 1]
    parents = [ref.random_tree(rng, N) for _ in lens]
    paths = []
    for b in range(len(lens)):
        n = max(range(N), key=lambda i: len(ref.ancestors(parents[b], i)))
        up = ref.ancestors(parents[b], n)[::-1]
        paths.append((up + [-1] * 6)[:6])
    for path in (None, paths):
        cache, k, v = make(rng, lens, [8] * len(lens), block, Hkv, D, N, dtype)
        gpu = ref.on_gpu(cache)
        nodes = [(list(range(N)) if path is None else path[b])[:acc[b] + 1] for b in range(len(lens))]
        r = sd.kv_append(k, v, gpu, count=torch.tensor(acc, dtype=torch.int32).cuda(), extra=1,
                         path=None if path is None else torch.tensor(path, dtype=torch.int32).cuda())
        same(gpu, expect(cache, k, v, nodes, block))
        assert r.length.tolist() == [n + a + 1 for n, a in zip(lens, acc)]
        assert r.row_status.tolist() == [0] * len(lens)


def test_scales_at_their_edges(sd):
    """Values at 448 * 2^k and one step past it, zeros, tiny and huge ones, non-finite ones."""
    block, Hkv, D = 16, 1, 16
    tops = [448.0, np.nextafter(np.float32(448.0), np.float32(1e9)), 447.9, 1e-38, 1e-45, 0.0,
            3.4e38, 448.0 * 2.0 ** -100, 448.0 * 2.0 ** -99, 1.0]
    B = len(tops)
    rng = np.random.default_rng(2)
    cache = ref.make_cache(rng, [0] * B, [4] * B, block, Hkv, D)
    x = np.zeros((B, 4, 1, D), dtype=np.float32)
    for b, t in enumerate(tops):
        x[b] = np.float32(t) * rng.uniform(-1, 1, (4, 1, D)).astype(np.float32)
        x[b, 2, 0, 5] = np.float32(t)
    x[-1, 0, 0, 0], x[-1, 1, 0, 1], x[-1, 3, 0, 2] = np.nan, np.inf, -np.inf
    k = torch.from_numpy(x).cuda()
    gpu = ref.on_gpu(cache)
    sd.kv_append(k, k, gpu)
    same(gpu, expect(cache, k, k, [[0, 1, 2, 3]] * B, block))


def test_growing_scale_recodes_what_stands_before(sd):
    """Token by token, each 4 times the last: the old codes lose bits step by step, as defined."""
    rng = np.random.default_rng(4)
    block, Hkv, D = 16, 2, 32
    for scales in ("pow2", "any"):
        cache = ref.make_cache(rng, [3], [12], block, Hkv, D, scales=scales)
        gpu = ref.on_gpu(cache)
        for step in range(9):
            x = rng.standard_normal((1, 1, Hkv, D)) * 4.0 ** step * 2.0 ** -6
            k = torch.from_numpy(x).to(torch.bfloat16).cuda()
            n = int(gpu.length[0])
            want = {}
            for name in ("k", "v"):
                values = getattr(gpu, name).cpu().double().numpy()
                scale = getattr(gpu, name + "_scale").cpu().double().numpy()
                ref.append(values, scale, k[0].double().cpu().numpy(), [0], n,
                           cache["block_table"][0].tolist(), block)
                want[name], want[name + "_scale"] = values, scale
            r = sd.kv_append(k, k, gpu)
            if scales == "pow2":
                same(gpu, want)
            else:   # a scale of another kind: codes are rounded through one more product
                for name in ("k", "v"):
                    assert np.allclose(getattr(gpu, name).cpu().double().numpy(), want[name],
                                       rtol=0.13, atol=2.0 ** -9, equal_nan=True)
            gpu.length = r.length


def test_requests_with_errors_append_nothing(sd):
    rng = np.random.default_rng(6)
    block, Hkv, D, N = 16, 1, 32, 5
    lens = [20, 20, 20, 20, 20, 20]
    cache, k, v = make(rng, lens, [8] * 6, block, Hkv, D, N, torch.float32)
    cache["block_table"][1, 1] = cache["k"].shape[0]      # a block id past the pool
    cache["length"][2] = -1
    path = torch.tensor([[0, 1, 2, 3, 4]] * 6, dtype=torch.int32)
    path[3, 2] = 5                                        # a node past N
    count = torch.tensor([4, 4, 4, 4, 5, 4], dtype=torch.int32)   # request 4: one too many
    gpu = ref.on_gpu(cache)
    before = {n: getattr(gpu, n).clone() for n in ("k", "v", "k_scale", "v_scale")}
    r = sd.kv_append(k, v, gpu, count=count.cuda(), extra=1, path=path.cuda())
    assert r.row_status.tolist() == [0, sd.ROW_BAD_CACHE, sd.ROW_BAD_CACHE, sd.ROW_BAD_TREE,
                                     sd.ROW_BAD_CACHE, 0]
    assert r.length.tolist() == [25, 20, -1, 20, 20, 25]
    good = [0, 5]
    nodes = [list(range(5)) if b in good else None for b in range(6)]
    same(gpu, expect({**cache, "k": before["k"].cpu().view(torch.uint8),
                      "v": before["v"].cpu().view(torch.uint8)}, k, v, nodes, block))


def test_pool_past_32_bits(sd):
    """Blocks whose codes start beyond 2^32 elements."""
    block, Hkv, D = 64, 8, 128
    per = Hkv * block * D
    nb = 2 ** 32 // per + 3
    f8 = torch.float8_e4m3fn
    pool = [torch.zeros(nb, Hkv, block, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ones = torch.ones(nb, Hkv, device="cuda")
    cache = sd.KVCache(pool[0].view(f8), pool[1].view(f8), ones.clone(), ones.clone(),
                       torch.tensor([[nb - 1, nb - 2]], dtype=torch.int32).cuda(),
                       torch.tensor([60], dtype=torch.int32).cuda())
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k = torch.randn(1, 10, Hkv, D, generator=g, device="cuda")
    v = torch.randn(1, 10, Hkv, D, generator=g, device="cuda")
    r = sd.kv_append(k, v, cache)
    assert r.length.tolist() == [70]
    for x, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        got = torch.cat((codes[nb - 1, :, 60:].float() * scale[nb - 1][:, None, None],
                         codes[nb - 2, :, :6].float() * scale[nb - 2][:, None, None]), 1)
        want = x[0].transpose(0, 1)
        assert ((got - want).abs() <= want.abs() * 2.0 ** -4 + scale[nb - 1].max() * 2.0 ** -10).all()
        assert not codes.view(torch.uint8)[:4].any()


def test_refusals(sd):
    rng = np.random.default_rng(8)
    cache = ref.on_gpu(ref.make_cache(rng, [3, 4], [4, 4], 16, 2, 32))
    x = torch.zeros(2, 4, 2, 32, device="cuda")
    with pytest.raises(TypeError):
        sd.kv_append(x.half(), x.half(), cache)
    with pytest.raises(TypeError):
        sd.kv_append(x, x.bfloat16(), cache)
    with pytest.raises(ValueError):
        sd.kv_append(x[:, :, :1], x, cache)
    with pytest.raises(ValueError):
        sd.kv_append(x[:1], x[:1], cache)
    with pytest.raises(ValueError):
        sd.kv_append(x, x, cache, count=torch.zeros(3, dtype=torch.int32).cuda())
    with pytest.raises(TypeError):
        sd.kv_append(x, x, cache, count=torch.zeros(2).cuda())
    with pytest.raises(ValueError):
        sd.kv_append(x.cpu(), x.cpu(), cache)
    with pytest.raises(sd.SpecdecError):   # the new length over the old one
        sd.kv_append(x, x, cache, out=sd.AppendOut(cache.length, torch.zeros_like(cache.length)))
    r = sd.kv_append(x[:, :0], x[:, :0], cache)
    assert r.length.tolist() == [3, 4] and r.row_status.tolist() == [0, 0]
