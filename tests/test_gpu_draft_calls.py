"""The draft side's calls in a program: other streams, captured graphs, two at once, under autograd in
a graph, and their bounded waits."""
import contextlib

import numpy as np
import pytest

from test_gpu_distill import cuda, teacher
from test_gpu_sample import floats, ints, normal, on_gpu, uniforms

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def case(sd, seed=1, B=6, R=2, V=20011, dtype="bf16"):
    x = on_gpu(normal(seed, B, R, V), dtype)
    u = torch.from_numpy(uniforms(np.random.default_rng(seed), (B, R, 2))).cuda()
    T = floats([1.0, 0.7, 0.0, 1.3, 0.5, 0.9][:B])
    k, p, m = ints([0, 40, 0, 900, 0, 7][:B]), floats([0.9, 0.8, 1.0, 0.95, 1.0, 1.0][:B]), floats([0.0, 0.0, 0.0, 0.01, 0.1, 0.0][:B])
    ids, z, lse = (cuda(a) for a in teacher(seed, x.double().cpu().numpy(), 30, 1.0, True))
    return dict(x=x, u=u, T=T, k=k, p=p, m=m, ids=ids, z=z, lse=lse)


def calls(sd, c):
    return {
        "sample": lambda **kw: sd.sample(c["x"], c["T"], c["u"], c["k"], c["p"], c["m"], **kw),
        "filter": lambda **kw: sd.filter_logits(c["x"], c["T"], c["k"], c["p"], c["m"], **kw),
        "top": lambda **kw: sd.top_logits(c["x"], 50, **kw),
        "distill": lambda **kw: sd.distill(c["x"], c["ids"], c["z"], c["lse"], **kw),
    }


def same(a, b):
    for n, v in vars(a).items():
        w = getattr(b, n)
        assert (v is None and w is None) or torch.equal(v, w), n


@pytest.mark.parametrize("name", ["sample", "filter", "top", "distill"])
def test_on_another_stream(sd, name):
    c = case(sd)
    call = calls(sd, c)[name]
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            x @ x
    got = call(stream=s)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            for n in (1 << 22, 1 << 20, 1 << 16, 1 << 12) for _ in range(4)]
    torch.cuda.synchronize()
    same(got, want)
    del junk


def test_two_at_once(sd):
    """Two batches on two streams, each several times, with nothing between them."""
    cs = [case(sd, seed) for seed in (3, 4)]
    want = [{n: f() for n, f in calls(sd, c).items()} for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(5):
        for i, c in enumerate(cs):
            got[i].append({n: f(stream=streams[i]) for n, f in calls(sd, c).items()})
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for n in r:
                same(r[n], want[i][n])


def test_in_captured_graphs(sd):
    """Captured calls take the inputs that stand there when they are replayed; two graphs that share a
    workspace run one after the other."""
    c, other = case(sd, 5), case(sd, 6)
    ws = torch.empty(sd.top_logits_workspace_size(6, 2, 20011, sd.BF16), dtype=torch.uint8, device="cuda")
    fs = calls(sd, c)
    fs["top"] = lambda **kw: sd.top_logits(c["x"], 50, workspace=ws, **kw)
    for f in fs.values():
        f()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append({n: f() for n, f in fs.items()})
        graphs.append(g)
    for n in c:
        c[n].copy_(other[n])
    want = {n: f() for n, f in calls(sd, other).items()}
    ws.fill_(255)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        for n in o:
            same(o[n], want[n])


def test_a_training_step_in_a_graph(sd):
    """Loss and gradient captured, in their own graph's leaf, replayed on other logits."""
    c, other = case(sd, 7, dtype="f32"), case(sd, 8, dtype="f32")
    w = torch.rand(6, 2, generator=torch.Generator().manual_seed(1)).cuda()
    leaf = c["x"].clone().requires_grad_(True)

    def step(x, c):
        return torch.autograd.grad(sd.distill_loss(x, c["ids"], c["z"], c["lse"], w).mean(), x)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(leaf, c)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(leaf, c)
    with torch.no_grad():
        leaf.copy_(other["x"])
        for n in ("ids", "z", "lse"):
            c[n].copy_(other[n])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, step(other["x"].clone().requires_grad_(True), other))


def test_verify_takes_what_sample_gives(sd):
    """A greedy draft equal to the target is accepted whole; drafts of the filtered draft under the
    filtered target are all possible there."""
    B, gamma, V = 8, 3, 5001
    x = on_gpu(normal(9, B, gamma + 1, V), "bf16")
    T, zero = floats([0.8] * B), floats([0.0] * B)
    u = torch.rand(B, gamma + 1, generator=torch.Generator().manual_seed(3)).clamp(1e-6, 1 - 1e-6).cuda()
    d = sd.sample(x, zero, u[:, :, None].contiguous())
    r = sd.verify_linear(x, d.rows[:, :gamma].contiguous(), d.tokens[:, :gamma, 0].contiguous(), zero, u)
    assert (r.row_status == 0).all() and (r.n_accepted == gamma).all()
    assert torch.equal(r.final_token, d.tokens[:, gamma, 0])
    f = dict(top_k=ints([30] * B), top_p=floats([0.9] * B))
    d = sd.sample(x, T, u[:, :, None].contiguous(), **f)
    rows = sd.filter_logits(x, T, **f).rows
    q = d.rows[:, :gamma].contiguous()
    r = sd.verify_linear(rows, q, d.tokens[:, :gamma, 0].contiguous(), T, u)
    assert (r.row_status == 0).all()
    # the same distribution on both sides: p / q is 1 but for q's half step of 2^-8
    ws = sd.alloc_workspace(B, gamma + 1, V, sd.BF16)
    sd.row_stats(rows, T, ws)
    assert (sd.row_alpha(rows, q, T, ws) >= 1 - 2.0 ** -8).all()
    for b in range(B):
        for i in range(int(r.n_accepted[b]) + 1):
            assert rows[b, i, int(r.out_tokens[b, i])] > -float("inf")


def test_offsets_past_32_bits(sd):
    """More than 2^31 logits: the last row gets what it gets alone."""
    B, R, V = 17, 1001, 128256
    x = torch.empty((B, R, V), dtype=torch.bfloat16, device="cuda")
    x.view(-1, V)[:] = on_gpu(normal(12, 1, 1, V), "bf16").view(1, V)
    last = on_gpu(normal(13, 1, 1, V), "bf16")
    x[-1, -1] = last[0, 0]
    T, p = torch.ones(B, device="cuda"), torch.full((B,), 0.9, device="cuda")
    u = torch.full((B, R, 1), 0.6, device="cuda")
    ids, z, lse = (cuda(a) for a in teacher(14, last.double().cpu().numpy(), 16, 1.0, True))
    wide = lambda t: t.expand(B, R, *t.shape[2:]).contiguous()
    r = sd.sample(x, T, u, top_p=p)
    one = sd.sample(last, T[:1], u[:1, :1].contiguous(), top_p=p[:1])
    assert torch.equal(r.rows[-1, -1], one.rows[0, 0]) and torch.equal(r.tokens[-1, -1], one.tokens[0, 0])
    assert torch.equal(r.rows[0, 0], r.rows[-1, -2]) and r.kept[0, 0] == r.kept[8, 500]
    t, one = sd.top_logits(x, 16), sd.top_logits(last, 16)
    assert torch.equal(t.ids[-1, -1], one.ids[0, 0]) and torch.equal(t.lse[-1, -1], one.lse[0, 0])
    r.rows = None
    d = sd.distill(x, wide(ids), wide(z), wide(lse))
    one = sd.distill(last, ids, z, lse)
    assert torch.equal(d.grad[-1, -1], one.grad[0, 0]) or (d.grad[-1, -1] - one.grad[0, 0]).abs().max() < 1e-6
    assert abs(float(d.loss[-1, -1] - one.loss[0, 0])) < 1e-5


# ---- waits that give up ----

@contextlib.contextmanager
def using(lib):
    from speculative_decoding_verification_64_gb300 import binding
    saved = binding.load_library()
    binding._lib = lib
    try:
        yield
    finally:
        binding._lib = saved


@pytest.mark.parametrize("B,R,V", [(1, 1, 128256), (6, 2, 20011), (300, 1, 1003)])
def test_waits_that_give_up(sd, B, R, V):
    """A build whose waits for copies give up at once: every row says so and holds no result, the calls
    return, and the regular library then gives what it did before."""
    from speculative_decoding_verification_64_gb300 import build
    lib = sd.load_library(build.build(variant="shortwait"))
    x = on_gpu(normal(11, B, R, V), "bf16")
    u = torch.full((B, R, 2), 0.5, device="cuda")
    T, k = torch.ones(B, device="cuda"), torch.arange(B, dtype=torch.int32).cuda() % 50
    p = torch.full((B,), 0.9, device="cuda")
    ids = torch.arange(8, dtype=torch.int32).cuda().expand(B, R, 8).contiguous()
    z = torch.zeros(B, R, 8, device="cuda")
    run = lambda: (sd.sample(x, T, u, k, p), sd.top_logits(x, 8), sd.distill(x, ids, z))
    want = run()
    with using(lib):
        s, t, d = run()
        torch.cuda.synchronize()
    for o in (s, t, d):
        assert (o.row_status & sd.ROW_INTERNAL).all()
    assert (s.tokens == -1).all() and (s.kept == 0).all() and s.rows.isnan().all()
    assert (t.ids == -1).all() and t.lse.isnan().all()
    assert d.loss.isnan().all() and d.grad.isnan().all()
    for a, b in zip(run(), want):
        same(a, b)
