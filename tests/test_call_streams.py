"""Calls on a stream other than the current one: what a call makes for itself (outputs, workspace,
staging) belongs to its stream, so that nobody else is given that memory while its kernels run."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

B, N, V, D = 2, 3, 8, 64
I32 = torch.int32


class Library:
    """Every entry point, doing nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


def calls(sd):
    x, q, tok = torch.zeros(B, N, V), torch.zeros(B, N - 1, V), torch.zeros(B, N - 1, dtype=I32)
    T, u, ws = torch.ones(B), torch.zeros(B, N), torch.zeros(256, dtype=torch.uint8)
    nodes, n32 = torch.zeros(B, N, dtype=I32), torch.zeros(B, dtype=I32)
    lin, tree = sd.LinearOut.empty(B, N - 1, "cpu"), sd.TreeOut.empty(B, N, 2, "cpu")
    a = torch.zeros(B, N, 2, D)
    f8 = torch.zeros(4, 2, 16, D, dtype=torch.uint8).view(torch.float8_e4m3fn)
    cache = sd.KVCache(f8, f8, torch.ones(4, 2), torch.ones(4, 2), torch.zeros(B, 2, dtype=I32), n32)
    freq = torch.zeros(D // 2, dtype=torch.int64)
    return {
        "verify_linear": lambda s: sd.verify_linear(x, q, tok, T, u, stream=s),
        "verify_linear, its own output": lambda s: sd.verify_linear(x, q, tok, T, u, out=lin, stream=s),
        "verify_linear_topk": lambda s: sd.verify_linear_topk(x, q, tok, T, u, 4, stream=s),
        "verify_tree": lambda s: sd.verify_tree(x, x, nodes, nodes, T, u, 2, stream=s),
        "verify_linear_host": lambda s: sd.verify_linear_host(x, q, tok, T, u, out=lin, stream=s,
                                                              sync=False, device="cpu"),
        "verify_tree_host": lambda s: sd.verify_tree_host(x, x, nodes, nodes, T, u, 2, out=tree, stream=s,
                                                          sync=False, device="cpu"),
        "philox_uniforms": lambda s: sd.philox_uniforms([1, 2], [0, 0, 0, 0], 0, 5, device="cpu", stream=s),
        "row_entropy": lambda s: sd.row_entropy(x, T, ws, stream=s),
        "final_mass": lambda s: sd.final_mass(ws, B, N, V, sd.F32, stream=s),
        "row_alpha": lambda s: sd.row_alpha(x, q, T, ws, stream=s),
        "path_logprob": lambda s: sd.path_logprob(x, T, nodes, n32, ws, stream=s),
        "rope": lambda s: sd.rope(a, a, freq, stream=s),
        "kv_append": lambda s: sd.kv_append(a, a, cache, stream=s),
        "attend": lambda s: sd.attend(a, a, a, cache, stream=s),
    }


NAMES = sorted(calls(__import__("speculative_decoding_verification_64_gb300.binding",
                                fromlist=["binding"])))


@pytest.mark.parametrize("name", NAMES)
def test_a_call_makes_its_tensors_on_its_stream(monkeypatch, name):
    from speculative_decoding_verification_64_gb300 import binding as sd
    current, made, empty = [], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    call = calls(sd)[name]
    monkeypatch.setattr(sd, "load_library", Library)
    monkeypatch.setattr(sd, "_cuda", lambda **tensors: None)
    monkeypatch.setattr(sd, "_here", lambda *args: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)

    def make(*args, **kw):
        made.append(current[-1] if current else None)
        return empty(*args, **kw)

    monkeypatch.setattr(torch, "empty", make)
    s = types.SimpleNamespace(cuda_stream=0)
    call(s)
    assert made and all(on is s for on in made)
    assert not current


@pytest.fixture(scope="module")
def gpu():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def busy(s):
    """A few milliseconds of work on stream s."""
    x = torch.randn(4096, 4096, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            x @ x
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["attend, several splits", "attend, large", "verify_linear"])
def test_memory_of_a_call_is_not_given_away_under_it(gpu, case):
    import numpy as np
    import attention_oracle as ref
    rng = np.random.default_rng(1)
    if case == "verify_linear":
        from speculative_decoding_verification_64_gb300 import workloads as W
        x = gpu.linear_inputs_to_device(W.make_workload("linear_b64_g5_v32000_bf16", B=40, V=8001))
        call = lambda **kw: gpu.verify_linear(*x, **kw)
    else:
        B, N, Hq, Hkv, D, dtype = (1, 5, 4, 1, 128, torch.float32) if "splits" in case else \
            (64, 6, 8, 2, 128, torch.bfloat16)
        lens = [20000] if B == 1 else [int(n) for n in rng.integers(0, 2000, B)]
        t = torch.from_numpy(rng.standard_normal((B, N, Hq + 2 * Hkv, D))).to(dtype).cuda()
        cache = ref.on_gpu(ref.make_cache(rng, lens, [0] * B, 64, Hkv, D))
        call = lambda **kw: gpu.attend(t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:], cache, **kw)
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    keep = busy(s)
    got = call(stream=s)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            for n in (1 << 25, 1 << 24, 1 << 22, 1 << 20, 1 << 16, 1 << 12) for _ in range(4)]
    torch.cuda.synchronize()
    for name, w in vars(want).items():
        assert torch.equal(getattr(got, name), w), name
    del junk, keep
