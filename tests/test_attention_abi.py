"""Argument checks of specdec_rope, specdec_kv_append and specdec_attend, before any device work
(no GPU), and the frequency tables of rope."""
import ctypes
import math

import pytest

P = ctypes.c_void_p
A, TWO, ODD, FOUR = 0x100000, 0x100002, 0x100001, 0x100004   # never dereferenced


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def cache(sd, **kw):
    v = dict(k=A, v=A, k_scale=A, v_scale=A, block_table=A, length=A, n_blocks=4, max_blocks=4,
             block=16, Hkv=2, D=64)
    v.update(kw)
    return sd._CacheStruct(*[v[n] for n, _ in sd._CacheStruct._fields_])


def rope(sd, **kw):
    v = dict(q=A, k=0x200000, dtype=sd.BF16, q_stride=256, k_stride=128, freq=A, positions=None,
             base=None, parent=None, B=2, N=3, Hq=4, Hk=2, D=64, rot=64, flags=0, magnitude=1.0,
             q_out=0x300000, k_out=0x400000, stream=None)
    v.update(kw)
    return sd.load_library().specdec_rope(*v.values())


def test_rope_checks(sd):
    assert rope(sd, B=0, q=None, freq=None) == 0 and rope(sd, N=0, q=None) == 0
    for bad in (dict(dtype=7), dict(B=-1), dict(N=-1), dict(Hq=0), dict(Hk=-1), dict(D=0),
                dict(rot=0), dict(rot=63), dict(rot=66), dict(flags=4), dict(q_stride=255),
                dict(k_stride=127), dict(positions=A, base=A), dict(positions=A, parent=A),
                dict(q=None), dict(freq=None), dict(q_out=None), dict(k=None), dict(k_out=None),
                dict(Hk=0), dict(q=ODD), dict(k_out=ODD), dict(freq=FOUR), dict(positions=TWO),
                dict(base=TWO), dict(parent=TWO), dict(q_out=A + 256), dict(q_out=A, q_stride=300),
                dict(k_out=0x300000), dict(k_out=A)):
        assert rope(sd, **bad) == 1, bad
    assert rope(sd, D=258, rot=64, q_stride=2000, k_stride=2000) == 2
    assert rope(sd, Hq=1025, q_stride=1025 * 64) == 2
    assert rope(sd, B=1 << 20, N=1 << 12) == 2


def append(sd, c=None, **kw):
    v = dict(k=A, v=A, dtype=sd.F32, k_stride=128, v_stride=128, count=None, extra=0, path=None,
             path_len=0, cache=None, B=2, N=3, new_length=0x300000, row_status=0x400000,
             stream=None)
    v.update(kw)
    keep = c if c is not None else cache(sd)
    v["cache"] = ctypes.addressof(keep) if v["cache"] is None else None
    return sd.load_library().specdec_kv_append(*v.values())


CACHE_BAD = [dict(n_blocks=0), dict(max_blocks=0), dict(block=8), dict(block=24), dict(Hkv=0),
             dict(D=8), dict(D=24), dict(k=None), dict(v=None), dict(k_scale=None),
             dict(block_table=None), dict(length=None), dict(k=A + 8), dict(v_scale=TWO),
             dict(length=ODD)]
CACHE_BIG = [dict(block=1040), dict(D=272), dict(Hkv=1025), dict(max_blocks=1 << 28)]


def test_append_checks(sd):
    assert append(sd, B=0, k=None, new_length=None) == 0
    for bad in CACHE_BAD:
        assert append(sd, cache(sd, **bad), k_stride=1 << 20, v_stride=1 << 20) == 1, bad
    for big in CACHE_BIG:
        assert append(sd, cache(sd, **big), k_stride=1 << 20, v_stride=1 << 20) == 2, big
    for bad in (dict(dtype=3), dict(B=-1), dict(N=-1), dict(k_stride=127), dict(v_stride=0),
                dict(path=A), dict(new_length=None), dict(row_status=None), dict(new_length=A),
                dict(k=None), dict(v=None), dict(k=TWO), dict(count=TWO),
                dict(path=TWO, path_len=3), dict(new_length=TWO), dict(cache=0)):
        assert append(sd, **bad) == 1, bad


def attend(sd, c=None, **kw):
    v = dict(q=A, k=A, v=A, dtype=sd.BF16, q_stride=256, k_stride=128, v_stride=128, parent=None,
             n_nodes=None, cache=None, B=2, N=3, Hq=4, scale=0.1, softcap=0.0, slopes=None,
             window=0, out=A, lse=None, row_status=A, workspace=None, workspace_bytes=0,
             stream=None)
    v.update(kw)
    keep = c if c is not None else cache(sd)
    v["cache"] = ctypes.addressof(keep) if v["cache"] is None else None
    return sd.load_library().specdec_attend(*v.values())


def test_attend_checks(sd):
    assert attend(sd, B=0, q=None) == 0 and attend(sd, N=0, q=None) == 0
    for bad in CACHE_BAD:
        assert attend(sd, cache(sd, **bad), q_stride=1 << 20, k_stride=1 << 20,
                      v_stride=1 << 20) == 1, bad
    for big in CACHE_BIG:
        assert attend(sd, cache(sd, **big), q_stride=1 << 20, k_stride=1 << 20,
                      v_stride=1 << 20) == 2, big
    for bad in (dict(dtype=3), dict(B=-1), dict(N=-1), dict(Hq=5), dict(Hq=0), dict(q_stride=255),
                dict(k_stride=127), dict(v_stride=127), dict(scale=math.inf),
                dict(scale=math.nan), dict(softcap=-1.0), dict(softcap=math.nan),
                dict(softcap=math.inf), dict(window=-1), dict(q=None), dict(k=None), dict(v=None),
                dict(out=None), dict(row_status=None), dict(q=ODD), dict(k=ODD), dict(v=ODD),
                dict(out=ODD), dict(parent=TWO), dict(n_nodes=TWO), dict(slopes=TWO),
                dict(lse=TWO), dict(row_status=TWO), dict(cache=0)):
        assert attend(sd, **bad) == 1, bad
    assert attend(sd, N=1025) == 2
    # a workspace that is missing, short or unaligned (these sizes need one)
    need = sd.attend_workspace_size(2, 3, 4, 2, 64, sd.BF16)
    assert need > 0
    assert attend(sd) == 3
    assert attend(sd, workspace=A, workspace_bytes=need - 1) == 3
    assert attend(sd, workspace=A + 8, workspace_bytes=need) == 3


def test_attend_workspace_size(sd):
    size = sd.attend_workspace_size
    for bad in ((0, 3, 4, 2, 64, sd.BF16), (2, 0, 4, 2, 64, sd.BF16), (2, 3, 5, 2, 64, sd.BF16),
                (2, 3, 4, 2, 65, sd.BF16), (2, 1025, 4, 2, 64, sd.BF16), (2, 3, 4, 2, 64, 9)):
        assert size(*bad) == 0, bad
    assert size(1, 5, 32, 8, 128, sd.BF16) > 0


def test_frequency_tables(sd):
    """Plain frequencies, all of them stretched, and stretched by bands."""
    f = [w / 2.0 ** 64 * 2 * math.pi for w in sd.rope_frequencies(64, 10000.0, device="cpu").tolist()]
    assert len(f) == 32
    for i, x in enumerate(f):
        assert abs(x - 10000.0 ** (-i / 32)) <= 2.0 ** -50 * x + 2.0 ** -60
    g = [w / 2.0 ** 64 * 2 * math.pi
         for w in sd.rope_frequencies(64, 10000.0, factor=4.0, device="cpu").tolist()]
    for x, y in zip(f, g):
        assert abs(y - x / 4) <= 2.0 ** -50 * x + 2.0 ** -58
    h = [w / 2.0 ** 64 * 2 * math.pi
         for w in sd.rope_frequencies(64, 10000.0, factor=4.0, original_length=2048,
                                      device="cpu").tolist()]
    assert abs(h[0] - f[0]) < 1e-12 and abs(h[-1] - f[-1] / 4) < 1e-12
    assert all(y <= x * (1 + 1e-12) and y >= x / 4 * (1 - 1e-12) for x, y in zip(f, h))
    for i, x in enumerate(f):   # pairs that turn more than 32, or less than once, over 2048 tokens
        turns = 2048 * x / (2 * math.pi)
        if turns > 32 * 10000.0 ** (1 / 32):
            assert abs(h[i] - x) < 1e-12 * x
        if turns < 10000.0 ** (-1 / 32):
            assert abs(h[i] - x / 4) < 1e-12 * x
    with pytest.raises(ValueError):
        sd.rope_frequencies(63, device="cpu")


def test_host_tensors_are_refused(sd):
    import torch
    x = torch.zeros(2, 3, 4, 64)
    f8 = torch.zeros(4, 4, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    c = sd.KVCache(f8, f8, torch.ones(4, 4), torch.ones(4, 4),
                   torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sd.rope(x, x, sd.rope_frequencies(64, device="cpu"))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sd.kv_append(x, x, c)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sd.attend(x, x, x, c)
