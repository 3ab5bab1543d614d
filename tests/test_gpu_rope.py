"""Rotary positions on the GPU against the formula in 64 bits.

Tolerance.  The phase is exact up to its cut to 32 bits and its rounding to
float32 (together at most pi 2^-24 of an angle), sincospi is good to 2^-22, and
each output is two products and a sum of float32: |error| <= 2^-20 (|x1| +
|x2|) magnitude.  A bfloat16 result adds its rounding, 2^-8 of the result (8
significant bits).
"""
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


def check(y, x, want, rot, interleaved, magnitude, dtype):
    """|error| element by element; the unrotated part is copied bit for bit."""
    a = x.abs()
    pair = a.clone()
    if interleaved:
        pair[..., 0:rot:2] = pair[..., 1:rot:2] = a[..., 0:rot:2] + a[..., 1:rot:2]
    else:
        pair[..., :rot // 2] = pair[..., rot // 2:rot] = a[..., :rot // 2] + a[..., rot // 2:rot]
    tol = pair * magnitude * 2.0 ** -20
    if dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8
    tol[..., rot:] = 0
    assert ((y.double().cpu() - want).abs() <= tol).all()


def inputs(rng, B, N, Hq, Hk, D, dtype, pad=0):
    """q and k as slices of a fused projection, `pad` elements between tokens."""
    x = torch.from_numpy(rng.standard_normal((B, N, (Hq + Hk) * D + pad))).to(dtype).cuda()
    q = x[:, :, :Hq * D].unflatten(2, (Hq, D))
    return q, x[:, :, Hq * D:(Hq + Hk) * D].unflatten(2, (Hk, D)) if Hk else None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hk,D,rot,pad", [
    (1, 1, 1, 1, 2, 2, 0), (1, 5, 4, 2, 64, 64, 0), (3, 7, 5, 1, 128, 64, 0),
    (2, 3, 3, 3, 96, 96, 8), (2, 3, 2, 1, 80, 20, 0), (2, 2, 3, 2, 33, 30, 0),
    (1, 4, 2, 1, 256, 256, 1), (2, 2, 4, 0, 48, 16, 16)])
@pytest.mark.parametrize("backward", [False, True])
def test_rope_matches_the_formula(sd, dtype, interleaved, B, N, Hq, Hk, D, rot, pad, backward):
    rng = np.random.default_rng(B * 1000 + D)
    q, k = inputs(rng, B, N, Hq, Hk, D, dtype, pad)
    freq = sd.rope_frequencies(rot, 10000.0)
    pos = torch.from_numpy(rng.integers(0, 2 ** 20, (B, N))).int()
    pos[0, 0] = 2 ** 31 - 1
    pos[-1, -1] = -5
    magnitude = 1.25
    qo, ko = sd.rope(q, k, freq, positions=pos.cuda(), interleaved=interleaved, backward=backward,
                     magnitude=magnitude)
    words = [w % 2 ** 64 for w in freq.tolist()]
    for x, y in ((q, qo), (k, ko)):
        if x is None:
            assert y is None
            continue
        want = ref.rope(x.double().cpu(), pos, words, interleaved, backward, magnitude)
        check(y, x.double().cpu(), want, rot, interleaved, magnitude, dtype)


def test_tree_and_chain_positions(sd):
    rng = np.random.default_rng(7)
    B, N = 4, 37
    q, k = inputs(rng, B, N, 2, 1, 64, torch.float32)
    freq = sd.rope_frequencies(64, 500000.0)
    parents = [ref.random_tree(rng, N) for _ in range(B)]
    base = torch.tensor([0, 5, 131071, 77], dtype=torch.int32)
    for parent in (None, torch.tensor(parents, dtype=torch.int32)):
        depth = [[len(ref.ancestors(None if parent is None else parents[b], n)) - 1
                  for n in range(N)] for b in range(B)]
        pos = (base[:, None] + torch.tensor(depth)).int().cuda()
        a = sd.rope(q, k, freq, positions=pos)
        b = sd.rope(q, k, freq, base=base.cuda(), parent=None if parent is None else parent.cuda())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # without a base, positions count from 0
    a = sd.rope(q, k, freq)
    b = sd.rope(q, k, freq, positions=torch.arange(N, dtype=torch.int32).cuda().repeat(B, 1))
    assert torch.equal(a[0], b[0])
    # a parent that is not below its node ends the walk
    wild = torch.full((B, N), 2 ** 31 - 1, dtype=torch.int32).cuda()
    a = sd.rope(q, k, freq, parent=wild)
    b = sd.rope(q, k, freq, positions=torch.zeros(B, N, dtype=torch.int32).cuda())
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_is_the_gradient(sd, interleaved):
    """<dy, rope(x + h) - rope(x - h)> / 2 h against <dx, e>: the map is linear, so differences
    carry rounding alone: 64 products of float32 of size |x| |dy| <= 25 over 2 h = 2: 64 * 25 *
    2^-22 < 4e-4 at most."""
    rng = np.random.default_rng(3)
    x, _ = inputs(rng, 2, 3, 2, 0, 64, torch.float32)
    dy, _ = inputs(rng, 2, 3, 2, 0, 64, torch.float32)
    freq = sd.rope_frequencies(48)
    base = torch.tensor([1000, 70000], dtype=torch.int32).cuda()
    run = lambda t, back=False: sd.rope(t, None, freq, base=base, interleaved=interleaved,
                                        backward=back, magnitude=0.75)[0]
    dx = run(dy, True)
    for _ in range(20):
        e = torch.zeros(2, 3, 2, 64, device="cuda")
        i = tuple(rng.integers(0, n) for n in e.shape)
        e[i] = 1.0
        diff = (run(x + e) - run(x - e)).double() / 2
        assert abs(float((diff * dy.double()).sum()) - float(dx[i])) <= 4e-4
    # and against the transpose of the formula
    pos = base.cpu()[:, None] + torch.arange(3)
    want = ref.rope(dy.double().cpu(), pos, [w % 2 ** 64 for w in freq.tolist()], interleaved,
                    True, 0.75)
    check(dx, dy.double().cpu(), want, 48, interleaved, 0.75, torch.float32)


def test_in_place_other_stream_and_empty(sd):
    rng = np.random.default_rng(5)
    freq = sd.rope_frequencies(128)
    q, k = inputs(rng, 2, 9, 4, 2, 128, torch.bfloat16)
    q, k = q.contiguous(), k.contiguous()
    want = sd.rope(q, k, freq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = sd.rope(q, k, freq, q_out=q, k_out=k)
    side.synchronize()
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    a, b = sd.rope(q[:0], k[:0], freq)
    assert a.shape == (0, 9, 4, 128) and b.shape == (0, 9, 2, 128)
    a, _ = sd.rope(q[:, :0], None, freq)
    assert a.shape == (2, 0, 4, 128)


def test_non_finite_elements_stay_in_their_pair(sd):
    q = torch.ones(1, 1, 1, 64, device="cuda")
    q[0, 0, 0, 3], q[0, 0, 0, 9] = float("nan"), float("inf")
    y, _ = sd.rope(q, None, sd.rope_frequencies(64), positions=torch.tensor([[11]]).int().cuda())
    bad = ~torch.isfinite(y[0, 0, 0])
    assert bad.nonzero().flatten().tolist() == [3, 9, 35, 41]


def test_refusals(sd):
    x = torch.zeros(2, 3, 4, 64, device="cuda")
    f = sd.rope_frequencies(64)
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        sd.rope(x.half(), None, f)
    with pytest.raises(TypeError):
        sd.rope(x, x.bfloat16(), f)
    with pytest.raises(TypeError):
        sd.rope(x, x, f.float())
    with pytest.raises(ValueError):
        sd.rope(x[0], None, f)
    with pytest.raises(ValueError):
        sd.rope(x, torch.zeros(2, 3, 4, 32, device="cuda"), f)
    with pytest.raises(ValueError):
        sd.rope(x.transpose(1, 2), None, f)
    with pytest.raises(ValueError):
        sd.rope(x, None, f, positions=torch.zeros(2, 4, **i32))
    with pytest.raises(ValueError):
        sd.rope(x.cpu(), None, f)
    with pytest.raises(sd.SpecdecError):   # more pairs than the head has
        sd.rope(x, None, sd.rope_frequencies(128))
    with pytest.raises(sd.SpecdecError):   # positions and a base
        sd.rope(x, None, f, positions=torch.zeros(2, 3, **i32), base=torch.zeros(2, **i32))
    fused = torch.zeros(2, 3, 6, 64, device="cuda")
    with pytest.raises(sd.SpecdecError):   # the output over a strided input
        sd.rope(fused[:, :, :4], None, f, q_out=fused.view(-1)[:x.numel()].view(2, 3, 4, 64))
