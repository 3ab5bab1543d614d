"""The cases of test_gpu_attend.py on the kernel that large bfloat16 calls take.

Which kernel a call takes goes by what its cache can hold and by how many requests and heads
there are, so the same cases, with their tolerances, run again with a block table that has room
for many more tokens (its further entries stay -1 and are not read), or, where a window bounds
what is read anyway, with the requests repeated.
"""
import dataclasses

import pytest

import test_gpu_attend as cases

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


class Large:
    """The binding, with calls made large."""

    def __init__(self, sd):
        self.sd = sd

    def __getattr__(self, name):
        return getattr(self.sd, name)

    def attend(self, q, k, v, cache, parent=None, n_nodes=None, window=0, **kw):
        B, room = q.shape[0], -(-40000 // cache.k.shape[2])
        table = cache.block_table
        if window == 0:
            more = torch.full((B, room), -1, dtype=torch.int32, device=table.device)
            cache = dataclasses.replace(cache, block_table=torch.cat([table, more], 1))
            return self.sd.attend(q, k, v, cache, parent=parent, n_nodes=n_nodes, **kw)
        times = 305 // (B * cache.k.shape[1]) + 1
        many = [None if t is None else t.repeat(times, *[1] * (t.dim() - 1))
                for t in (q, k, v, table, cache.length, parent, n_nodes)]
        cache = dataclasses.replace(cache, block_table=many[3], length=many[4])
        r = self.sd.attend(*many[:3], cache, parent=many[5], n_nodes=many[6], window=window, **kw)
        return dataclasses.replace(r, out=r.out[:B], row_status=r.row_status[:B],
                                   lse=None if r.lse is None else r.lse[:B])


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return Large(binding)


@pytest.mark.parametrize("lens,N,Hq,Hkv,D,block,pad", [s for s in cases.SHAPES if s[4] <= 128])
def test_chains(sd, lens, N, Hq, Hkv, D, block, pad):
    cases.test_chains(sd, BF16, lens, N, Hq, Hkv, D, block, pad)


@pytest.mark.parametrize("softcap,bias,window", [(0.0, False, 0), (30.0, False, 0), (0.0, True, 0),
                                                 (0.0, False, 5), (20.0, True, 33)])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(64, 8, 2, 128), (23, 3, 3, 64), (130, 2, 1, 96),
                                        (9, 8, 2, 64), (3, 4, 1, 128)])
def test_trees(sd, softcap, bias, window, N, Hq, Hkv, D):
    cases.test_trees(sd, BF16, softcap, bias, window, N, Hq, Hkv, D)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (128, 1)])
def test_non_finite_values_reach_only_the_rows_that_see_them(sd, D, G):
    cases.test_non_finite_values_reach_only_the_rows_that_see_them(sd, BF16, D, G)


def test_wide_ranges(sd):
    cases.test_wide_ranges(sd, BF16)


@pytest.mark.parametrize("N,G", [(1, 1), (6, 4), (40, 4)])
def test_a_flat_tail_under_a_sink(sd, N, G):
    cases.test_a_flat_tail_under_a_sink(sd, BF16, N, G)


def test_scores_of_minus_infinity_and_plus_infinity(sd):
    cases.test_scores_of_minus_infinity_and_plus_infinity(sd)


def test_misaligned_activations_and_outputs(sd):
    cases.test_misaligned_activations_and_outputs(sd)


def test_a_late_copying_warp_is_not_overtaken(sd):
    """Hundreds of requests of a few tokens, again and again behind other work: a CTA passes from
    request to request at every other tile, and results stay the same to the bit."""
    g = torch.Generator().manual_seed(5)
    B, N, Hkv, D, block = 300, 1, 2, 64, 32
    q, k, v = (torch.randn(B, N, Hkv, D, generator=g).to(BF16).cuda() for _ in range(3))
    lens = torch.randint(0, 400, (B,), generator=g, dtype=torch.int32)
    n_nodes = torch.randint(0, 2, (B,), generator=g, dtype=torch.int32).cuda()
    blocks = -(-400 // block)
    cache = sd.KVCache.empty(B, blocks, B * blocks, block, Hkv, D)
    cache.k.view(torch.uint8).random_(0, 120)
    cache.v.view(torch.uint8).random_(0, 120)
    cache.k_scale.fill_(2.0 ** -8)
    cache.v_scale.fill_(2.0 ** -8)
    cache.block_table.copy_(torch.randperm(B * blocks, generator=g).view(B, blocks))
    cache.length.copy_(lens)
    first = None
    noise = torch.randn(1024, 1024, device="cuda", dtype=BF16)
    side = torch.cuda.Stream()
    for i in range(400):
        with torch.cuda.stream(side):
            noise @ noise
        r = sd.sd.attend(q, k, v, cache, n_nodes=n_nodes)
        if first is None:
            first = r
            assert (r.row_status == 0).all()
        assert torch.equal(r.out, first.out) and torch.equal(r.lse, first.lse), i
