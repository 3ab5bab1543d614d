"""Bounded waits of the tensor-core attention kernel that give up.

In the "shortwait" build of the library (test_gpu_wait_expiry.py) the products of this kernel do
not wait for the copies of every second CTA: of a quarter of the CTAs from their second segment (a
request's head, or a part of its tiles) on, of another quarter from the start.  What those CTAs were
to do is left out, while the other CTAs finish.  Every copy still lands before its CTA leaves, and no
wait is left without an end.  A request of which anything was left out reports SPECDEC_ROW_INTERNAL,
whatever head that was of and whether another kernel joins it; the others have their results, to the
bit, and the regular library gives all of them on the same device afterwards.
"""
import math

import numpy as np
import pytest

import attention_oracle as ref
from test_gpu_attend import tokens
from test_gpu_wait_expiry import shortwait, using  # noqa: F401  (shortwait: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


def parts(lens, N, G, Hkv, box, ctas):
    """The requests of which the shortwait build leaves something out, from the kernel's plan: a
    line of units (request, head, row tile), each 4 units of cost and its tiles of 128 tokens, cut
    evenly over the CTAs; a cut inside of the 4 falls before the first tile."""
    rows = N * G
    RN = 32 if rows <= 32 else 48 if rows <= 48 else 64 if rows <= 64 else 128
    units = Hkv * -(-rows // RN)
    ctas *= 2 if RN <= 64 else 1
    line = [(b, max(1, -(-N // 128)) + -(-n // 128)) for b, n in enumerate(lens) for _ in range(units)]
    cost = [tiles + 4 for _, tiles in line]
    total, lost, begun = sum(cost), set(), [0] * ctas
    at = 0
    for (b, tiles), c in zip(line, cost):
        for i in range(ctas):
            lo, hi = total * i // ctas, total * (i + 1) // ctas
            t0, t1 = max(0, lo - at - 4), min(tiles, max(0, hi - at - 4))
            if lo < at + c and hi > at and t0 < t1:   # a segment of this CTA
                if i % 4 == 3 or (i % 4 == 1 and begun[i] > 0):
                    lost.add(b)
                begun[i] += 1
        at += c
    return lost


@pytest.mark.parametrize("B,N,Hq,Hkv,D,most", [
    (120, 3, 8, 2, 64, 900),     # whole units and cut ones, several a CTA
    (40, 9, 8, 2, 128, 3000),    # 36 rows
    (20, 64, 4, 2, 128, 1500),   # 128 rows: four groups of softmax warps
    (3, 5, 4, 1, 128, 30000),    # every unit cut many times
    (400, 1, 1, 1, 96, 200),     # one row, many short requests
])
def test_what_is_given_up_is_reported(shortwait, B, N, Hq, Hkv, D, most):  # noqa: F811
    from speculative_decoding_verification_64_gb300 import binding as sd
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, most, B)]
    q, k, v = tokens(rng, B, N, Hq, Hkv, D, BF16)
    cache = ref.on_gpu(ref.make_cache(rng, lens, [0] * B, 64, Hkv, D))
    more = torch.full((B, 700), -1, dtype=torch.int32, device="cuda")   # room for a large call
    cache.block_table = torch.cat([cache.block_table, more], 1)
    want = sd.attend(q, k, v, cache)
    ws = sd.alloc_attend_workspace(q, cache)
    torch.cuda.synchronize()
    assert (want.row_status == 0).all() and torch.isfinite(want.lse).all()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lost = parts(lens, N, Hq // Hkv, Hkv, 64, sms)
    assert lost
    for _ in range(3):
        ws.fill_(255)
        with using(shortwait):
            got = sd.attend(q, k, v, cache, workspace=ws)
        torch.cuda.synchronize()
        internal = got.row_status.cpu() == sd.ROW_INTERNAL
        assert internal[sorted(lost)].all()
        assert ((got.row_status.cpu() == 0) | internal).all()
        ok = (~internal).cuda()
        assert torch.equal(got.out[ok], want.out[ok]) and torch.equal(got.lse[ok], want.lse[ok])
        # a row of a request that reports it is as it should be, or left out
        gone = (got.lse == -math.inf) & (got.out == 0).all(-1)
        same = (got.lse == want.lse) & (got.out == want.out).all(-1)
        assert (gone | same).all()
    again = sd.attend(q, k, v, cache)
    assert torch.equal(again.out, want.out) and torch.equal(again.lse, want.lse)
    assert (again.row_status == 0).all()
