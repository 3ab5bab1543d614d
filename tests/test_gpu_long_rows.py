"""The draft side's calls on sequences of more than 2^29 logits a request: the last row gets what it gets
alone."""
import numpy as np
import pytest

from test_gpu_distill import cuda, teacher
from test_gpu_sample import floats, normal, on_gpu

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def check(sd, x, last):
    """x [B, R, V], whose last row is `last` [1, 1, V]."""
    B, R, V = x.shape
    one, T, p = on_gpu(last, "bf16"), floats([0.8] * B), floats([0.9] * B)
    ids, z, lse = (cuda(a) for a in teacher(2, one.double().cpu().numpy(), 16, 1.0, True))
    u = torch.full((B, R, 1), 0.3, device="cuda")
    want = sd.sample(one, T[:1], u[:1, :1].contiguous(), top_p=p[:1])
    s = sd.sample(x, T, u, top_p=p)
    assert torch.equal(s.rows[-1, -1], want.rows[0, 0]) and torch.equal(s.tokens[-1, -1], want.tokens[0, 0])
    assert torch.equal(s.kept[-1, -1], want.kept[0, 0]) and (s.row_status == 0).all()
    del s
    want = sd.top_logits(one, 16)
    t = sd.top_logits(x, 16)
    assert torch.equal(t.ids[-1, -1], want.ids[0, 0]) and torch.equal(t.values[-1, -1], want.values[0, 0])
    # (sums of as many CTAs as the call has rows for)
    assert abs(float(t.lse[-1, -1] - want.lse[0, 0])) < 1e-5 and (t.row_status == 0).all()
    wide = lambda a: a.expand(B, R, *a.shape[2:]).contiguous()
    want = sd.distill(one, ids, z, lse)
    d = sd.distill(x, wide(ids), wide(z), wide(lse))
    assert (d.grad[-1, -1] - want.grad[0, 0]).abs().max() < 1e-6
    assert abs(float(d.loss[-1, -1] - want.loss[0, 0])) < 1e-5 and (d.row_status == 0).all()


def rows(B, R, V):
    x = torch.empty((B, R, V), dtype=torch.bfloat16, device="cuda")
    x.view(-1, V)[:] = on_gpu(normal(1, 1, 1, V), "bf16").view(1, V)
    last = np.float64(normal(2, 1, 1, V))
    x[-1, -1] = on_gpu(last, "bf16")[0, 0]
    return x, last


def test_one_long_sequence(sd):
    x, last = rows(1, 4096, 152064)
    check(sd, x, last)


def test_the_last_position_of_long_sequences(sd):
    x, last = rows(2, 8192, 128256)
    check(sd, x[:, -1:], last)
    check(sd, x[1:, -3:], last)


def test_a_filter_and_a_gradient_in_place(sd):
    """Written at the far end of the logits themselves."""
    x, last = rows(1, 4200, 128256)
    one, T, p = on_gpu(last, "bf16"), floats([0.8]), floats([0.9])
    want = sd.filter_logits(one, T, top_p=p)
    keep = x[:, -2].clone()
    f = sd.filter_logits(x[:, -1:], T, top_p=p, out=sd.SampleOut(None, x[:, -1:], want.kept.clone(),
                                                                 want.row_status.clone()))
    assert torch.equal(x[0, -1], want.rows[0, 0]) and torch.equal(f.kept, want.kept)
    assert torch.equal(x[:, -2], keep)
