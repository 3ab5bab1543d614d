"""Argument checks of specdec_sample, specdec_top_logits and specdec_distill, before any device
work (no GPU), and the float64 forms that the GPU tests compare with."""
import numpy as np
import pytest

import draft_oracle as ref

A, TWO, ODD = 0x100000, 0x100002, 0x100001   # never dereferenced
FAR = 0x40000000


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def sample(sd, **kw):
    v = dict(logits=A, dtype=sd.BF16, request=3000, row=1000, temperature=A, top_k=A, top_p=A,
             min_p=A, uniforms=A, B=2, R=3, V=1000, S=2, flags=0, tokens=A, rows=FAR,
             rows_request=3000, rows_row=1000, kept=A, status=A, stream=None)
    v.update(kw)
    return sd.load_library().specdec_sample(*v.values())


def top(sd, **kw):
    v = dict(logits=A, dtype=sd.BF16, request=3000, row=1000, temperature=1.0, B=2, R=3, V=1000,
             K=16, values=A, ids=A, lse=A, status=A, workspace=A, nbytes=0, stream=None)
    v.update(kw)
    return sd.load_library().specdec_top_logits(*v.values())


def distill(sd, **kw):
    v = dict(logits=A, dtype=sd.BF16, request=3000, row=1000, ids=A, teacher=A, lse=A, weight=A,
             temperature=1.0, B=2, R=3, V=1000, K=16, loss=A, grad=FAR, grad_request=3000,
             grad_row=1000, status=A, stream=None)
    v.update(kw)
    return sd.load_library().specdec_distill(*v.values())


def backward(sd, **kw):
    v = dict(logits=A, dtype=sd.BF16, request=3000, row=1000, ids=A, teacher=A, lse=A, weight=A,
             dloss=A, temperature=1.0, B=2, R=3, V=1000, K=16, grad=FAR, grad_request=3000,
             grad_row=1000, stream=None)
    v.update(kw)
    return sd.load_library().specdec_distill_backward(*v.values())


ROWS = [dict(dtype=7), dict(B=-1), dict(R=0), dict(V=0), dict(row=999), dict(request=2999),
        dict(row=-1000), dict(request=-1), dict(request=1 << 60), dict(logits=None), dict(logits=ODD),
        dict(dtype=0, logits=TWO)]
WIDE = dict(V=(1 << 19) + 1, row=1 << 20, request=1 << 22)


def test_sample_checks(sd):
    assert sample(sd, B=0, logits=None) == 0
    for bad in ROWS + [dict(S=-1), dict(flags=2), dict(temperature=None), dict(kept=None),
                       dict(status=None), dict(uniforms=None), dict(tokens=None), dict(rows=ODD),
                       dict(rows_row=999), dict(rows_request=2999), dict(temperature=TWO),
                       dict(top_k=TWO), dict(top_p=TWO), dict(min_p=TWO), dict(uniforms=TWO),
                       dict(tokens=TWO), dict(kept=TWO), dict(status=TWO),
                       dict(rows=A, rows_row=1008, rows_request=3024),  # over the logits, elsewhere
                       dict(rows=A + 16)]:
        assert sample(sd, **bad) == 1, bad
    for far in (dict(WIDE, rows_row=1 << 20, rows_request=1 << 22), dict(S=65),
                dict(B=1 << 20, R=1 << 10, request=1 << 30, rows_request=1 << 30)):
        assert sample(sd, **far) == 2, far


def test_top_logits_checks(sd):
    size = sd.top_logits_workspace_size
    assert size(0, 3, 1000, sd.BF16) == 0 and size(2, 0, 1000, sd.BF16) == 0
    assert size(2, 3, (1 << 21) + 1, sd.BF16) == 0 and size(2, 3, 1000, 5) == 0
    assert size(2, 3, 1000, sd.BF16) >= 6 * (8 + 64)
    assert size(2, 3, 128256, sd.BF16) >= 6 * 32 * (8 + 64)
    assert top(sd, B=0, logits=None) == 0
    for bad in ROWS + [dict(K=0), dict(K=1001), dict(temperature=0.0), dict(temperature=-1.0),
                       dict(temperature=float("nan")), dict(temperature=2.0 ** 21), dict(values=None),
                       dict(ids=None), dict(lse=None), dict(status=None), dict(values=TWO),
                       dict(ids=TWO), dict(lse=TWO), dict(status=TWO)]:
        assert top(sd, **bad) == 1, bad
    assert top(sd, K=1025, V=2000, row=2000, request=6000) == 2
    assert top(sd, V=(1 << 21) + 1, row=1 << 22, request=1 << 24) == 2
    assert top(sd) == 3 and top(sd, workspace=None, nbytes=1 << 30) == 3
    assert top(sd, workspace=A + 8, nbytes=1 << 30) == 3


def test_distill_checks(sd):
    assert distill(sd, B=0, logits=None) == 0 and backward(sd, B=0, logits=None) == 0
    both = ROWS + [dict(K=0), dict(temperature=0.0), dict(temperature=float("inf")), dict(ids=None),
                   dict(teacher=None), dict(ids=TWO), dict(teacher=TWO), dict(lse=TWO),
                   dict(weight=TWO), dict(grad=ODD), dict(grad_row=999), dict(grad_request=2999),
                   dict(grad=A + 16), dict(grad=A, grad_row=1008, grad_request=3024)]
    for bad in both + [dict(loss=None), dict(status=None), dict(loss=TWO), dict(status=TWO)]:
        assert distill(sd, **bad) == 1, bad
    for bad in both + [dict(grad=None), dict(grad=A), dict(dloss=None), dict(dloss=TWO)]:
        assert backward(sd, **bad) == 1, bad
    for far in (dict(K=1025), dict(WIDE, grad_row=1 << 20, grad_request=1 << 22)):
        assert distill(sd, **far) == 2 and backward(sd, **far) == 2, far


def test_host_tensors_are_refused(sd):
    torch = pytest.importorskip("torch")
    x, T, u = torch.zeros(1, 2, 8), torch.ones(1), torch.zeros(1, 2, 1)
    ids, z = torch.zeros(1, 2, 1, dtype=torch.int32), torch.zeros(1, 2, 1)
    for call in (lambda: sd.sample(x, T, u), lambda: sd.filter_logits(x, T),
                 lambda: sd.top_logits(x, 1), lambda: sd.distill(x, ids, z),
                 lambda: sd.distill_loss(x.clone().requires_grad_(True), ids, z)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_shapes_and_types_are_checked(sd, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(sd, "_here", lambda *args: 0)
    x, T, u = torch.zeros(2, 2, 8), torch.ones(2), torch.zeros(2, 2, 1)
    ids, z = torch.zeros(2, 2, 3, dtype=torch.int32), torch.zeros(2, 2, 3)
    out = sd.SampleOut(None, None, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32))
    wrong = [
        lambda: sd.sample(x[0], T, u), lambda: sd.sample(x.double(), T, u), lambda: sd.sample(x, T[:1], u),
        lambda: sd.sample(x, T, u[:, :, 0]), lambda: sd.sample(x, T, u[:1]),
        lambda: sd.sample(x, T, u.double()), lambda: sd.sample(x.transpose(1, 2), T, u),
        lambda: sd.sample(x, T, u, top_k=torch.ones(2)), lambda: sd.sample(x, T, u, top_p=torch.ones(3)),
        lambda: sd.sample(x, T, u, min_p=torch.ones(2).double()), lambda: sd.sample(x, T, u, out=out),
        lambda: sd.top_logits(x[0], 2), lambda: sd.top_logits(x.half(), 2),
        lambda: sd.distill(x, ids[0], z), lambda: sd.distill(x, ids.long(), z),
        lambda: sd.distill(x, ids, z[:, :, :2]), lambda: sd.distill(x, ids, z.double()),
        lambda: sd.distill(x, ids, z, lse=z), lambda: sd.distill(x, ids, z, weight=T),
        lambda: sd.distill(x, ids, z, out=sd.DistillOut(u[:, :, 0].contiguous(), x[:, :, :4], out.kept)),
    ]
    for call in wrong:
        with pytest.raises((ValueError, TypeError)):
            call()


def test_the_oracle_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    assert ref.keep(x, 1.0)[0].all()
    assert ref.keep(x, 1.0, k=3)[0].tolist() == [False, True, True, True, False]
    assert ref.keep(x, 1.0, k=2)[0].tolist() == [False, True, True, False, False]  # the lower index
    assert ref.keep(x, 1.0, p=0.7)[0].tolist() == [False, True, True, True, False]
    assert ref.keep(x, 1.0, p=0.0)[0].tolist() == [False, True, False, False, False]
    assert ref.keep(x, 1.0, k=3, p=0.6)[0].tolist() == [False, True, True, False, False]  # of 0.8
    assert ref.keep(x, 1.0, m=0.45)[0].tolist() == [False, True, True, True, False]
    assert ref.keep(x, 0.0)[0].tolist() == [False, True, False, False, False]
    tokens, q, _ = ref.sample(x, 1.0, [0.05, 0.15, 0.55, 0.95])
    assert tokens == [0, 1, 2, 4] and np.allclose(q, np.exp(x))
    # a draw's law, by a fine grid of uniforms
    us = (np.arange(1000) + 0.5) / 1000
    tokens, q, _ = ref.sample(x, 0.7, us, p=0.85)
    assert np.allclose(np.bincount(tokens, minlength=5) / 1000, q, atol=1e-3)


def test_the_oracle_gradient_by_differences():
    rng = np.random.default_rng(1)
    x, z = rng.standard_normal(9) * 2, rng.standard_normal(3)
    ids = [7, -1, 2]
    for lse in (None, 1.5):
        loss, g = ref.distill(x, ids, z, lse, T=1.3)
        assert loss > 0
        for v in range(9):
            e = np.zeros(9)
            e[v] = 1e-5
            d = (ref.distill(x + e, ids, z, lse, T=1.3)[0] - ref.distill(x - e, ids, z, lse, T=1.3)[0]) / 2e-5
            assert abs(d - g[v]) < 1e-8
