"""Which rows the draft side's calls take: strides of any size that the rows' bytes allow (host checks, no
GPU)."""
import pytest

import test_draft_abi as abi

sd = abi.sd  # the fixture

# Each call with one argument that is refused with a code of its own once the rows have passed.
CALLS = {
    "sample": (lambda sd, **kw: abi.sample(sd, S=65, rows=None, **kw), 2),
    "filter": (lambda sd, request, row, **kw: abi.sample(sd, S=65, flags=1, request=request, row=row,
                                                         rows_request=request, rows_row=row, **kw), 2),
    "top": (lambda sd, **kw: abi.top(sd, nbytes=0, **kw), 3),
    "distill": (lambda sd, request, row, **kw: abi.distill(sd, K=1025, request=request, row=row,
                                                           grad_request=request, grad_row=row, **kw), 2),
    "distill, the loss": (lambda sd, **kw: abi.distill(sd, K=1025, grad=None, **kw), 2),
    "backward": (lambda sd, request, row, **kw: abi.backward(sd, K=1025, request=request, row=row,
                                                             grad_request=request, grad_row=row, **kw), 2),
}


def whole(B, R, V):
    return dict(B=B, R=R, V=V, request=R * V, row=V)


FINE = {
    "one long sequence": whole(1, 4096, 152064),
    "one just below 2^29 elements": whole(1, 4185, 128256),
    "one just above": whole(1, 4187, 128256),
    "long sequences": whole(2, 8192, 128256),
    "the last position of each": dict(whole(2, 8192, 128256), R=1),
    "one of them": dict(whole(2, 8192, 128256), B=1, R=1),
    "[R, B, V]": dict(B=8192, R=2, V=128256, request=128256, row=8192 * 128256),
    "many requests": dict(whole(1 << 20, 1, 1000), request=1 << 33),
    "a stride of one request": dict(B=1, R=3, V=1000, request=1 << 62, row=1000),
    "a negative one": dict(B=1, R=3, V=1000, request=-5, row=1000),
    "a stride of one row": dict(B=3, R=1, V=1000, request=1000, row=1 << 62),
    "strides of none": dict(B=1, R=1, V=1000, request=0, row=-(1 << 62)),
    "2^56 bytes": dict(B=3, R=1, V=1024, request=(1 << 54) - 512, row=0),
}

BAD = {
    "rows that overlap": dict(B=1, R=4096, V=152064, request=0, row=152063),
    "requests that overlap": dict(B=2, R=8192, V=128256, request=8192 * 128256 - 1, row=128256),
    "more than 2^56 bytes": dict(B=3, R=1, V=1024, request=(1 << 54) - 511, row=0),
    "a span past 2^63 elements": dict(B=5, R=1, V=1000, request=1 << 61, row=0),
    "past 2^64": dict(B=1 << 20, R=2, V=1000, request=1 << 62, row=1000),
    "both past 2^63": dict(B=3, R=3, V=1000, request=1 << 62, row=1 << 61),
    "rows' stride past 2^64": dict(B=2, R=1 << 20, V=1000, request=1000, row=1 << 62),
    "negative rows": dict(B=1, R=2, V=1000, request=0, row=-1000),
    "negative requests": dict(B=2, R=1, V=1000, request=-1000, row=0),
}


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("rows", sorted(FINE))
def test_strides_that_are_taken(sd, call, rows):
    f, code = CALLS[call]
    assert f(sd, dtype=sd.BF16, **FINE[rows]) == code


@pytest.mark.parametrize("call", sorted(CALLS))
@pytest.mark.parametrize("rows", sorted(BAD))
def test_strides_that_are_refused(sd, call, rows):
    assert CALLS[call][0](sd, dtype=sd.BF16, **BAD[rows]) == 1
    assert CALLS[call][0](sd, dtype=sd.F32, **BAD[rows]) == 1


def test_overlaps_far_apart(sd):
    """Rows written within the span of the rows read, beyond 2^32 bytes."""
    long = dict(B=1, R=8192, V=128256, request=0, row=128256)
    end = abi.A + 2 * 8192 * 128256
    at = lambda rows: abi.sample(sd, dtype=sd.BF16, kept=None, rows=rows, rows_request=0, rows_row=128256, **long)
    to = lambda grad: abi.distill(sd, dtype=sd.BF16, grad=grad, grad_request=0, grad_row=128256, loss=None, **long)
    assert at(end - 2) == 1 and to(end - 2) == 1
    # (apart: refused for what is missing behind)
    assert abi.sample(sd, dtype=sd.BF16, kept=abi.ODD, rows=end, rows_request=0, rows_row=128256, **long) == 1
