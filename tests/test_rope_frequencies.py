"""The frequency tables of rope where they are stretched by bands: a pair that turns more than
beta_fast times over the original length is kept, one that turns fewer than beta_slow times is
stretched by the whole factor, and the ramp between is linear in the pair's index (its ends rounded
outwards to whole pairs).

Tables are words of 2^-64 turns: a frequency f turns is off by 2^-64 at most, and its computation in
double by a few 2^-53 of itself."""
import math

import pytest


@pytest.fixture(scope="module")
def sd():
    from speculative_decoding_verification_64_gb300 import binding
    return binding


def turns(sd, *args, **kw):
    return [w % 2 ** 64 / 2.0 ** 64 for w in sd.rope_frequencies(*args, device="cpu", **kw).tolist()]


@pytest.mark.parametrize("rot,theta,original,fast,slow", [
    (128, 10000.0, 131072, 32.0, 1.0),     # the ramp ends past the last pair
    (64, 10000.0, 1 << 20, 32.0, 1.0),
    (128, 10000.0, 4096, 32.0, 1.0),       # and inside
    (128, 500000.0, 8192, 32.0, 1.0),
    (64, 10000.0, 100, 32.0, 1.0),         # begins before the first pair
    (64, 10000.0, 4, 32.0, 1.0),           # all of it before the first pair
    (32, 10.0, 100000, 32.0, 1.0),         # all of it past the last pair
    (96, 10000.0, 65536, 8.0, 2.0)])
def test_bands(sd, rot, theta, original, fast, slow):
    factor = 4.0
    plain = turns(sd, rot, theta)
    got = turns(sd, rot, theta, factor=factor, original_length=original, beta_fast=fast, beta_slow=slow)
    at = lambda n: rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta))
    low, high = math.floor(at(fast)), math.ceil(at(slow))
    step = theta ** (2.0 / rot)   # between neighbouring pairs: the ramp's ends are whole pairs
    for i, (f, g) in enumerate(zip(plain, got)):
        keep = 1.0 - min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
        want = f * keep + f / factor * (1.0 - keep)
        assert abs(g - want) <= 2.0 ** -48 * f + 2.0 ** -62, (i, g, want)
        n = f * original
        if n > fast * step:
            assert abs(g - f) <= 2.0 ** -48 * f + 2.0 ** -62, i
        if n < slow / step:
            assert abs(g - f / factor) <= 2.0 ** -48 * f + 2.0 ** -62, i
        if slow * step < n < fast / step and high > low:   # on the ramp: neither
            assert f / factor < g < f, i
