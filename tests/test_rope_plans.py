"""The frequencies of mla_rope_plan against the scalings' definitions, written out here: every pair of every
even width, both layouts. CPU only."""
import math

import pytest

from tests.test_abi_serving import mla

__all__ = ["mla"]

TWO_PI = 2 * math.pi
PARAMETERS = [
    # theta, factor, original, fast, slow
    (10000.0, 40.0, 4096, 32.0, 1.0),
    (10000.0, 4.0, 4096, 32.0, 1.0),
    (500000.0, 8.0, 8192, 4.0, 1.0),
    (1000000.0, 2.5, 32768, 32.0, 1.0),
    (10000.0, 16.0, 512, 64.0, 0.5),
    (10000.0, 1.0, 4096, 32.0, 1.0),
    (10000.0, 0.5, 100, 20.0, 2.0),
    (2.0, 3.0, 7, 1.5, 0.25),
]
ROTS = list(range(2, 257, 2))


def turns(theta, rot, i, original):
    """Turns of pair i (a real number) over the original context."""
    return original * theta ** (-2.0 * i / rot) / TWO_PI


def pair_of(theta, rot, original, want):
    """The pair, a real number, that turns `want` times: bisection, the turns falling with i."""
    lo, hi = -1e6, 1e6
    for _ in range(200):
        mid = (lo + hi) / 2
        # logarithms: the turns of far pairs leave a float's range
        if math.log(original / TWO_PI) - 2.0 * mid / rot * math.log(theta) > math.log(want):
            lo = mid
        else:
            hi = mid
    return (lo + hi) / 2


def yarn(theta, rot, factor, original, fast, slow):
    low = max(math.floor(pair_of(theta, rot, original, fast)), 0)
    high = min(math.ceil(pair_of(theta, rot, original, slow)), rot - 1)
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if i <= low:
            divided = 0.0
        elif i >= high:
            divided = 1.0
        else:
            divided = (i - low) / (high - low)
        out.append((1 - divided) * f + divided * f / factor)
    return out


def bands(theta, rot, factor, original, fast, slow):
    out = []
    for i in range(rot // 2):
        f, n = theta ** (-2.0 * i / rot), turns(theta, rot, i, original)
        kept = 1.0 if n >= fast else 0.0 if n <= slow else (n - slow) / (fast - slow)
        out.append(kept * f + (1 - kept) * f / factor)
    return out


def ntk(theta, rot, factor):
    """theta grows so that the slowest pair (one pair alone has no other) is divided by factor, and each
    pair is the one before it times the same ratio."""
    if rot == 2:
        return [1.0]
    slowest = theta ** (-(rot - 2.0) / rot) / factor
    ratio = math.exp(math.log(slowest) / (rot // 2 - 1))
    return [ratio ** i for i in range(rot // 2)]


def assert_near(plan, want, what):
    got = list(plan.freq)[:len(want)]
    # pow and log of 64 bits, their arguments' roundings times logarithms under 20: within 1e-12
    bad = [(i, g, w) for i, (g, w) in enumerate(zip(got, want)) if not abs(g - w) <= 1e-12 * w]
    assert not bad, (what, bad[:3])


@pytest.mark.parametrize("theta,factor,original,fast,slow", PARAMETERS)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_frequencies(mla, layout, theta, factor, original, fast, slow):  # noqa: F811
    for rot in ROTS:
        def plan(scaling):
            p = mla.rope_plan(rot, theta=theta, scaling=scaling, factor=factor, original=original,
                              fast=fast, slow=slow, layout=layout)
            assert (p.rot, p.layout) == (rot, {"interleaved": 0, "half": 1}[layout])
            return p
        plain = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
        for scaling, want, magnitude in (
                ("none", plain, 1.0),
                ("linear", [f / factor for f in plain], 1.0),
                ("ntk", ntk(theta, rot, factor), 1.0),
                ("yarn", yarn(theta, rot, factor, original, fast, slow), 1 + 0.1 * math.log(factor)),
                ("bands", bands(theta, rot, factor, original, fast, slow), 1.0)):
            p = plan(scaling)
            assert_near(p, want, (scaling, rot))
            assert abs(p.magnitude - magnitude) <= 2 ** -24 * magnitude + 1e-12, scaling


def test_ramps_have_all_three_parts(mla):  # noqa: F811
    """Of the usual parameters: pairs kept, pairs divided and pairs in between, by yarn's ramp over pairs
    and by the one over turns, which differ."""
    kw = dict(theta=10000.0, factor=40.0, original=4096, fast=32.0, slow=1.0)
    plain = mla.rope_plan(64).freq
    got = {}
    for scaling in ("yarn", "bands"):
        p = mla.rope_plan(64, scaling=scaling, **kw)
        got[scaling] = [p.freq[i] / plain[i] for i in range(32)]
        kept, divided = (sum(abs(r - x) < 1e-12 for r in got[scaling]) for x in (1.0, 1 / 40.0))
        assert kept >= 8 and divided >= 5 and kept + divided < 28, scaling
    assert max(abs(a - b) for a, b in zip(got["yarn"], got["bands"])) > 0.05
