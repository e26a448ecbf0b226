"""Outputs of mla_rope whose rows lie on top of each other are refused. CPU only: the calls are made with a
width that is refused later than that, so that nothing is launched."""
import ctypes
import random

import pytest

from tests.test_abi_contexts import ROPE
from tests.test_abi_serving import INVALID, P, UNSUPPORTED, call, mla

__all__ = ["mla"]


def overlap(tokens, heads, width, by_token, by_head):
    seen = set()
    for t in range(tokens):
        for h in range(heads):
            row = set(range(t * by_token + h * by_head, t * by_token + h * by_head + width))
            if seen & row:
                return True
            seen |= row
    return False


def rope(mla, out, tokens, heads, rot, by_token, by_head, width=5000):  # noqa: F811
    plan = mla.rope_plan(rot)
    good = dict(x=P, x_token=10 ** 6, x_head=5000, tokens=tokens, heads=heads, width=width, offset=0,
                plan=ctypes.byref(plan), pos=P, y=P, y_token=10 ** 6, y_head=256, rest=None, rest_token=0,
                rest_head=0, stream=None)
    if out == "y":
        good.update(y_token=by_token, y_head=by_head)
    else:
        good.update(rest=P, rest_token=by_token, rest_head=by_head)
    return call(mla.lib(), "mla_rope", ROPE, good)


@pytest.mark.parametrize("tokens,heads,rot,by_token,by_head", [
    (2, 2, 64, 64, 64),      # head 1 of a token on head 0 of the next
    (5, 3, 64, 128, 64),     # on head 0 of the next
    (8, 4, 64, 192, 96),     # partly
    (3, 100, 8, 800, 16),    # far heads on the next token
    (100, 3, 8, 16, 800),
    (9, 7, 8, 40, 64),
])
def test_refused(mla, tokens, heads, rot, by_token, by_head):  # noqa: F811
    assert overlap(tokens, heads, rot, by_token, by_head)
    assert rope(mla, "y", tokens, heads, rot, by_token, by_head) == INVALID


@pytest.mark.parametrize("tokens,heads,rot,by_token,by_head", [
    (5, 3, 64, 192, 64), (5, 3, 64, 64, 320), (1, 9, 64, 0, 64), (9, 1, 64, 64, 0), (2, 2, 64, 128, 192),
    (2, 3, 64, 64, 128), (1 << 24, 4096, 256, 256 * 4096, 256), (1 << 24, 4096, 256, 256, 256 << 24),
    (1 << 20, 4096, 2, 2 ** 62, 2), (1 << 20, 4096, 2, 2, 2 ** 62)])
def test_taken(mla, tokens, heads, rot, by_token, by_head):  # noqa: F811
    if tokens * heads < 1000:
        assert not overlap(tokens, heads, rot, by_token, by_head)
    assert rope(mla, "y", tokens, heads, rot, by_token, by_head) == UNSUPPORTED


@pytest.mark.parametrize("out", ["y", "rest"])
def test_any_strides(mla, out):  # noqa: F811
    rng = random.Random(1)
    found = {True: 0, False: 0}
    for _ in range(3000):
        tokens, heads = rng.randint(1, 6), rng.randint(1, 6)
        rot = 2 * rng.randint(1, 4)
        # (the others of a head of 5000 values are many: steps near that)
        size, unit = (rot, 1) if out == "y" else (5000 - rot, 1250)
        by_token, by_head = (rng.randint(0, 40) * unit + rng.randint(0, 1) for _ in range(2))
        a, b = by_token // unit, by_head // unit
        if out == "rest":
            # the same question in units: rows of 4 or a little less, at multiples or one value on
            if by_token % unit or by_head % unit:
                continue
            want = overlap(tokens, heads, 4, a, b)
        else:
            want = overlap(tokens, heads, size, by_token, by_head)
        found[want] += 1
        got = rope(mla, out, tokens, heads, rot, by_token, by_head)
        assert got == (INVALID if want else UNSUPPORTED), (tokens, heads, rot, by_token, by_head)
    assert min(found.values()) > 100, found
