"""Decode attention behind shared prefixes keeps sequences apart: a NaN or an infinity in a cached row
reaches the tokens that see the row, and those are NaN, and no others, whose results stay the same bits."""
import numpy as np
import pytest
import torch

from tests.test_gpu_shared import mla, run, shared_case

__all__ = ["mla"]
pytestmark = pytest.mark.gpu

BAD = {"nan": 0x7FC0, "inf": 0x7F80, "-inf": 0xFF80}
NAMES = {
    # groups, lone ones, places (sequence, row) of the bad value
    "no group": ([(0, [70, 9])], (300, 64, 65, 90, 130, 200, 1), [(0, 69), (1, 0), (2, 150), (3, 63), (8, 0)]),
    "a group": ([(640, [700, 800, 0, 650, 1000, 641, 642, 643, 100, 30])], (5, 300),
                [(0, 640), (1, 799), (4, 900), (4, 5), (4, 300), (8, 70), (9, 29), (11, 299)]),
    # (draft tokens whose rows lie in common pages)
    "no tail": ([(1024, [1024] * 6 + [1020, 1001])], (), [(0, 1023), (3, 1022), (5, 1017), (7, 1000), (6, 960)]),
    "prefix of no page": ([(63, [64, 65, 90, 300, 20, 1, 500, 77])], (), [(3, 64), (6, 499), (5, 0)]),
}


def seen_by(d, page, slot):
    """[sequences, s_q]: the tokens that see this row of the cache."""
    s_q, got = d["s_q"], np.zeros((len(d["lens"]), d["s_q"]), bool)
    for b, n in enumerate(d["lens"]):
        for k in np.nonzero(d["table"][b, :-(-n // 64)] == page)[0]:
            for t in range(s_q):
                got[b, t] |= 64 * k + slot <= n - s_q + t
    return got


def poisoned(d, at, column, bits):
    b, row = at
    page, slot = int(d["table"][b, row // 64]), row % 64
    bad = dict(d, bits=d["bits"].copy())
    bad["bits"][page, slot, column] = bits
    return bad, seen_by(d, page, slot)


@pytest.mark.parametrize("heads,s_q", [(16, 1), (16, 3), (32, 1), (32, 2), (64, 1), (16, 8),
                                       (64, 2)])
@pytest.mark.parametrize("name", list(NAMES))
def test_rows_that_are_not_finite(mla, name, heads, s_q):  # noqa: F811
    groups, lone, places = NAMES[name]
    d = shared_case(21, heads, s_q, groups, lone)
    B = len(d["lens"])
    out, lse, _ = run(mla, d)
    out, lse = out.reshape(B, s_q, heads, 512), lse.reshape(B, s_q, heads)
    assert torch.isfinite(out).all()
    kinds = list(BAD)
    for i, at in enumerate(places):
        # columns in both CTAs' halves of V, and one of the rotated key
        for k, column in enumerate((0, 311, 511, 540)):
            kind = kinds[(i + k) % 3]
            bad, sees = poisoned(d, at, column, BAD[kind])
            got, glse, status = run(mla, bad)
            got, glse = got.reshape(out.shape), glse.reshape(lse.shape)
            assert status == 0
            sees = torch.from_numpy(sees).cuda()
            what = (at, column, kind)
            assert torch.equal(got[~sees], out[~sees]), what
            assert torch.equal(glse[~sees], lse[~sees]), what
            if column < 512 or kind == "nan":
                assert torch.isnan(got[sees]).any(-1).all(), what


@pytest.mark.parametrize("heads", [16, 32, 64])
def test_bad_rows_of_many_at_once(mla, heads):  # noqa: F811
    """Every second sequence has a row that is not finite, in its own or in a page of the prefix's that it
    fills and another does not."""
    d = shared_case(22, heads, 1, [(320, [400, 350, 1, 64, 63, 700, 330, 321, 999])], (3, 64, 128, 200))
    out, lse, _ = run(mla, d)
    bad = dict(d, bits=d["bits"].copy())
    sees = np.zeros((len(d["lens"]), 1), bool)
    for i, b in enumerate(range(1, len(d["lens"]), 2)):
        row = d["lens"][b] - 1
        page, slot = int(d["table"][b, row // 64]), row % 64
        bad["bits"][page, slot, 37 * i % 512] = BAD[list(BAD)[i % 3]]
        sees |= seen_by(d, page, slot)
    assert 0 < sees.sum() < len(sees)
    got, glse, status = run(mla, bad)
    sees = torch.from_numpy(sees[:, 0]).cuda()
    assert status == 0
    assert torch.equal(got[~sees], out[~sees]) and torch.equal(glse[~sees], lse[~sees])
    assert torch.isnan(got[sees]).any(-1).all()


def test_queries_that_are_not_finite(mla):  # noqa: F811
    d = shared_case(23, 16, 1, [(640, [700, 800, 0, 650, 1000, 641, 642, 643, 100, 30])], (5, 300))
    out, lse, _ = run(mla, d)
    for b, bits in ((0, 0x7FC0), (4, 0x7F80), (10, 0xFF80)):
        bad = dict(d, q=d["q"].copy())
        bad["q"][b, :, ::7] = bits
        got, glse, status = run(mla, bad)
        rest = torch.arange(len(d["lens"]), device="cuda") != b
        assert status == 0 and torch.equal(got[rest], out[rest]) and torch.equal(glse[rest], lse[rest])
        assert torch.isnan(got[b]).any(-1).all()


@pytest.mark.parametrize("heads,s_q", [(16, 1), (32, 2)])
def test_rows_of_an_fp8_cache_that_are_not_finite(mla, heads, s_q):  # noqa: F811
    """Exponents that no row of bf16 values has (a page never written may hold any)."""
    d = shared_case(24, heads, s_q, [(640, [700, 800, 0, 650, 1000, 641, 642, 643, 100, 30])], (5, 300), fp8=True)
    out, lse, _ = run(mla, d)
    for b, row in ((0, 640), (1, 799), (4, 5), (8, 70), (11, 299)):
        page, slot = int(d["table"][b, row // 64]), row % 64
        bad = dict(d, exps=d["exps"].copy())
        bad["exps"][page, slot] = 127
        got, glse, status = run(mla, bad)
        sees = torch.from_numpy(seen_by(d, page, slot).reshape(-1)).cuda()
        assert status == 0
        assert torch.equal(got[~sees], out[~sees]) and torch.equal(glse[~sees], lse[~sees])
        assert torch.isnan(got[sees]).any(-1).all()
