"""Decode attention behind shared prefixes: a NaN is not lost where an item's parts are merged."""
import pytest
import torch

from tests.test_gpu_shared import mla, run, shared_case

__all__ = ["mla"]
pytestmark = pytest.mark.gpu

CASES = {
    # (heads, groups, rows of the bad value): items of many parts (four threads to a row) and of few
    "one of 128 heads": (128, [(0, [8000])], (0, 10, 4000, 7999)),
    "eight samples": (16, [(9000, [9001 + 130 * i for i in range(8)])], (0, 5000, 8959)),
    "twenty of 64 heads": (64, [(700, [701 + 30 * i for i in range(20)])], (0, 333, 639)),
}


@pytest.mark.parametrize("bits", [0x7FC0, 0x7F80], ids=["nan", "inf"])
@pytest.mark.parametrize("name", list(CASES))
def test_a_bad_row_of_a_cut_item(mla, name, bits):  # noqa: F811
    """Every token sees the row, by way of one part only."""
    heads, groups, rows = CASES[name]
    d = shared_case(31, heads, 1, groups)
    table = d["table"]
    longest = max(range(len(d["lens"])), key=lambda b: d["lens"][b])
    for row in rows:
        bad = dict(d, bits=d["bits"].copy())
        bad["bits"][table[longest, row // 64], row % 64, :512] = bits
        out, lse, status = run(mla, bad)
        assert status == 0
        assert torch.isnan(out).all() and torch.isnan(lse).all(), row
