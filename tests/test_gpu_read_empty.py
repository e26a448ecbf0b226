"""Rows of the paged cache read back where most of the batch's sequences are not read: the same rows, and in
about the time of a batch of those sequences alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B = 4096
STARTS = {
    "between two": ([0] + [1] * (B - 1) + [64], [0, 1, 64]),
    "before": ([0] * B + [64], [0, 64]),
    "behind": ([0] + [64] * B, [0, 64]),
    "in two places": ([0] * 1000 + [5] * 2000 + [31] * 1096 + [64], [0, 5, 31, 64]),
    "every hundredth": ([min(64, i // 100 + 1 if i else 0) for i in range(B)] + [64], list(range(65))),
}


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def tensors(starts, seed=1):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = len(starts) - 1
    table = torch.randint(0, 500, (n, 1), device="cuda", generator=gen, dtype=torch.int32)
    first = torch.randint(0, 1, (n,), device="cuda", generator=gen, dtype=torch.int32)
    cache = torch.randn(500, 64, 576, device="cuda", generator=gen).to(torch.bfloat16)
    return cache, table, first, torch.tensor(starts, dtype=torch.int32, device="cuda")


def microseconds(mla, starts):
    """The shortest of some replays of a graph of 20 reads, a read."""
    cache, table, first, at = tensors(starts)
    out = torch.zeros(64, 576, dtype=torch.bfloat16, device="cuda")
    ws = mla.alloc_workspace(mla.WS_HEADER_BYTES)
    call = lambda: mla.read_kv(cache, table, first, at, out=out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(20):
            call()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = 1e9
    for _ in range(10):
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 20 * 1e3)
    return best


@pytest.mark.parametrize("name", list(STARTS))
def test_rows(mla, name):
    starts = STARTS[name][0]
    assert len(starts) == B + 1 and sorted(starts) == starts
    cache, table, first, at = tensors(starts)
    out, ws = mla.read_kv(cache, table, first, at, rows=70)
    assert mla.check_device_status(ws) == 0
    r = torch.arange(64, device="cuda")
    b = torch.searchsorted(at[:-1].long(), r, right=True) - 1
    pos = first[b].long() + r - at[b]
    assert torch.equal(out[:64], cache[table[b, 0].long(), pos])
    assert not out[64:].any()


@pytest.mark.parametrize("name", list(STARTS))
def test_time_goes_with_the_rows(mla, name):
    """(One load for each empty sequence took 18 and 100 times as long.)"""
    many, few = (microseconds(mla, s) for s in STARTS[name])
    assert many < 6 * few, (many, few)


@pytest.mark.parametrize("at,value", [(0, -1), (B, 71), (700, 64), (4095, 65), (2047, -5)])
def test_starts_that_do_not_ascend(mla, at, value):
    """Recorded wherever they are among the sequences."""
    starts = [min(64, i // 64) for i in range(B + 1)]
    starts[at] = value
    cache, table, first, on = tensors(starts)
    _, ws = mla.read_kv(cache, table, first, on, rows=70)
    assert mla.check_device_status(ws) == 4
