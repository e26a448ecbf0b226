"""The norms of large batches: wrong token ranges are recorded wherever they are, and looking for them does not
take longer than the work."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def step(mla, fp4, starts, tokens):
    """A call that appends `tokens` tokens of these ranges, and its workspace."""
    B = len(starts) - 1
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn(tokens, 64 + 576, device="cuda", generator=gen).to(torch.bfloat16)
    w_q, w_kv = (torch.ones(n, device="cuda", dtype=torch.bfloat16) for n in (64, 512))
    at = torch.tensor(starts, dtype=torch.int32, device="cuda")
    table = torch.arange(B, device="cuda", dtype=torch.int32).reshape(B, 1)
    lens = torch.full((B,), 64, device="cuda", dtype=torch.int32)
    c_q = torch.zeros(tokens, 64, device="cuda", dtype=torch.bfloat16)
    ws = mla.alloc_workspace(mla.WS_HEADER_BYTES)
    if not fp4:
        cache = torch.zeros(B, 64, 576, device="cuda", dtype=torch.bfloat16)
        return lambda: mla.norm_rope_append(x, w_q, w_kv, at, lens, table, cache, c_q=c_q, workspace=ws), ws
    cache = [torch.zeros(B, 64, *s, device="cuda", dtype=t) for s, t in (
        ((256,), torch.uint8), ((32,), torch.uint8), ((), torch.int8), ((64,), torch.bfloat16))]
    plan = mla.rope_plan()
    return lambda: mla.norm_rope_append_fp4(x, w_q, w_kv, at, lens, table, *cache, plan, c_q=c_q,
                                            workspace=ws), ws


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "fp4"])
@pytest.mark.parametrize("at,value", [(None, 0), (0, -1), (4096, 65), (700, 40), (4095, 63), (4095, 65), (2047, -5)])
def test_ranges_that_do_not_ascend(mla, fp4, at, value):
    starts = [min(64, i // 64) for i in range(4097)]
    if at is not None:
        starts[at] = value
    call, ws = step(mla, fp4, starts, 64)
    call()
    # (the start of sequence 4095 is 63 as it is: nothing is wrong with that one)
    wrong = sorted(starts) != starts or starts[0] < 0 or starts[-1] > 64
    assert wrong == (at is not None and (at, value) != (4095, 63))
    assert mla.check_device_status(ws) == (4 if wrong else 0)


def microseconds(call):
    """The shortest of some replays of a graph of 20 calls, a call."""
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


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "fp4"])
def test_time_goes_with_the_tokens(mla, fp4):
    """64 tokens of 4096 sequences and of 64 (one warp that looked over all ranges took 15 times as long)."""
    many = microseconds(step(mla, fp4, [min(64, i) for i in range(4097)], 64)[0])
    few = microseconds(step(mla, fp4, list(range(65)), 64)[0])
    assert many < 5 * few, (many, few)
