"""Window decode in batches of every size against the clusters, and both ragged calls replayed from
graphs over lengths, token ranges, tables and queries that have changed in place."""
import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.helpers import dev_i32
from tests.test_gpu_rows import _cache, _q, check, run_window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def lengths(seed, n, most, s_q):
    """Unequal ones, with none at all, fewer rows than tokens, and the longest among them."""
    rng = np.random.default_rng(seed)
    lens = [int(v) for v in rng.integers(1, most + 1, n)]
    for k, v in enumerate((0, most, 1, s_q, max(0, s_q - 1), 64, 65)):
        lens[(k * 11 + 3) % n] = v
    return lens


# (the clusters of the device this library is for number 76)
@pytest.mark.parametrize("n", [20, 39, 57, 76, 77])
@pytest.mark.parametrize("heads,s_q", [(128, 1), (64, 1), (16, 3)])
@pytest.mark.parametrize("fp8", [False, True])
def test_window_of_several_tiles(mla, n, heads, s_q, fp8):
    lens = lengths(n, n, 900, s_q)
    d = R.attention_case(50, heads, [s_q] * n, lens, 450, 70, fp8=fp8)
    check(d, *run_window(mla, d, s_q))


@pytest.mark.parametrize("heads,s_q", [(16, 1), (16, 8), (32, 3), (64, 2), (128, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_window_scheduled(mla, heads, s_q, fp8):
    lens = lengths(heads + s_q, 200, 600, s_q)
    d = R.attention_case(51, heads, [s_q] * 200, lens, 130, 4, fp8=fp8)
    check(d, *run_window(mla, d, s_q))


@pytest.mark.parametrize("n", [5, 50, 150])
@pytest.mark.parametrize("fp8", [False, True])
def test_window_is_the_same_every_time(mla, n, fp8):
    d = R.attention_case(52, 64, [2] * n, lengths(n, n, 700, 2), 300, 4, fp8=fp8)
    out, lse, st = run_window(mla, d, 2)
    assert st == 0
    for _ in range(3):
        o, l, _ = run_window(mla, d, 2)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)


class Places:
    """Device arrays that every one of `cases` fits in, and how to put one there."""

    def __init__(self, cases, most):
        self.cases = cases
        pool = max(d["pool"] for d in cases)
        B, T, H = len(cases[0]["lens"]), cases[0]["tokens"], cases[0]["heads"]
        self.q = [torch.zeros(T, H, n, dtype=torch.bfloat16, device="cuda") for n in (512, 64)]
        self.cache = [torch.zeros(pool, *c.shape[1:], dtype=c.dtype, device="cuda")
                      for c in _cache(cases[0])]
        self.table = torch.full((B, -(-most // 64)), -1, dtype=torch.int32, device="cuda")
        self.starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.out = torch.zeros_like(self.q[0])
        self.lse = torch.zeros(T, H, device="cuda")

    def put(self, k):
        d = self.cases[k]
        for to, x in zip(self.q, _q(d)):
            to.copy_(x)
        for to, x in zip(self.cache, _cache(d)):
            to[:len(x)].copy_(x)
        self.table.fill_(-1)
        self.table[:, :d["table"].shape[1]] = dev_i32(d["table"])
        self.starts.copy_(dev_i32(d["starts"]))
        self.lens.copy_(dev_i32(d["lens"]))
        self.out.zero_(), self.lse.zero_()
        return d


def replay(mla, places, call, ws):
    places.put(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(side)
    for k in [*range(len(places.cases)), 0]:
        d = places.put(k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(d, places.out, places.lse, mla.check_device_status(ws))


CHUNKS = {  # token counts with one sum
    "ranges": (32, 1000, [([5, 1, 40], [300, 700, 90]), ([40, 6, 0], [900, 6, 400]),
                          ([0, 2, 44], [0, 1000, 64])]),
    "scheduled": (128, 700, [([60, 1, 70], [200, 300, 150]), ([1, 100, 30], [700, 100, 500]),
                             ([131, 0, 0], [131, 700, 0]), ([0, 100, 31], [5, 3, 650])]),
}


@pytest.mark.parametrize("mode", list(CHUNKS))
@pytest.mark.parametrize("fp8", [False, True])
def test_replayed_chunks_of_other_lengths(mla, mode, fp8):
    heads, most, batches = CHUNKS[mode]
    cases = [R.attention_case(53 + k, heads, c, n, 200 * (mode == "ranges"), 3, fp8=fp8)
             for k, (c, n) in enumerate(batches)]
    p = Places(cases, most)
    d = cases[0]
    ws = mla.alloc_workspace(mla.chunk_workspace_size(3, d["tokens"], heads, most, d["window"], 3))
    run = mla.chunk_attention_fp8 if fp8 else mla.chunk_attention
    replay(mla, p, lambda s: run(*p.q, *p.cache, p.table, p.starts, p.lens, most, d["scale"],
                                 window=d["window"], sinks=3, out=p.out, lse=p.lse, workspace=ws,
                                 stream=s), ws)


@pytest.mark.parametrize("n", [4, 60, 130])  # ranges of a sequence, whole ones, scheduled
@pytest.mark.parametrize("fp8", [False, True])
def test_replayed_windows_of_other_lengths(mla, n, fp8):
    most = 800
    cases = [R.attention_case(57 + k, 32, [2] * n, lengths(k, n, most, 2) if n > 10 else
                              [most, 0, 65 * k, 1 + k], 300, 5, fp8=fp8) for k in range(3)]
    p = Places(cases, most)
    ws = mla.alloc_workspace(mla.decode_window_workspace_size(n, 2, 32, most, 300, 5))
    run = mla.decode_attention_window_fp8 if fp8 else mla.decode_attention_window

    def shaped(t):
        return t.view(n, 2, *t.shape[1:])

    replay(mla, p, lambda s: run(*map(shaped, p.q), *p.cache, p.table, p.lens, most, 300, 5,
                                 R.SCALE, out=shaped(p.out), lse=shaped(p.lse), workspace=ws,
                                 stream=s), ws)
