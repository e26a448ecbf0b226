"""The pages' calls and plain decode over the same lengths and table, on one stream with nothing
between them: the lengths that a call has just written are the ones that the next one uses."""
import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.helpers import dev_i32, host_bits, host_f64_from_bf16

pytestmark = pytest.mark.gpu

HEADS, ROWS, MOST, POOL = 16, 140, 12, 3000
CTX = 64 * MOST


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


class State:
    """Rows of a server, most of the pool held by others (so that the free pages lie several passes
    of the plan's scan behind its start), and the buffers of every call."""

    def __init__(self, mla, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.mla, self.rng = mla, np.random.default_rng(seed)
        pages = 40000
        self.cache = torch.zeros(pages, 64, 576, device="cuda", dtype=torch.bfloat16)
        self.cache[-POOL:] = torch.randn(POOL, 64, 576, device="cuda", generator=gen).to(
            torch.bfloat16)
        self.refs = torch.ones(pages, dtype=torch.int32, device="cuda")
        self.refs[-POOL:] = 0
        self.table = torch.full((ROWS, MOST), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.model = np.zeros(ROWS, int)
        self.every = dev_i32(np.arange(ROWS))
        self.new = torch.zeros_like(self.lens)
        self.gone = dev_i32(np.arange(0, ROWS, 7))
        q = (0.6 * torch.randn(ROWS, HEADS, 576, device="cuda", generator=gen)).to(torch.bfloat16)
        self.q = q[..., :512].contiguous(), q[..., 512:].contiguous()
        self.q_bits = host_bits(q)
        self.x = torch.randn(ROWS, 576, device="cuda", generator=gen).to(torch.bfloat16)
        self.ones = torch.ones(512, device="cuda", dtype=torch.bfloat16)
        self.starts = dev_i32(np.arange(ROWS + 1))
        self.ws_pages = mla.alloc_workspace(mla.pages_workspace_size(pages, ROWS))
        self.ws_norm = mla.alloc_workspace(mla.WS_HEADER_BYTES)
        self.ws = [mla.alloc_workspace(mla.decode_workspace_size(ROWS, HEADS, CTX))
                   for _ in range(2)]
        self.out = [torch.empty_like(self.q[0]) for _ in range(3)]
        self.lse = [torch.empty(ROWS, HEADS, device="cuda") for _ in range(3)]
        assert mla.decode_plan(ROWS, HEADS, CTX)[0] == 0  # the balanced schedule

    def turn(self, what):
        """The lengths change, and decode follows at once."""
        m, state = self.mla, (self.refs, self.table, self.lens)
        m.pages_free(*state, self.gone, self.ws_pages)
        if what != "free":
            m.pages_extend(*state, self.every, self.new, self.ws_pages)
        if what == "append":
            # a kernel between: it starts its successors early too
            m.norm_rope_append(self.x, None, self.ones, self.starts, self.lens, self.table,
                               self.cache, workspace=self.ws_norm)
        args = (*self.q, self.cache, self.table, self.lens, CTX, R.SCALE, 0)
        m.decode_attention(*args, self.out[0], self.lse[0], self.ws[0])
        if what == "free":  # the lengths change between two plans too
            m.pages_extend(*state, self.every, self.new, self.ws_pages)
        m.decode_prepare(self.lens, ROWS, HEADS, CTX, 0, self.ws[1])
        m.decode_attention_prepared(*args, self.out[1], self.lse[1], self.ws[1])
        m.decode_attention_noalloc(*args, self.out[2], self.lse[2])

    def choose(self):
        """New lengths for the next turn; returns those after the release and after the growth."""
        freed = self.model.copy()
        freed[::7] = 0
        grown = np.minimum(CTX, freed + self.rng.integers(1, 300, ROWS))
        grown[self.rng.random(ROWS) < 0.2] = CTX
        grown = np.maximum(grown, freed)
        self.new.copy_(dev_i32(grown))
        self.model = grown
        return freed, grown

    def check(self, freed, grown, what):
        m = self.mla
        for ws in (self.ws_pages, self.ws_norm, *self.ws):
            assert m.check_device_status(ws) == 0
        assert np.array_equal(self.lens.cpu().numpy(), grown)
        table = self.table.cpu().numpy()
        used = np.unique(table[table >= 0])
        small = np.full_like(table, -1)
        small[table >= 0] = np.searchsorted(used, table[table >= 0])
        cache = host_f64_from_bf16(self.cache[torch.from_numpy(used).long().cuda()])
        for k, (out, lse) in enumerate(zip(self.out, self.lse)):
            lens = freed if what == "free" and k == 0 else grown
            d = dict(heads=HEADS, counts=[1] * ROWS, lens=list(lens), window=0, sinks=0,
                     scale=R.SCALE, table=small, starts=np.arange(ROWS + 1), q=self.q_bits,
                     cache=cache)
            ref, lref, tol, ltol = R.attention(d)
            R.assert_within(host_f64_from_bf16(out), ref, tol, "out")
            R.assert_within(lse.cpu().numpy().astype(np.float64), lref, ltol, "lse")


@pytest.mark.parametrize("what", ["free", "extend", "append"])
def test_decode_right_after_the_lengths_change(mla, what):
    s = State(mla, 1)
    for _ in range(3):
        now = s.choose()
        torch.cuda.synchronize()
        s.turn(what)
        torch.cuda.synchronize()
        s.check(*now, what)


@pytest.mark.parametrize("what", ["free", "extend", "append"])
def test_the_same_in_a_replayed_graph(mla, what):
    s = State(mla, 2)
    now = s.choose()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.turn(what)
    torch.cuda.synchronize()
    s.check(*now, what)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.turn(what)
    for _ in range(3):
        now = s.choose()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        s.check(*now, what)


def test_decode_right_after_a_fork(mla):
    """Children get their lengths from the fork; their rows are their parents' ones."""
    s = State(mla, 3)
    lens = 100 + np.arange(ROWS // 2) * 9
    half = dev_i32(np.arange(ROWS // 2))
    other = dev_i32(np.arange(ROWS // 2, ROWS))
    lens_dev = dev_i32(lens)
    torch.cuda.synchronize()
    state = (s.refs, s.table, s.lens)
    mla.pages_extend(*state, half, lens_dev, s.ws_pages)
    mla.pages_fork(*state, half, other, [s.cache[None]], s.ws_pages)
    mla.decode_attention(*s.q, s.cache, s.table, s.lens, CTX, R.SCALE, 0, s.out[0], s.lse[0],
                         s.ws[0])
    torch.cuda.synchronize()
    s.out, s.lse = s.out[:1], s.lse[:1]
    both = np.concatenate([lens, lens])
    s.check(both, both, "fork")
