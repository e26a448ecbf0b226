"""The ragged serving calls run together as a server would: prompts get pages, are projected,
normed and appended, attend in one ragged call, are forked, one ends, the pool is compacted, and the
rest decodes under a window. Every stage is checked against its 64-bit form on the inputs
that it really got."""
import numpy as np
import pytest
import torch

from mla_latent_kv_13_gb300 import synth
from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_f64_from_bf16

pytestmark = pytest.mark.gpu

DM, QL, H, PAGES, ROWS, MOST = 256, 128, 16, 40, 8, 6
EPS, THETA = 1e-6, 10000.0


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


class Server:
    """The state a server keeps, and for each sequence the cache rows it should hold."""

    def __init__(self, mla, fp8):
        self.mla, self.fp8 = mla, fp8
        rng = np.random.default_rng(0)
        self.rng = rng

        def w(*shape):
            return R.bf16_bits((rng.standard_normal(shape) / np.sqrt(shape[-1])).astype(np.float32))

        self.w = {k: dev_bf16(w(*s)) for k, s in dict(
            down=(QL + 576, DM), uq=(H * 128, QL), qr=(H * 64, QL), uk=(H, 128, 512),
            uv=(H, 128, 512), o=(DM, H * 128)).items()}
        self.w_q = dev_bf16(R.bf16_bits(1 + 0.2 * rng.standard_normal(QL).astype(np.float32)))
        self.w_kv = dev_bf16(R.bf16_bits(1 + 0.2 * rng.standard_normal(512).astype(np.float32)))
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.table = torch.full((ROWS, MOST), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        if fp8:
            self.cache = (torch.full((PAGES, 64, 576), 0x7F, dtype=torch.uint8, device="cuda"),
                          torch.zeros((PAGES, 64), dtype=torch.int8, device="cuda"))
        else:
            self.cache = (torch.full((PAGES, 64, 576), float("nan"), dtype=torch.bfloat16,
                                     device="cuda"),)
        self.pools = [c[None] for c in self.cache]
        self.ws = mla.alloc_workspace(max(mla.pages_workspace_size(PAGES, ROWS),
                                          mla.chunk_workspace_size(ROWS, 400, H, 64 * MOST)))
        self.held = {}

    def rows_of(self, b):
        n = int(self.lens[b])
        j = torch.arange(n, device="cuda")
        page = self.table[b, j // 64].long()
        if self.fp8:
            c, e = (t[page, j % 64].cpu().numpy() for t in self.cache)
            return R.fp8_values(c, e)
        return host_f64_from_bf16(self.cache[0][page, j % 64])

    def ok(self):
        assert self.mla.check_device_status(self.ws) == 0

    def same_rows(self):
        for b, rows in self.held.items():
            assert int(self.lens[b]) == len(rows)
            assert np.array_equal(self.rows_of(b), rows), b

    def step(self, batch, new, window=0, sinks=0):
        """`new` tokens for each sequence of `batch`; returns the layer's outputs."""
        m, total = self.mla, sum(new)
        lens = [int(self.lens[b]) + n for b, n in zip(batch, new)]
        m.pages_extend(self.refs, self.table, self.lens, dev_i32(batch), dev_i32(lens), self.ws)
        starts = dev_i32(np.concatenate([[0], np.cumsum(new)]))
        table, seq = self.table[batch].contiguous(), self.lens[batch].contiguous()
        hid = dev_bf16(R.bf16_bits(self.rng.standard_normal((total, DM)).astype(np.float32)))
        x = (hid.float() @ self.w["down"].float().T).to(torch.bfloat16)
        call = m.norm_rope_append_fp8 if self.fp8 else m.norm_rope_append
        c_q, _ = call(x, self.w_q, self.w_kv, starts, seq, table, *self.cache, THETA, EPS,
                      workspace=self.ws)
        pos = np.concatenate([np.arange(n - k, n) for n, k in zip(lens, new)])
        q_lat, q_rope, ws = m.absorb_q_latent(c_q, self.w["uq"], self.w["qr"], self.w["uk"],
                                              dev_i32(pos), THETA)
        assert m.check_device_status(ws) == 0
        self.check_query(c_q, q_lat, q_rope, pos)
        if window:
            call = m.decode_attention_window_fp8 if self.fp8 else m.decode_attention_window
            o, lse, _ = call(q_lat, q_rope, *self.cache, table, seq, 64 * MOST, window, sinks,
                             R.SCALE, workspace=self.ws)
        else:
            call = m.chunk_attention_fp8 if self.fp8 else m.chunk_attention
            o, lse, _ = call(q_lat, q_rope, *self.cache, table, starts, seq, 64 * MOST, R.SCALE,
                             workspace=self.ws)
        self.ok()
        # the rows appended, and those from before
        self.check_rows(x, batch, new, lens)
        d = dict(heads=H, counts=new, lens=lens, window=window, sinks=sinks, scale=R.SCALE,
                 starts=starts.cpu().numpy(), tokens=total, table=table.cpu().numpy(),
                 q=torch.cat([q_lat, q_rope], -1).view(torch.int16).cpu().numpy().view(np.uint16))
        if self.fp8:
            d["cache"] = R.fp8_values(*(t.cpu().numpy() for t in self.cache))
        else:
            d["cache"] = host_f64_from_bf16(self.cache[0])
        ref, lref, tol, ltol = R.attention(d)
        R.assert_within(host_f64_from_bf16(o), ref, tol, "out")
        R.assert_within(lse.cpu().numpy().astype(np.float64), lref, ltol, "lse")
        y, ws = m.out_absorb(o, self.w["uv"], self.w["o"])
        assert m.check_device_status(ws) == 0
        return y

    def check_query(self, c_q, q_lat, q_rope, pos):
        f = host_f64_from_bf16
        c = f(c_q)
        qn = (c @ f(self.w["uq"]).T).reshape(-1, H, 128)
        ref = np.einsum("thn,hnc->thc", qn, f(self.w["uk"]))
        # q_nope is rounded to bf16 between the products, and the result
        size = np.einsum("thn,hnc->thc", np.abs(qn), np.abs(f(self.w["uk"])))
        tol = R.HALF_STEP_BF16 * (size + np.abs(ref)) * 1.01 + 1e-4 * size
        R.assert_within(f(q_lat), ref, tol, "q_lat")
        r = (c @ f(self.w["qr"]).T).reshape(-1, H, 32, 2)
        z = (r[..., 0] + 1j * r[..., 1]) * np.exp(
            1j * pos[:, None] * THETA ** (-2.0 * np.arange(32) / 64))[:, None, :]
        ref = np.stack([z.real, z.imag], -1).reshape(-1, H, 64)
        tol = R.HALF_STEP_BF16 * np.abs(ref) * 1.01 + 1e-4 * np.repeat(np.abs(z), 2, -1) + 1e-6
        R.assert_within(f(q_rope), ref, tol, "q_rope")

    def check_rows(self, x, batch, new, lens):
        x = host_f64_from_bf16(x)[:, QL:]
        w = host_f64_from_bf16(self.w_kv)
        at = 0
        for b, n, length in zip(batch, new, lens):
            old = self.held.get(b, np.zeros((0, 576)))
            rows = self.rows_of(b)
            assert len(rows) == length and np.array_equal(rows[:len(old)], old)
            got, v = rows[len(old):], x[at:at + n]
            ref = np.empty_like(v)
            c = v[:, :512]
            ref[:, :512] = c / np.sqrt((c * c).mean(-1, keepdims=True) + EPS) * w
            z = (v[:, 512::2] + 1j * v[:, 513::2]) * np.exp(
                1j * np.arange(length - n, length)[:, None] * THETA ** (-2.0 * np.arange(32) / 64))
            ref[:, 512::2], ref[:, 513::2] = z.real, z.imag
            slack = 2.0 ** -19 * (np.abs(ref) + 10)
            if self.fp8:  # half a step of 3 bits, or of the scale's subnormals
                top = np.abs(ref).max(1, keepdims=True)
                tol = 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * 2 * top / 448 + slack
            else:
                tol = R.HALF_STEP_BF16 * np.abs(ref) + slack
            R.assert_within(got, ref, tol, "rows")
            self.held[b] = rows
            at += n


@pytest.mark.parametrize("fp8", [False, True])
def test_a_server_s_life(mla, fp8):
    s = Server(mla, fp8)
    # three prompts in one ragged call, then more of them beside a new one
    s.step([0, 3, 5], [70, 130, 64])
    s.step([3, 1, 0], [1, 90, 33])
    # samples of two of them
    mla.pages_fork(s.refs, s.table, s.lens, dev_i32([0, 3, 0]), dev_i32([2, 4, 6]), s.pools, s.ws)
    s.ok()
    for parent, child in ((0, 2), (3, 4), (0, 6)):
        s.held[child] = s.held[parent]
    s.same_rows()
    # all decode, each its own next token, under a window
    s.step([0, 1, 2, 3, 4, 5, 6], [1] * 7, window=50, sinks=4)
    s.same_rows()
    # two end, the pool is packed, the rest goes on
    mla.pages_free(s.refs, s.table, s.lens, dev_i32([0, 5]), s.ws)
    for b in (0, 5):
        del s.held[b]
    _, _, live, _ = mla.pages_compact(s.refs, s.table, s.lens, s.pools, workspace=s.ws)
    s.ok()
    s.same_rows()
    n = live.item()
    assert (s.refs[:n] > 0).all() and (s.refs[n:] == 0).all()
    y = s.step([6, 2, 7, 1, 3], [1, 1, 40, 3, 1])
    s.same_rows()
    assert torch.isfinite(y.float()).all()
