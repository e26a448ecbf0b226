"""The calls for long and common contexts run together as a server would: a system prompt is kept in
four bits, read back into pages of the pool, forked for many requests whose new tokens are rotated by a
long context's plan, and every request decodes with the prompt's pages multiplied once. Every stage is
checked against its 64-bit form on the inputs that it really got."""
import numpy as np
import pytest
import torch

from tests import fp4_ref as F
from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_f64_from_bf16
from tests.test_gpu_fp4 import cache4, to_bf16

pytestmark = pytest.mark.gpu

QL, H, PAGES, ROWS, MOST, PROMPT = 128, 16, 60, 12, 8, 300
EPS = 1e-6


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def weights(rng):
    def w(*shape):
        return dev_bf16(R.bf16_bits((rng.standard_normal(shape) / np.sqrt(shape[-1])).astype(np.float32)))

    one = {k: dev_bf16(R.bf16_bits(1 + 0.2 * rng.standard_normal(n).astype(np.float32)))
           for k, n in (("w_q", QL), ("w_kv", 512))}
    return dict(one, uq=w(H * 128, QL), qr=w(H * 64, QL), uk=w(H, 128, 512))


def hidden(rng, n):
    return dev_bf16(R.bf16_bits(rng.standard_normal((n, QL + 576)).astype(np.float32)))


def latents(x, w):
    c = host_f64_from_bf16(x)[:, QL:QL + 512]
    return c / np.sqrt((c * c).mean(-1, keepdims=True) + EPS) * host_f64_from_bf16(w["w_kv"])


def turned(pairs, pos, plan):
    """[n, .., 64] of pairs side by side at their positions, and the pairs' lengths."""
    z = pairs[..., 0::2] + 1j * pairs[..., 1::2]
    at = np.exp(1j * pos[:, None] * np.array(plan.freq[:32]))
    z = plan.magnitude * z * at.reshape(len(pos), *[1] * (pairs.ndim - 2), 32)
    return np.stack([z.real, z.imag], -1).reshape(pairs.shape), np.repeat(np.abs(z), 2, -1)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_requests_behind_one_prompt(mla, fp8):
    rng = np.random.default_rng(3)
    w = weights(rng)
    plan = mla.rope_plan(scaling="yarn", factor=40.0, original=4096)
    refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    table = torch.full((ROWS, MOST), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    if fp8:
        cache = (torch.full((PAGES, 64, 576), 0x7F, dtype=torch.uint8, device="cuda"),
                 torch.zeros((PAGES, 64), dtype=torch.int8, device="cuda"))
    else:
        cache = (torch.full((PAGES, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda"),)
    ws = mla.alloc_workspace(max(mla.pages_workspace_size(PAGES, ROWS),
                                 mla.decode_shared_workspace_size(ROWS, 1, H, 64 * MOST, 1)))
    mla.pages_extend(refs, table, lens, dev_i32([0]), dev_i32([PROMPT]), ws)

    # ---- the prompt: into a 4-bit store and from there into the pool's pages; or into the FP8 pool
    x = hidden(rng, PROMPT)
    starts, length = dev_i32([0, PROMPT]), lens[:1].contiguous()
    keys, size = turned(host_f64_from_bf16(x)[:, QL + 512:], np.arange(PROMPT), plan)
    if fp8:
        c_q, _ = mla.norm_rope_append_scaled_fp8(x, w["w_q"], w["w_kv"], starts, length,
                                                 table[:1].contiguous(), *cache, plan, EPS, workspace=ws)
    else:
        store, there = cache4(5), dev_i32([[3, 0, 4, 1, 2]])
        c_q, _ = mla.norm_rope_append_fp4(x, w["w_q"], w["w_kv"], starts, length, there, *store, plan, EPS,
                                          workspace=ws)
        first_pages = table[0, :5].cpu().numpy()
        assert np.array_equal(first_pages, np.arange(5))  # a run of pages: the pool's rows 0 .. 299
        mla.read_kv_fp4(*store, there, None, starts, out=cache[0].view(-1, 576)[:PROMPT], workspace=ws)
        got = host_f64_from_bf16(cache[0].view(-1, 576)[:PROMPT])
        assert np.array_equal(got[:, :512], F.values(*F.quantize(to_bf16(latents(x, w)))))
        assert np.all(np.abs(got[:, 512:] - keys) <= R.HALF_STEP_BF16 * np.abs(keys) + 2.0 ** -19 * size)
    assert mla.check_device_status(ws) == 0

    # ---- nine requests share it
    kids = list(range(1, 10))
    pools = [c[None] for c in cache]
    mla.pages_fork(refs, table, lens, dev_i32([0] * 9), dev_i32(kids), pools, ws)
    assert mla.check_device_status(ws) == 0
    group, prefix = dev_i32([0, 10]), dev_i32([PROMPT])
    for turn in range(3):
        # some bring several tokens first, so that their lengths part
        new = [1 if turn == 2 else 1 + (7 * b + 3 * turn) % 40 for b in range(10)]
        goal = [int(lens[b]) + n for b, n in enumerate(new)]
        mla.pages_extend(refs, table, lens, dev_i32(range(10)), dev_i32(goal), ws)
        rows, seq = table[:10].contiguous(), lens[:10].contiguous()
        x = hidden(rng, sum(new))
        starts = dev_i32(np.concatenate([[0], np.cumsum(new)]))
        append = mla.norm_rope_append_scaled_fp8 if fp8 else mla.norm_rope_append_scaled
        c_q, _ = append(x, w["w_q"], w["w_kv"], starts, seq, rows, *cache, plan, EPS, workspace=ws)
        assert mla.check_device_status(ws) == 0

        # the last token of each: its query, absorbed without a rotation, then turned in place
        last = torch.tensor(np.cumsum(new) - 1, device="cuda")
        c_last = c_q[last].contiguous()
        pos = seq - 1
        q_lat, q_rope, ws_q = mla.absorb_q_latent(c_last, w["uq"], w["qr"], w["uk"], torch.zeros_like(pos))
        assert mla.check_device_status(ws_q) == 0
        plain = host_f64_from_bf16(q_rope)
        mla.rope(q_rope, pos, plan, out=q_rope)
        want, length_of = turned(plain, pos.cpu().numpy(), plan)
        assert np.all(np.abs(host_f64_from_bf16(q_rope) - want) <=
                      R.HALF_STEP_BF16 * np.abs(want) + 2.0 ** -20 * length_of + 1e-30)

        call = mla.decode_attention_shared_fp8 if fp8 else mla.decode_attention_shared
        o, lse, _ = call(q_lat, q_rope, *cache, rows, seq, group, prefix, 64 * MOST, R.SCALE, workspace=ws)
        assert mla.check_device_status(ws) == 0
        value = (R.fp8_values(*(t.cpu().numpy() for t in cache)) if fp8 else host_f64_from_bf16(cache[0]))
        d = dict(heads=H, counts=[1] * 10, lens=goal, window=0, sinks=0, scale=R.SCALE,
                 starts=np.arange(11), tokens=10, table=rows.cpu().numpy(), cache=value,
                 q=torch.cat([q_lat, q_rope], -1).view(torch.int16).cpu().numpy().view(np.uint16))
        ref, lref, tol, ltol = R.attention(d)
        R.assert_within(host_f64_from_bf16(o), ref, tol + 1e-5 * np.abs(ref).max(), "out")
        R.assert_within(lse.cpu().numpy().astype(np.float64), lref, ltol + 1e-5, "lse")

    # ---- half of them end, the pool is packed, and the rest still agree with plain decode
    mla.pages_free(refs, table, lens, dev_i32([1, 3, 5, 7, 9]), ws)
    mla.pages_compact(refs, table, lens, pools, workspace=ws)
    assert mla.check_device_status(ws) == 0
    rows, seq = table[:10].contiguous(), lens[:10].contiguous()
    o, lse, _ = call(q_lat, q_rope, *cache, rows, seq, group, prefix, 64 * MOST, R.SCALE, workspace=ws)
    plain = mla.decode_attention_fp8 if fp8 else mla.decode_attention
    po, plse, _ = plain(q_lat, q_rope, *cache, rows, seq, 64 * MOST, R.SCALE)
    assert mla.check_device_status(ws) == 0
    alive = [0, 2, 4, 6, 8]
    assert torch.isneginf(lse[[1, 3, 5, 7, 9]]).all() and not o[[1, 3, 5, 7, 9]].any()
    assert torch.allclose(lse[alive], plse[alive], atol=1e-3, rtol=0)
    # each within half a step and a little of the same values
    assert (o.double() - po.double())[alive].norm() <= 2 ** -7 * po.double()[alive].norm()
