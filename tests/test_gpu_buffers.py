"""Calls on a stream of their own that make their buffers themselves, while the current stream is
busy: what the buffers are filled with may not land on top of the results."""
import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_f64_from_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


class Raw:
    """A stream by its handle alone."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.fixture(params=[False, True], ids=["stream", "handle"])
def side(request):
    s = torch.cuda.Stream()
    yield Raw(s) if request.param else s


def busy():
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about a tenth of a second on the current stream


def test_chunk(mla, side):
    d = R.attention_case(40, 32, [3, 1, 20], [200, 70, 33], pad=5)
    args = (dev_bf16(d["q"][..., :512]), dev_bf16(d["q"][..., 512:]), dev_bf16(d["bits"]),
            dev_i32(d["table"]), dev_i32(d["starts"]), dev_i32(d["lens"]), 200, d["scale"])
    busy()
    out, lse, ws = mla.chunk_attention(*args, stream=side)
    torch.cuda.synchronize()
    assert mla.check_device_status(ws) == 0
    ref, lref, tol, ltol = R.attention(d)
    n = d["tokens"]
    R.assert_within(host_f64_from_bf16(out)[:n], ref[:n], tol[:n], "out")
    R.assert_within(lse.cpu().numpy().astype(np.float64)[:n], lref[:n], ltol[:n], "lse")
    assert (out[n:] == 0).all() and torch.isneginf(lse[n:]).all()


def test_window(mla, side):
    d = R.attention_case(41, 32, [1] * 3, [200, 70, 33], 50, 2)
    args = (dev_bf16(d["q"][..., :512]), dev_bf16(d["q"][..., 512:]), dev_bf16(d["bits"]),
            dev_i32(d["table"]), dev_i32(d["lens"]), 200, 50, 2, d["scale"])
    busy()
    out, lse, ws = mla.decode_attention_window(*args, stream=side)
    torch.cuda.synchronize()
    assert mla.check_device_status(ws) == 0
    ref, lref, tol, ltol = R.attention(d)
    R.assert_within(host_f64_from_bf16(out), ref, tol, "out")
    R.assert_within(lse.cpu().numpy().astype(np.float64), lref, ltol, "lse")


def test_norm(mla, side):
    x = torch.ones(7, 64 + 576, dtype=torch.bfloat16, device="cuda")
    w_q, w_kv = (torch.ones(n, dtype=torch.bfloat16, device="cuda") for n in (64, 512))
    cache = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    args = (x, w_q, w_kv, dev_i32([0, 3, 5]), dev_i32([3, 2]), dev_i32([[0], [1]]), cache)
    busy()
    c_q, ws = mla.norm_rope_append(*args, stream=side)
    torch.cuda.synchronize()
    assert mla.check_device_status(ws) == 0
    # rms of ones is 1 (eps takes 5e-7 of it)
    assert (c_q[:5] == 1).all() and (c_q[5:] == 0).all()


def test_absorbed_query(mla, side):
    rng = np.random.default_rng(0)
    w = [dev_bf16(R.bf16_bits(0.1 * rng.standard_normal(s).astype(np.float32)))
         for s in ((2, 64), (16 * 128, 64), (16 * 64, 64), (16, 128, 512))]
    pos = dev_i32([3, 70])
    want = mla.absorb_q_latent(*w, pos)[:2]
    busy()
    got = mla.absorb_q_latent(*w, pos, stream=side)
    torch.cuda.synchronize()
    assert mla.check_device_status(got[2]) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_pages(mla, side):
    refs, table = dev_i32([0] * 9), dev_i32(-np.ones((3, 4)))
    lens, rows, new = dev_i32([0] * 3), dev_i32([2, 0]), dev_i32([130, 64])
    pool = torch.arange(9, device="cuda").to(torch.int16)[None, :, None].repeat(1, 1, 8)
    busy()
    ws = [mla.pages_extend(refs, table, lens, rows, new, stream=side),
          mla.pages_free(refs, table, lens, rows[:1], stream=side)]
    *_, live, w = mla.pages_compact(refs, table, lens, [pool], stream=side)
    torch.cuda.synchronize()
    assert all(mla.check_device_status(k) == 0 for k in (*ws, w))
    assert live.item() == 1 and refs.tolist() == [1] + [0] * 8
    assert lens.tolist() == [64, 0, 0] and table[0, 0].item() == 0
    assert pool[0, 0, 0].item() == 3  # where the 64 rows were
