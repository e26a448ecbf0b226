"""Chunk attention over the paged cache and decode with a sliding window and sinks, through the
C ABI, against the plain 64-bit form (tests/rows_ref.py says how the bounds come about)."""
import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_bits, host_f64_from_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def _cache(d):
    if "codes" in d:
        return (torch.from_numpy(d["codes"]).cuda(), torch.from_numpy(d["exps"]).cuda())
    return (dev_bf16(d["bits"]),)


def _q(d):
    return dev_bf16(d["q"][..., :512]), dev_bf16(d["q"][..., 512:])


def run_chunk(mla, d, **kw):
    q_lat, q_rope = _q(d)
    call = mla.chunk_attention_fp8 if "codes" in d else mla.chunk_attention
    out, lse, ws = call(q_lat, q_rope, *_cache(d), dev_i32(d["table"]), dev_i32(d["starts"]),
                        dev_i32(d["lens"]), max(d["lens"]), d["scale"], window=d["window"],
                        sinks=d["sinks"], **kw)
    return out, lse, mla.check_device_status(ws)


def run_window(mla, d, s_q, splits=0, **kw):
    q_lat, q_rope = (t.reshape(-1, s_q, *t.shape[1:]) for t in _q(d))
    call = mla.decode_attention_window_fp8 if "codes" in d else mla.decode_attention_window
    out, lse, ws = call(q_lat, q_rope, *_cache(d), dev_i32(d["table"]), dev_i32(d["lens"]),
                        max(d["lens"]), d["window"], d["sinks"], d["scale"], splits, **kw)
    T = d["tokens"]
    return out.reshape(T, *out.shape[2:]), lse.reshape(T, -1), mla.check_device_status(ws)


def check(d, out, lse, status=0):
    assert status == 0
    ref, lref, tol, ltol = R.attention(d)
    n = d["tokens"]
    R.assert_within(lse.cpu().numpy().astype(np.float64)[:n], lref[:n], ltol[:n], "lse")
    R.assert_within(host_f64_from_bf16(out)[:n], ref[:n], tol[:n], "out")


CHUNKS = {
    "one token each": ([1, 1, 1, 1], [1, 64, 65, 300]),
    "whole prompts": ([5, 64, 1, 130], [5, 64, 1, 130]),
    "mixed": ([1, 9, 0, 33, 1], [500, 9, 77, 64, 1]),
    "more tokens than rows": ([4, 3], [2, 0]),
    "page edges": ([2, 2, 2], [128, 129, 130]),
    "one long": ([40], [1000]),
}


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("name", list(CHUNKS))
def test_chunk(mla, name, heads):
    counts, lens = CHUNKS[name]
    d = R.attention_case(1, heads, counts, lens)
    check(d, *run_chunk(mla, d))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 4), (64, 0), (65, 64), (100, 130),
                                          (1000, 5), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_window(mla, window, sinks, fp8):
    d = R.attention_case(2, 32, [1, 7, 30, 0, 2], [700, 65, 333, 40, 1], window, sinks, fp8=fp8)
    check(d, *run_chunk(mla, d))


@pytest.mark.parametrize("heads,counts,lens", [(16, [9, 1, 20], [9, 700, 129]),
                                               (128, [2, 1], [200, 515])])
def test_chunk_fp8(mla, heads, counts, lens):
    d = R.attention_case(3, heads, counts, lens, fp8=True)
    check(d, *run_chunk(mla, d))


@pytest.mark.parametrize("heads", [16, 128])
def test_chunk_padded_batch_keeps_the_rows_behind(mla, heads):
    d = R.attention_case(4, heads, [3, 12], [90, 40], pad=6)
    out = torch.full((21, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((21, heads), 5.0, device="cuda")
    check(d, *run_chunk(mla, d, out=out, lse=lse))
    assert (out[15:] == 7).all() and (lse[15:] == 5).all()


def test_chunk_spread_scores(mla):
    # scores from -60 to 60: the reference is raised time and again
    d = R.attention_case(5, 64, [17], [900], size=20.0)
    d["cache"][...] *= 1.0
    check(d, *run_chunk(mla, d))


def test_chunk_many_items(mla):
    # far more items than clusters, every share cut somewhere
    d = R.attention_case(6, 128, [60, 1, 70], [200, 300, 150])
    check(d, *run_chunk(mla, d))


def test_chunk_is_the_same_every_time(mla):
    d = R.attention_case(7, 64, [33, 1, 20], [900, 2000, 300])
    out, lse, _ = run_chunk(mla, d)
    for _ in range(3):
        o, l, _ = run_chunk(mla, d)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)


@pytest.mark.parametrize("heads,s_q", [(16, 1), (16, 8), (32, 3), (64, 2), (128, 1)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_window_decode(mla, heads, s_q, splits):
    lens = [1, 2, 64, 65, 200, 777, 1500]
    d = R.attention_case(8, heads, [s_q] * len(lens), lens, 150, 4)
    check(d, *run_window(mla, d, s_q, splits))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (65, 1), (128, 70), (5000, 0)])
@pytest.mark.parametrize("fp8", [False, True])
def test_window_sizes(mla, window, sinks, fp8):
    lens = [0, 1, 63, 64, 129, 192, 500, 1000]
    d = R.attention_case(9, 64, [1] * len(lens), lens, window, sinks, fp8=fp8)
    check(d, *run_window(mla, d, 1))


def test_window_more_sequences_than_clusters(mla):
    lens = [1 + (37 * k) % 700 for k in range(200)]
    d = R.attention_case(10, 16, [2] * 200, lens, 130, 4)
    check(d, *run_window(mla, d, 2))


def test_wide_window_is_plain_decode(mla):
    lens = [100, 700, 64, 1]
    d = R.attention_case(11, 128, [1] * 4, lens, 10 ** 6, 0)
    out, lse, st = run_window(mla, d, 1)
    check(d, out, lse, st)
    q_lat, q_rope = _q(d)
    o2, l2, _ = mla.decode_attention(q_lat, q_rope, *_cache(d), dev_i32(d["table"]),
                                     dev_i32(lens), 700, d["scale"])
    assert (lse - l2).abs().max() < 1e-4
    assert (out.float() - o2.float()).abs().max() < 0.02
