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


def _place(d, pages, seed=0):
    """The same batch in a pool of `pages` pages, at its far end."""
    e = dict(d)
    table = d["table"].copy()
    table[table >= 0] += pages - d["pool"]
    e["table"], e["far"] = table, pages
    return e


def test_far_pages(mla):
    """Page ids whose rows lie past 4 GiB, in 16-bit values past 2^31."""
    pages = 62000  # 4.6 GB
    d = R.attention_case(12, 32, [3, 1], [200, 90], 70, 3)
    far = _place(d, pages)
    pool = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    pool[pages - d["pool"]:] = _cache(d)[0]
    q_lat, q_rope = _q(d)
    out, lse, ws = mla.chunk_attention(q_lat, q_rope, pool, dev_i32(far["table"]),
                                       dev_i32(d["starts"]), dev_i32(d["lens"]), 200, d["scale"],
                                       window=70, sinks=3)
    check(d, out, lse, mla.check_device_status(ws))


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
@pytest.mark.parametrize("fp8", [False, True])
def test_bad_page_is_recorded_and_masked(mla, bad, fp8):
    d = R.attention_case(13, 16, [2, 9, 1], [300, 200, 64], fp8=fp8)
    e = dict(d)
    e["table"] = d["table"].copy()
    e["table"][0, 2] = bad
    out, lse, st = run_chunk(mla, e)
    assert st == 4
    # the reference without rows 128 .. 191 of sequence 0
    keep = R.visible
    try:
        def without(length, count, i, window, sinks):
            j = keep(length, count, i, window, sinks)
            return j[(j < 128) | (j >= 192)] if length == 300 else j
        R.visible = without
        check(d, out, lse)
    finally:
        R.visible = keep


def test_lengths_out_of_range_are_recorded_and_clamped(mla):
    d = R.attention_case(14, 16, [2, 1], [100, 64])
    q_lat, q_rope = _q(d)
    args = (q_lat, q_rope, *_cache(d), dev_i32(d["table"]), dev_i32(d["starts"]))
    out, lse, ws = mla.chunk_attention(*args, dev_i32([105, -3]), 100, d["scale"])
    assert mla.check_device_status(ws) == 4
    e = dict(d, lens=[100, 0])
    check(e, out, lse)
    win = R.attention_case(14, 16, [1, 1], [100, 64], 50, 2)
    q_lat, q_rope = _q(win)
    o, l, ws = mla.decode_attention_window(q_lat, q_rope, *_cache(win), dev_i32(win["table"]),
                                           dev_i32([101, -1]), 100, 50, 2, win["scale"])
    assert mla.check_device_status(ws) == 4
    check(dict(win, lens=[100, 0]), o, l)


@pytest.mark.parametrize("starts", [[0, 3, 2], [0, 2, 99], [-1, 1, 2], [3, 3, 2]])
def test_token_ranges_that_do_not_ascend_write_nothing(mla, starts):
    d = R.attention_case(15, 16, [2, 1], [100, 64])
    q_lat, q_rope = _q(d)
    out = torch.full((3, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 16), 7.0, device="cuda")
    _, _, ws = mla.chunk_attention(q_lat, q_rope, *_cache(d), dev_i32(d["table"]), dev_i32(starts),
                                   dev_i32(d["lens"]), 100, d["scale"], out=out, lse=lse)
    assert mla.check_device_status(ws) == 4
    assert (out == 7).all() and (lse == 7).all()


def test_rows_before_the_first_sequence_are_kept(mla):
    d = R.attention_case(16, 64, [2, 1], [100, 64], pad=4)
    d["q"] = np.roll(d["q"], 3, axis=0)
    out = torch.full((7, 64, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((7, 64), 7.0, device="cuda")
    e = dict(d, starts=d["starts"] + 3, tokens=7)
    o, l, st = run_chunk(mla, e, out=out, lse=lse)
    assert st == 0 and (o[:3] == 7).all() and (l[:3] == 7).all() and (o[6:] == 7).all()
    ref, lref, tol, ltol = R.attention(e)
    R.assert_within(host_f64_from_bf16(o)[3:6], ref[3:6], tol[3:6], "out")
    R.assert_within(l.cpu().numpy().astype(np.float64)[3:6], lref[3:6], ltol[3:6], "lse")


def test_empty_batches(mla):
    for heads in (16, 128):
        d = R.attention_case(17, heads, [2, 0, 1], [0, 5, 0])
        out, lse, st = run_chunk(mla, d)
        assert st == 0 and (out == 0).all() and torch.isneginf(lse).all()
        d = R.attention_case(17, heads, [1, 1], [0, 0], 5, 1)
        out, lse, st = run_window(mla, d, 1)
        assert st == 0 and (out == 0).all() and torch.isneginf(lse).all()
    d = R.attention_case(17, 16, [0, 0], [70, 5], pad=1)
    out, lse, st = run_chunk(mla, d)
    assert st == 0


def test_more_sequences_than_threads(mla):
    # 4096 sequences; all but a few bring nothing
    counts = [1 if b % 500 == 3 else 0 for b in range(4096)]
    d = R.attention_case(18, 16, counts, [5 + b % 90 for b in range(4096)])
    check(d, *run_chunk(mla, d))


def test_more_items_than_threads(mla):
    d = R.attention_case(19, 128, [700, 800, 3], [700, 900, 66])
    out, lse, st = run_chunk(mla, d)
    assert st == 0
    # every 40th token of the 1503 against the reference
    keep = [t for t in range(1503) if t % 40 == 0 or t > 1499]
    ref, lref, tol, ltol = R.attention(d, only=set(keep))
    R.assert_within(host_f64_from_bf16(out)[keep], ref[keep], tol[keep], "out")
    R.assert_within(lse.cpu().numpy().astype(np.float64)[keep], lref[keep], ltol[keep], "lse")


def test_other_stream_and_replayed_graphs(mla):
    """Two graphs that share a workspace, replayed in turn with new inputs in the same places."""
    d = R.attention_case(20, 32, [5, 1, 40], [300, 700, 90])
    w = R.attention_case(21, 32, [1, 1], [300, 700], 100, 4)
    side = torch.cuda.Stream()
    q_lat, q_rope = _q(d)
    cache, table = _cache(d), dev_i32(d["table"])
    starts, lens = dev_i32(d["starts"]), dev_i32(d["lens"])
    wq, wcache, wtable, wlens = _q(w), _cache(w), dev_i32(w["table"]), dev_i32(w["lens"])
    need = max(mla.chunk_workspace_size(3, 46, 32, 700),
               mla.decode_window_workspace_size(2, 1, 32, 700, 100, 4))
    ws = mla.alloc_workspace(need)
    out, lse = torch.zeros_like(q_lat), torch.zeros(46, 32, device="cuda")
    wout, wlse = torch.zeros_like(wq[0]), torch.zeros(2, 32, device="cuda")
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: mla.chunk_attention(q_lat, q_rope, *cache, table, starts, lens, 700,
                                             d["scale"], out=out, lse=lse, workspace=ws,
                                             stream=side),
                 lambda: mla.decode_attention_window(*wq, *wcache, wtable, wlens, 700, 100, 4,
                                                     w["scale"], out=wout, lse=wlse, workspace=ws,
                                                     stream=side)):
        call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        graphs.append(g)
    for turn in range(2):
        out.zero_(), wout.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert mla.check_device_status(ws) == 0
        check(d, out, lse)
        check(w, wout, wlse)
        # new queries and lengths in place
        d = R.attention_case(20, 32, [5, 1, 40], [300, 700, 90])
        d["q"] = d["q"][::-1].copy()
        q_lat.copy_(_q(d)[0]), q_rope.copy_(_q(d)[1])


def test_two_streams_at_once(mla):
    cases = [R.attention_case(30 + k, 64, [9, 30, 1], [500, 800, 1500]) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    held = []
    for d in cases:
        held.append([*_q(d), *_cache(d), dev_i32(d["table"]), dev_i32(d["starts"]),
                     dev_i32(d["lens"])])
    wss = [mla.alloc_workspace(mla.chunk_workspace_size(3, 40, 64, 1500)) for _ in cases]
    outs = [(torch.zeros(40, 64, 512, dtype=torch.bfloat16, device="cuda"),
             torch.zeros(40, 64, device="cuda")) for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, s in enumerate(streams):
            mla.chunk_attention(*held[k], 1500, cases[k]["scale"], out=outs[k][0], lse=outs[k][1],
                                workspace=wss[k], stream=s)
    torch.cuda.synchronize()
    for d, (o, l), ws in zip(cases, outs, wss):
        check(d, o, l, mla.check_device_status(ws))


def test_wide_exponents_of_an_fp8_cache(mla):
    """Rows from 2^-40 to 2^20 in one cache: their factors take one or two exact steps."""
    d = R.attention_case(22, 16, [4, 1], [130, 200], fp8=True, size=0.01)
    rng = np.random.default_rng(1)
    d["exps"] = rng.integers(-47, 13, d["exps"].shape).astype(np.int8)
    live = ~(d["codes"] == 0x7F).all(-1)
    vals = R.fp8_values(np.where(live[..., None], d["codes"], 0), d["exps"])
    d["cache"] = vals
    d["q"] = R.bf16_bits(1e-6 * rng.standard_normal(d["q"].shape).astype(np.float32))
    check(d, *run_chunk(mla, d))


@pytest.mark.parametrize("chunk", [False, True])
def test_longest_sequence(mla, chunk):
    """Positions up to the last of 32 bits: what a window of 70 rows and 3 sinks see moves up by
    whole pages, and the answer stays."""
    d = R.attention_case(31, 16, [2], [383], 70, 3)  # 383 and 2^31 - 1 end a page alike
    most = 1 << 25
    table = torch.full((1, most), -1, dtype=torch.int32, device="cuda")
    table[0, :1] = dev_i32(d["table"][0, :1])
    table[0, most - 5:] = dev_i32(d["table"][0, 1:])
    q_lat, q_rope = _q(d)
    lens, last = dev_i32([2 ** 31 - 1]), 2 ** 31 - 1
    if chunk:
        out, lse, ws = mla.chunk_attention(q_lat, q_rope, *_cache(d), table, dev_i32([0, 2]), lens,
                                           last, d["scale"], window=70, sinks=3)
    else:
        out, lse, ws = mla.decode_attention_window(q_lat[None], q_rope[None], *_cache(d), table, lens,
                                                   last, 70, 3, d["scale"])
    check(d, out.reshape(2, 16, 512), lse.reshape(2, 16), mla.check_device_status(ws))


def test_numbers_from_numpy(mla):
    """Sizes and scales of numpy's types, 32-bit ones too, are taken as python's own."""
    d = R.attention_case(32, 16, [1, 1], [90, 200], 64, 2)
    d["scale"] = 0.125
    want = [run_window(mla, d, 1)[0], run_chunk(mla, d)[0]]
    d.update(scale=np.float32(0.125), window=np.int32(64), sinks=np.int64(2),
             lens=[np.int32(90), np.int32(200)])
    got = [run_window(mla, d, 1, np.int64(0))[0], run_chunk(mla, d)[0]]
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))


# Chunks run in fixed ranges or by the schedule (include/mla.h has one contract for both): shapes of
# either, with items cut into many parts, few parts and none.
MODES = {
    "ranges of many sequences": (16, [b % 3 for b in range(36)], [70 * (b % 8) + 3 for b in range(36)]),
    "whole items of many sequences": (16, [1 + b % 3 for b in range(45)], [9 * b + 3 for b in range(45)]),
    "ranges of one long item": (32, [3], [6000]),
    "scheduled cut items": (128, [3, 90], [700, 600]),
    "scheduled parts of one long item": (16, [8], [50100]),
    "scheduled empty and long": (16, [1] * 90 + [0, 20], [b for b in range(90)] + [7, 3000]),
}


@pytest.mark.parametrize("name", list(MODES))
@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_modes(mla, name, fp8):
    heads, counts, lens = MODES[name]
    d = R.attention_case(33, heads, counts, lens, fp8=fp8)
    check(d, *run_chunk(mla, d))


@pytest.mark.parametrize("more", [0, 100])  # fixed ranges; scheduled
def test_wrong_ranges_and_lengths_in_either_mode(mla, more):
    counts, lens = [2, 0, 1] + [1] * more, [100, 64, 70] + [9] * more
    d = R.attention_case(34, 16, counts, lens)
    q_lat, q_rope = _q(d)
    T = d["tokens"]
    args = (q_lat, q_rope, *_cache(d), dev_i32(d["table"]))
    # a length out of range of a sequence without tokens
    out, lse, ws = mla.chunk_attention(*args, dev_i32(d["starts"]), dev_i32([100, 999] + lens[2:]),
                                       100, d["scale"])
    check(d, out, lse)
    assert mla.check_device_status(ws) == 4
    for at, wrong in ((1, -1), (2, T + 1), (3, 1), (len(counts), T + 1)):
        starts = d["starts"].copy()
        starts[at] = wrong
        out = torch.full((T, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, 16), 7.0, device="cuda")
        _, _, ws = mla.chunk_attention(*args, dev_i32(starts), dev_i32(lens), 100, d["scale"], out=out,
                                       lse=lse)
        assert mla.check_device_status(ws) == 4
        assert (out == 7).all() and (lse == 7).all()


def test_a_workspace_serves_shorter_sequences(mla):
    for heads, tokens, B in ((16, 8, 1), (16, 300, 40), (128, 70, 70)):
        sizes = [mla.chunk_workspace_size(B, tokens, heads, n) for n in range(0, 60000, 500)]
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [16, 128])
def test_one_visible_row_is_returned(mla, heads, fp8):
    """Softmax over one row is 1: its latent comes back bit for bit, however it is reached."""
    d = R.attention_case(35, heads, [1] * 5, [1, 64, 65, 129, 900], 1, 0, fp8=fp8)
    rows = [d["cache"][d["table"][b, (n - 1) // 64], (n - 1) % 64, :512] for b, n in enumerate(d["lens"])]
    for run in (lambda: run_window(mla, d, 1), lambda: run_window(mla, d, 1, 3),
                lambda: run_chunk(mla, d)):
        out, lse, st = run()
        got = host_f64_from_bf16(out)
        assert st == 0
        for b, row in enumerate(rows):
            assert np.array_equal(got[b], np.broadcast_to(row, (heads, 512)))
    # the first token of a prompt
    d = R.attention_case(36, heads, [3, 1], [3, 1], fp8=fp8)
    got = host_f64_from_bf16(run_chunk(mla, d)[0])
    for t, b in ((0, 0), (3, 1)):
        assert np.array_equal(got[t], np.broadcast_to(d["cache"][d["table"][b, 0], 0, :512], (heads, 512)))


def test_few_visible_rows_lose_little(mla):
    """Up to four visible rows in one tile: the top weight is 1, and against the output's own rounding
    the others' adds under a quarter (each is off by half a step of bf16, 2^-8 of at most half the
    sum, and what they weigh is independent: 1.11 times in expectation over many rows)."""
    for window, fp8 in ((2, False), (3, True), (4, False)):
        d = R.attention_case(37, 64, [1] * 40, [10 + 5 * b for b in range(40)], window, 0, fp8=fp8)
        out, _, st = run_window(mla, d, 1)
        ref = R.attention(d)[0]
        got = host_f64_from_bf16(out)
        plain = torch.from_numpy(ref).to(torch.bfloat16).double().numpy()
        assert st == 0
        assert np.linalg.norm(got - ref) <= 1.25 * np.linalg.norm(plain - ref)
