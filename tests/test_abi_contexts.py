"""Host-side refusals of the calls for long and common contexts. CPU only: every call here returns
before anything is launched (addresses are made up and never read)."""
import ctypes

import pytest

from tests.test_abi_serving import (ATTENTION, ATTENTION_REFUSALS, INVALID, MAX, NORM, P,
                                    UNSUPPORTED, call, check, fp8, mla)

__all__ = ["mla"]

SHARED = ("q_lat q_rope kv num_blocks table max_blocks seqlens group_starts prefix_lens groups B s_q "
          "H max_seqlen scale ws ws_bytes out lse stream").split()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_shared_decode(mla, cache):  # noqa: F811
    name, order = "mla_decode_attention_shared", SHARED
    more = [({"kv": None}, INVALID), ({"kv": P + 4}, INVALID)]
    if cache == "fp8":
        name, order = name + "_fp8", fp8(order)
        more = [({"codes": None}, INVALID), ({"exps": None}, INVALID), ({"exps": P + 8}, INVALID)]
    good = dict(ATTENTION, group_starts=P, prefix_lens=P, groups=1)
    refusals = [r for r in ATTENTION_REFUSALS if r[0] != {"sinks": -1}]
    check(mla, name, order, good, refusals + more + [
        ({"group_starts": None}, INVALID), ({"prefix_lens": None}, INVALID),
        ({"group_starts": P + 2}, INVALID), ({"prefix_lens": P + 1}, INVALID),
        ({"groups": 0}, INVALID), ({"groups": -1}, INVALID), ({"groups": 4097}, INVALID),
        ({"s_q": 0}, INVALID), ({"s_q": 9}, UNSUPPORTED), ({"s_q": MAX}, UNSUPPORTED),
        # the schedule's weights would pass 32 bits
        ({"B": 4096, "max_blocks": 1 << 20, "max_seqlen": 1 << 26}, UNSUPPORTED),
    ])


def test_shared_workspace_sizes(mla):  # noqa: F811
    size = mla.decode_shared_workspace_size
    assert size(8, 1, 16, 5000, 2) >= size(8, 1, 16, 100, 2) > mla.WS_HEADER_BYTES
    assert size(9, 1, 16, 5000, 2) >= size(8, 1, 16, 5000, 2)
    assert size(8, 1, 16, 5000, 3) >= size(8, 1, 16, 5000, 2)
    for bad in (dict(B=0), dict(B=4097), dict(s_q=0), dict(s_q=9), dict(H=24), dict(max_seqlen=-1),
                dict(groups=0)):
        with pytest.raises(mla.MLAError):
            size(**dict(dict(B=2, s_q=1, H=16, max_seqlen=9, groups=1), **bad))


ROPE = ("x x_token x_head tokens heads width offset plan pos y y_token y_head rest rest_token "
        "rest_head stream").split()


def test_rope(mla):  # noqa: F811
    good = dict(x=P, x_token=640, x_head=80, tokens=4, heads=8, width=80, offset=16,
                plan=ctypes.byref(mla.rope_plan(64)), pos=P, y=P, y_token=512, y_head=64, rest=P, rest_token=128,
                rest_head=16, stream=None)
    lib, name = mla.lib(), "mla_rope"
    for change, want in [
            *(({k: None}, INVALID) for k in ("x", "plan", "pos", "y")),
            ({"tokens": 0}, INVALID), ({"heads": 0}, INVALID), ({"width": 0}, INVALID),
            ({"offset": -1}, INVALID), ({"offset": 17}, INVALID), ({"width": 79}, INVALID),
            ({"x_token": -1}, INVALID), ({"x_head": -80}, INVALID), ({"y_token": -1}, INVALID),
            ({"y_head": 63}, INVALID), ({"y_token": 8}, INVALID), ({"rest_head": 15}, INVALID),
            ({"rest_token": 0}, INVALID), ({"x": P + 1}, INVALID), ({"y": P + 1}, INVALID),
            ({"rest": P + 1}, INVALID), ({"pos": P + 2}, INVALID),
            ({"tokens": (1 << 24) + 1}, UNSUPPORTED), ({"heads": 4097}, UNSUPPORTED),
            ({"width": 4097, "rest_head": 5000, "rest_token": 50000}, UNSUPPORTED),
            ({"offset": MAX}, INVALID)]:
        assert call(lib, name, ROPE, good, **change) == want, change
    for bad in (dict(rot=0), dict(rot=-2), dict(rot=258), dict(rot=2 ** 31 - 1), dict(layout=2),
                dict(magnitude=float("inf")), dict(magnitude=float("nan")), dict(freq=-1e-3),
                dict(freq=70000.0), dict(freq=float("nan"))):
        p = mla.rope_plan(64)
        for k, v in bad.items():
            if k == "freq":
                p.freq[1] = v
            else:
                setattr(p, k, v)
        assert call(lib, name, ROPE, good, plan=ctypes.byref(p)) == INVALID, bad


def test_rope_plan(mla):  # noqa: F811
    good = dict(rot=64, theta=10000.0, scaling="yarn", factor=4.0, original=4096, fast=32.0, slow=1.0)
    plan = mla.rope_plan(**good)
    assert plan.rot == 64 and plan.layout == 0 and abs(plan.magnitude - 1.1386294) < 1e-6
    # fast pairs stay, slow ones are divided by the factor
    assert plan.freq[0] == 1.0 and abs(plan.freq[31] * 4 / 10000.0 ** (-62 / 64) - 1) < 1e-12
    assert all(a > b > 0 for a, b in zip(plan.freq[:31], plan.freq[1:32]))
    assert mla.rope_plan(64, magnitude=2.0).magnitude == 2.0
    assert mla.rope_plan(64, layout="half").layout == 1
    # the slowest pair of the changed base is the one of positions divided by the factor
    ntk = mla.rope_plan(64, scaling="ntk", factor=8.0)
    assert abs(ntk.freq[31] * 8 / 10000.0 ** (-62 / 64) - 1) < 1e-12 and ntk.freq[0] == 1.0
    for bad in (dict(rot=0), dict(rot=3), dict(rot=-2), dict(theta=0.0), dict(theta=-1.0),
                dict(theta=float("inf")), dict(factor=0.0), dict(factor=float("nan")),
                dict(original=0), dict(slow=0.0), dict(fast=1.0), dict(fast=float("inf")),
                dict(theta=1.0)):
        with pytest.raises(mla.MLAError) as e:
            mla.rope_plan(**dict(good, **bad))
        assert e.value.code == INVALID, bad
    with pytest.raises(mla.MLAError) as e:
        mla.rope_plan(258)
    assert e.value.code == UNSUPPORTED
    for bad in (dict(scaling="more"), dict(layout="both")):
        with pytest.raises(ValueError):
            mla.rope_plan(**dict(good, **bad))


READ = "kv num_blocks table max_blocks first row_starts B rows out ws ws_bytes stream".split()
CACHES = {"": ("kv",), "_fp8": ("codes", "exps"), "_fp4": ("codes", "scales", "exps", "keys")}


def over(order, kind):
    return [x for k in order for x in (CACHES[kind] if k == "kv" else (k,))]


@pytest.mark.parametrize("kind", list(CACHES))
def test_read_kv(mla, kind):  # noqa: F811
    good = dict(kv=P, codes=P, exps=P, scales=P, keys=P, num_blocks=9, table=P, max_blocks=4, first=P,
                row_starts=P, B=2, rows=100, out=P, ws=P, ws_bytes=256, stream=None)
    check(mla, "mla_read_kv" + kind, over(READ, kind), good, [
        *(({k: None}, INVALID) for k in ("table", "row_starts", "out", "ws", *CACHES[kind])),
        ({CACHES[kind][0]: P + 8}, INVALID),
        ({"num_blocks": 0}, INVALID), ({"max_blocks": 0}, INVALID), ({"B": 0}, INVALID),
        ({"B": 4097}, INVALID), ({"rows": 0}, INVALID), ({"first": P + 2}, INVALID),
        ({"row_starts": P + 2}, INVALID), ({"table": P + 1}, INVALID), ({"out": P + 16}, INVALID),
        ({"ws": P + 64}, INVALID), ({"num_blocks": (1 << 24) + 1}, UNSUPPORTED),
        ({"max_blocks": 1 << 25}, UNSUPPORTED), ({"rows": (1 << 30) + 1}, UNSUPPORTED),
    ])


@pytest.mark.parametrize("kind", list(CACHES))
def test_norm_rope_append_plans(mla, kind):  # noqa: F811
    plan = mla.rope_plan(64)
    narrow = mla.rope_plan(32)
    broken = mla.rope_plan(64)
    broken.freq[3] = -1.0
    good = dict(x=P, ldx=640, q_lora=64, w_q=P, w_kv=P, eps=1e-6, q_starts=P, seqlens=P, B=2,
                tokens=5, table=P, max_blocks=4, kv=P, codes=P, exps=P, scales=P, keys=P,
                num_blocks=9, theta=ctypes.byref(plan), c_q=P, ws=P, ws_bytes=256, stream=None)
    name = "mla_norm_rope_append" + ("_fp4" if kind == "_fp4" else "_scaled" + kind)
    check(mla, name, over(NORM, kind), good, [
        *(({k: None}, INVALID) for k in ("x", "w_q", "w_kv", "q_starts", "seqlens", "table", "c_q",
                                         "ws", "theta", *CACHES[kind])),
        ({"theta": ctypes.byref(narrow)}, INVALID), ({"theta": ctypes.byref(broken)}, INVALID),
        ({"B": 0}, INVALID), ({"tokens": 0}, INVALID), ({"q_lora": 60}, INVALID),
        ({"ldx": 632}, INVALID), ({"eps": -1e-6}, INVALID), ({CACHES[kind][0]: P + 8}, INVALID),
        ({"ws": P + 64}, INVALID), ({"max_blocks": 1 << 25}, UNSUPPORTED),
    ] + ([({"scales": P + 8}, INVALID), ({"keys": P + 4}, INVALID)] if kind == "_fp4" else []))
