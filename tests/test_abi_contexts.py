"""Host-side refusals of the calls for long and common contexts. CPU only: every call here returns
before anything is launched (addresses are made up and never read)."""
import pytest

from tests.test_abi_serving import (ATTENTION, ATTENTION_REFUSALS, INVALID, MAX, P, UNSUPPORTED,
                                    check, fp8, mla)

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
