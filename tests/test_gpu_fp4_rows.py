"""What the 4-bit append quantises: the exact latent norm to the nearest bf16, which the bf16 append's own row,
formed in fp32, may miss by a step where the value lies next to a border."""
import numpy as np
import pytest
import torch

from mla_latent_kv_13_gb300 import synth
from tests import fp4_ref as F
from tests.helpers import dev_bf16, dev_i32, host_bits
from tests.test_gpu_fp4 import EPS, append, cache4, inputs, mla, to_bf16

__all__ = ["mla"]
pytestmark = pytest.mark.gpu


def test_rows(mla):  # noqa: F811
    d = inputs(41, [3000], [3000], 0)
    x, w = (synth.bf16_bits_to_f64(d[k]) for k in ("x", "w_kv"))
    exact = x[:, :512] / np.sqrt((x[:, :512] ** 2).mean(-1, keepdims=True) + EPS) * w
    nearest = to_bf16(exact)
    plan = mla.rope_plan()
    at = [np.arange(3000) // 64, np.arange(3000) % 64]
    at[0] = d["table"][0, at[0]]

    bf16 = torch.zeros(d["pool"], 64, 576, dtype=torch.bfloat16, device="cuda")
    _, ws = mla.norm_rope_append_scaled(dev_bf16(d["x"]), None, dev_bf16(d["w_kv"]), dev_i32(d["starts"]),
                                        dev_i32(d["lens"]), dev_i32(d["table"]), bf16, plan, EPS)
    assert mla.check_device_status(ws) == 0
    row = synth.bf16_bits_to_f64(host_bits(bf16))[at[0], at[1], :512]
    # half a step (2^-9 of the power of two above the value), and the fp32 arithmetic: a sum of 512 squares
    # by eights and halves, a division, a root and two products, each rounding 2^-24, well within 2^-19
    step = 2.0 ** (np.frexp(exact)[1] - 8.0)
    assert np.all(np.abs(row - exact) <= step / 2 + 2.0 ** -19 * np.abs(exact))
    off = row != nearest
    assert np.all(np.abs(row - nearest)[off] <= step[off] * 1.0001)

    cache = cache4(d["pool"])
    _, status = append(mla, d, cache, plan)
    assert status == 0
    codes, scales, exps = F.quantize(nearest)
    got = F.unpack(cache[0].cpu().numpy())[at[0], at[1]]
    got[got == 8] = 0  # a zero's sign is not specified
    assert np.array_equal(got, codes)
    assert np.array_equal(cache[1].cpu().numpy()[at[0], at[1]].astype(int), scales)
    assert np.array_equal(cache[2].cpu().numpy()[at[0], at[1]].astype(int), exps)
    print(f"{off.sum()} of {off.size} values of the bf16 rows are a step off")
