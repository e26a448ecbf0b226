"""The latent norms over every magnitude that bf16 has: the squares of a row may be past fp32's
range, above or (without eps) below, while the normed row is of the size of its weights."""
import numpy as np
import pytest
import torch

from mla_latent_kv_13_gb300 import synth
from tests import rows_ref as R
from tests.helpers import dev_bf16, dev_i32, host_f64_from_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


POWERS = [-130, -120, -100, -64, -46, -45, -44, -30, -1, 0, 30, 58, 61, 62, 63, 64, 70, 100, 125]


@pytest.mark.parametrize("q_lora", [8, 64, 1536, 4000])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1e30])
@pytest.mark.parametrize("fp8", [False, True])
def test_magnitudes(mla, q_lora, eps, fp8):
    rng = np.random.default_rng(q_lora)
    n = len(POWERS)
    # both latents of a token at one power of two, the rotated part of size 1
    x = rng.standard_normal((n, q_lora + 576)).clip(-3.9, 3.9)
    x[:, :q_lora + 512] *= 2.0 ** np.array(POWERS)[:, None]
    with np.errstate(over="raise"):
        bits = R.bf16_bits(x.astype(np.float32))
    w_q, w_kv = (R.bf16_bits(1 + 0.3 * rng.standard_normal(m).astype(np.float32))
                 for m in (q_lora, 512))
    f = synth.bf16_bits_to_f64
    xs, eps = f(bits), float(np.float32(eps))
    assert np.isfinite(xs).all()
    cache = [torch.zeros(1, 64, 576, dtype=torch.uint8, device="cuda"),
             torch.zeros(1, 64, dtype=torch.int8, device="cuda")] if fp8 else [
                 torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")]
    call = mla.norm_rope_append_fp8 if fp8 else mla.norm_rope_append
    c_q, ws = call(dev_bf16(bits), dev_bf16(w_q), dev_bf16(w_kv), dev_i32([0, n]), dev_i32([n]),
                   dev_i32([[0]]), *cache, 10000.0, eps)
    assert mla.check_device_status(ws) == 0

    def rms(v, w):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * f(w)

    # as in the norms' other tests: 2^-20 relative before the rounding. Beside it a result below
    # 2^-100 (eps far above the row's squares) may have gone through fp32's subnormals.
    tiny = 2.0 ** -100
    ref = rms(xs[:, :q_lora], w_q)
    R.assert_within(host_f64_from_bf16(c_q), ref,
                    (R.HALF_STEP_BF16 + 2.0 ** -20) * np.abs(ref) + tiny, "c_q")
    ref = rms(xs[:, q_lora:q_lora + 512], w_kv)
    if not fp8:
        R.assert_within(host_f64_from_bf16(cache[0])[0, :n, :512], ref,
                        (R.HALF_STEP_BF16 + 2.0 ** -20) * np.abs(ref) + tiny, "rows")
        return
    codes, exps = (t.cpu().numpy()[0, :n] for t in cache)
    step = 2.0 ** exps.astype(float)[:, None]
    R.assert_within(R.fp8_values(codes, exps)[:, :512], ref,
                    2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * step + 2.0 ** -20 * np.abs(ref) + tiny,
                    "rows")
