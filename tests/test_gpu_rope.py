"""Rotary positions of heads, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALINGS = {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=8.0),
            "yarn": dict(factor=40.0, original=4096),
            "bands": dict(theta=500000.0, factor=8.0, original=8192, fast=4.0, slow=1.0)}


@pytest.fixture(scope="module")
def mla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_13_gb300 import mla as m
    return m


def turned(x, pos, plan, offset):
    """The rotated values of x [T, H, width] in 64 bits, and the bound of an error: half a step of
    bf16 of the value, and of the pair's length 2^-21 for the fp32 arithmetic (cosine, sine and
    magnitude each within 2^-23 of their value, three more roundings) and the angles."""
    rot = plan.rot
    v = x.double().cpu()[..., offset:offset + rot]
    f = torch.tensor(plan.freq[:rot // 2], dtype=torch.float64)
    turns = pos.cpu().double()[:, None] * f / (2 * np.pi)
    angle = ((turns - turns.round()) * 2 * np.pi)[:, None]
    # pos f has an error of 2^-53 of itself in radians
    blur = (pos.cpu().double().abs()[:, None] * f * 2.0 ** -51)[:, None]
    if plan.layout:
        a, b = v[..., :rot // 2], v[..., rot // 2:]
    else:
        a, b = v[..., 0::2], v[..., 1::2]
    m = plan.magnitude
    p = m * (a * angle.cos() - b * angle.sin())
    q = m * (a * angle.sin() + b * angle.cos())
    size = abs(m) * torch.hypot(a, b)
    slack = size * (2.0 ** -21 + blur)

    def join(u, w):
        return torch.cat([u, w], -1) if plan.layout else torch.stack([u, w], -1).reshape(v.shape)

    want = join(p, q)
    return want, want.abs() * 2.0 ** -8 + 1.01 * join(slack, slack) + 1e-38


def inputs(seed, tokens, heads, width, far=100000):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads, width, generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, far, (tokens,), generator=g, dtype=torch.int32).cuda()
    return x, pos


def check(got, x, pos, plan, offset):
    want, tol = turned(x, pos, plan, offset)
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(err).all() and (err <= tol).all(), float((err - tol).max())


def others(x, plan, offset):
    return torch.cat([x[..., :offset], x[..., offset + plan.rot:]], -1)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("tokens,heads,width,offset,rot", [
    (1, 1, 2, 0, 2), (3, 2, 64, 0, 64), (128, 16, 192, 128, 64), (7, 5, 77, 3, 50), (65, 3, 80, 16, 32),
    (2, 128, 256, 0, 256), (33, 1, 12, 4, 4), (1000, 1, 8, 0, 8), (5, 7, 100, 36, 64), (1, 300, 66, 2, 64)])
def test_rope(mla, tokens, heads, width, offset, rot, scaling, layout):
    plan = mla.rope_plan(rot, scaling=scaling, layout=layout, **SCALINGS[scaling])
    x, pos = inputs(1, tokens, heads, width)
    # apart, split, and where it lies
    check(mla.rope(x, pos, plan, offset=offset), x, pos, plan, offset)
    y, rest = mla.rope(x, pos, plan, offset=offset, split=True)
    check(y, x, pos, plan, offset)
    assert torch.equal(rest, others(x, plan, offset))
    z = x.clone()
    mla.rope(z, pos, plan, offset=offset, out=z[..., offset:offset + rot])
    assert torch.equal(z[..., offset:offset + rot], y)
    assert torch.equal(others(z, plan, offset), rest)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8])
def test_strides_and_alignment(mla, shift, layout):
    """Views at any place of larger tensors, heads before tokens, and a key that all heads share."""
    plan = mla.rope_plan(32, layout=layout)
    big, pos = inputs(2, 9, 11, 64 + shift)
    x = big[:, 2:9, shift:shift + 48]
    out = torch.zeros(7, 9, 40 + shift, dtype=torch.bfloat16, device="cuda")
    rest = torch.zeros(9, 20, 16 + shift, dtype=torch.bfloat16, device="cuda")
    y = out.transpose(0, 1)[..., shift:shift + 32]
    r = rest[:, 1:15:2, shift:]
    mla.rope(x, pos, plan, offset=8, out=y, rest=r)
    check(y, x, pos, plan, 8)
    assert torch.equal(r, others(x, plan, 8))
    # nothing beside them was written
    assert not out[..., :shift].any() and not out[..., shift + 32:].any()
    assert not rest[:, 0::2].any() and not rest[:, 15:].any() and not rest[..., :shift].any()
    one = big[:, :1, shift:shift + 32].expand(9, 6, 32)
    check(mla.rope(one, pos, plan), one, pos, plan, 0)


@pytest.mark.parametrize("pos", [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1])
def test_far_positions(mla, pos):
    plan = mla.rope_plan(64, scaling="bands", **SCALINGS["bands"])
    x, _ = inputs(3, 4, 3, 64)
    at = torch.full((4,), pos, dtype=torch.int32, device="cuda")
    y = mla.rope(x, at, plan)
    if pos == 0:
        assert torch.equal(y, x)
    check(y, x, at, plan, 0)


@pytest.mark.parametrize("tokens,heads,width,offset,rot", [(2, 4096, 40, 4, 32), (1, 1, 4096, 2000, 256),
                                                           (20000, 1, 6, 1, 4), (3, 5, 64, 0, 64)])
def test_largest_and_whole(mla, tokens, heads, width, offset, rot):
    plan = mla.rope_plan(rot)
    x, pos = inputs(9, tokens, heads, width)
    y, rest = mla.rope(x, pos, plan, offset=offset, split=True)  # (of a whole head nothing is left)
    check(y, x, pos, plan, offset)
    assert torch.equal(rest, others(x, plan, offset))
    z = x.clone()
    mla.rope(z, pos, plan, offset=offset, out=z[..., offset:offset + rot])
    assert torch.equal(z[..., offset:offset + rot], y) and torch.equal(others(z, plan, offset), rest)


def test_turned_back(mla):
    plan = mla.rope_plan(64, scaling="linear", factor=2.0)
    x, pos = inputs(4, 50, 4, 64)
    y = mla.rope(x, pos, plan)
    z = mla.rope(y, -pos, plan)
    # two roundings of each value of a pair, of at most the pair's length
    size = torch.hypot(x[..., 0::2].float(), x[..., 1::2].float()).repeat_interleave(2, -1)
    assert ((z.float() - x.float()).abs() <= 2 * 1.5 * 2.0 ** -8 * size).all()


def test_own_frequencies(mla):
    plan = mla.rope_plan(8, magnitude=0.25)
    for i in range(4):
        plan.freq[i] = [3.0, 0.0, 1e-12, 65536.0][i]
    x, pos = inputs(5, 20, 2, 8)
    check(mla.rope(x, pos, plan), x, pos, plan, 0)


def test_stream_and_graph(mla):
    plan = mla.rope_plan(64, scaling="yarn", factor=40.0, original=4096)
    x, pos = inputs(6, 40, 8, 192)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, rest = mla.rope(x, pos, plan, offset=128, split=True, stream=st)
    st.synchronize()
    check(y, x, pos, plan, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.rope(x, pos, plan, offset=128, out=y, rest=rest)
    plan.freq[0] = 0.5  # (a plan is read before the call returns)
    pos += 1000
    g.replay()
    torch.cuda.synchronize()
    check(y, x, pos, mla.rope_plan(64, scaling="yarn", factor=40.0, original=4096), 128)


def test_special_values(mla):
    """Infinities and NaN stay in their pairs."""
    plan = mla.rope_plan(8)
    x, pos = inputs(7, 3, 2, 8)
    x[1, 0, 2], x[2, 1, 5] = float("inf"), float("nan")
    y = mla.rope(x, pos, plan)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 2:4] = True
    want[2, 1, 4:6] = True
    assert torch.equal(bad, want)


def test_refused(mla):
    plan = mla.rope_plan(64)
    x, pos = inputs(8, 4, 2, 64)
    for bad in (dict(offset=1), dict(offset=-1)):
        with pytest.raises(mla.MLAError):
            mla.rope(x, pos, plan, **bad)
    with pytest.raises(ValueError):
        mla.rope(x, pos[:3], plan)
    with pytest.raises(ValueError):
        mla.rope(x.transpose(1, 2), pos, plan)
    with pytest.raises(ValueError):
        mla.rope(x, pos, plan, out=torch.empty(4, 2, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        mla.rope(x.float(), pos, plan)
    with pytest.raises(TypeError):
        mla.rope(x, pos.long(), plan)
    with pytest.raises(TypeError):
        mla.rope(x, pos, b"plan")
    with pytest.raises(mla.MLAError):  # no tokens
        mla.rope(x[:0], pos[:0], plan)
    with pytest.raises(mla.MLAError):  # rows of the output on top of each other
        mla.rope(x, pos, plan, out=torch.empty(4, 1, 64, dtype=torch.bfloat16,
                                               device="cuda").expand(4, 2, 64))
