"""Workloads of the operators that serve long and partly common contexts from a paged latent cache:
decode attention of batches that share a prefix, rotary positions scaled for long contexts, and the
4-bit cache, quantised as it is written and read back (as are FP8 and bf16 caches).

Each case runs in two forms: elementary torch operations in 32 bits, 64 where they are needed (`own`
false), or the calls a program makes of this framework (`own` true).

Shared prefix: query token t of s_q of sequence b stands at position lens[b] - s_q + t and sees every
cached row up to it; the sequences of group g hold the same pages for their first prefix[g] // 64 pages.
  s_j = scale (q_lat . c_j + q_rope . r_j), out = sum_j softmax(s)_j c_j, lse = ln sum_j exp(s_j)
Rotation: `rot` values of each head from `offset` on, as pairs (2i, 2i + 1) or (i, i + rot / 2), turn by
pos * freq[i] and are multiplied by `magnitude`; the head's other values are passed on or stay.
4-bit cache: a token's 512 latent values, normed and rounded to bf16, as e2m1 codes (0, 1/2, 1, 3/2, 2, 3,
4, 6 and negatives), one e4m3 scale for each 16 of them and one exponent e for the token:
  e the smallest with max |x| <= 6 * 448 * 2^e, scale = e4m3(max |x| of the 16 / 6 / 2^e),
  code = e2m1(x / scale / 2^e); the rotated key stays bf16.
"""
import math
import random

import torch

own = False

D_C, D_R, D = 512, 64, 576
PAGE = 64
GROUP = 16
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # four samples of one prompt, a head shard: a single call's latency
        dict(name="shared four samples", op="shared", batch=4, heads=16, tokens=1, groups=1,
             prefix=1900, tail=150, idle=0.0, fp8=False, lens=1),
        # two agents' tool prompts with two draft tokens each to verify, FP8 cache, a padded batch
        dict(name="shared drafts fp8", op="shared", batch=48, heads=16, tokens=2, groups=2,
             prefix=12000, tail=700, idle=0.1, fp8=True, lens=2),
        # several system prompts of different lengths, every sequence with a turn of its own
        dict(name="shared prompts", op="shared", batch=128, heads=32, tokens=1, groups=5,
             prefix=6000, tail=900, idle=0.0, fp8=False, lens=3),
        # many samples of one long document, half of the heads
        dict(name="shared document", op="shared", batch=96, heads=64, tokens=1, groups=1,
             prefix=16000, tail=1500, idle=0.0, fp8=False, lens=4),
        # a decode batch's queries, rotated where they lie
        dict(name="rope decode", op="rope", tokens=128, heads=16, width=64, offset=0, rot=64,
             layout="interleaved", scaling="yarn", split=False, far=100000, lens=5),
        # a prefill chunk's queries, rotated and split as the expanded attention takes them
        dict(name="rope prefill split", op="rope", tokens=4096, heads=128, width=192, offset=128,
             rot=64, layout="interleaved", scaling="yarn", split=True, far=160000, lens=6),
        # part of an odd head in halves, another model's shape
        dict(name="rope half odd", op="rope", tokens=1001, heads=24, width=77, offset=3, rot=50,
             layout="half", scaling="bands", split=False, far=131072, lens=7),
        # the new tokens of a decode batch into the 4-bit cache, and what it then holds
        dict(name="fp4 decode batch", op="store", batch=128, chunk=1, singles=1.0, q_lora=1536,
             ctx=8192, layout="interleaved", scaling="yarn", pad=0, lens=8),
        # a prefill step's tokens, read back for the expanded attention
        dict(name="fp4 prefill", op="store", batch=37, chunk=500, singles=0.2, q_lora=1536, ctx=4096,
             layout="interleaved", scaling="yarn", pad=3, lens=9),
        # one prompt's rows out of an FP8 cache
        dict(name="read prompt fp8", op="read", kind="fp8", batch=1, ctx=1900, lens=10),
        # a batch's contexts out of the 4-bit cache
        dict(name="read batch fp4", op="read", kind="fp4", batch=48, ctx=8192, lens=11),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo..hi."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9))))


def draw(rng):
    largest = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["shared", "shared", "rope", "store", "read"])
        c = dict(op=op, lens=rng.randrange(1 << 30))
        if op == "shared":
            heads = rng.choice([16, 32, 64, 128])
            batch = _log(rng, 1, 160)
            c.update(batch=batch, heads=heads, tokens=rng.randint(1, min(3, 128 // heads)),
                     groups=min(batch, _log(rng, 1, 8)), prefix=_log(rng, 1, 20000),
                     tail=_log(rng, 1, 2000), idle=rng.choice([0.0, 0.0, 0.2]),
                     fp8=rng.random() < 0.4)
        elif op == "rope":
            rot = 2 * _log(rng, 1, 64)
            rest = rng.choice([0, 0, 128, rng.randint(0, 130)])
            c.update(tokens=_log(rng, 1, 5000), heads=_log(rng, 1, 128), width=rot + rest,
                     offset=rng.choice([0, rest, rng.randint(0, rest)]), rot=rot,
                     layout=rng.choice(["interleaved", "half"]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                     split=rng.random() < 0.5, far=_log(rng, 100, 1000000))
        elif op == "store":
            c.update(batch=_log(rng, 1, 200), chunk=_log(rng, 1, 500),
                     singles=round(rng.random(), 2), q_lora=64 * rng.randint(0, 28),
                     ctx=_log(rng, 600, 16000), layout=rng.choice(["interleaved", "half"]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                     pad=rng.choice([0, 5]))
        else:
            c.update(kind=rng.choice(["bf16", "fp8", "fp4", "fp4"]), batch=_log(rng, 1, 100),
                     ctx=_log(rng, 1, 16000))
        if _cost(c) <= largest:
            return c


# ------------------------------------------------------------------ shapes from the case alone

def _shared_shape(case):
    """The sequences' groups, prefixes and lengths: (first sequence of each group and the batch's
    end, prefix rows of each group, length of each sequence)."""
    rng = random.Random(case["lens"])
    b, g, n = case["batch"], case["groups"], case["tokens"]
    cuts = sorted(rng.sample(range(1, b), g - 1))
    starts = [0] + cuts + [b]
    prefix = [case["prefix"]] + [rng.randint(max(1, case["prefix"] // 3), case["prefix"])
                                 for _ in range(g - 1)]
    lens = []
    for k in range(g):
        for _ in range(starts[k], starts[k + 1]):
            tail = rng.randint(n, max(n, case["tail"]))
            lens.append(0 if rng.random() < case["idle"] else prefix[k] + tail)
    return starts, prefix, lens


def _ragged(case):
    """(new tokens, length after them) of every sequence."""
    rng = random.Random(case["lens"])
    counts, lens = [], []
    for _ in range(case["batch"]):
        n = 1 if rng.random() < case["singles"] else rng.randint(
            max(1, case["chunk"] // 3), case["chunk"])
        n = min(n, case["ctx"])
        counts.append(n)
        lens.append(rng.randint(max(n, case["ctx"] // 3), case["ctx"]))
    return counts, lens


def _spans(case):
    """(first row, rows) that are read of every sequence."""
    rng = random.Random(case["lens"])
    got = []
    for _ in range(case["batch"]):
        n = rng.randint(max(1, case["ctx"] // 2), case["ctx"])
        got.append((rng.choice([0, 0, rng.randint(0, 200)]), n))
    return got


ROW_BYTES = dict(bf16=2 * D, fp8=D + 1, fp4=D_C // 2 + D_C // GROUP + 1 + 2 * D_R)


def work(case):
    op = case["op"]
    if op == "shared":
        starts, prefix, lens = _shared_shape(case)
        n, heads = case["tokens"], case["heads"]
        read = 0
        for k, p in enumerate(prefix):
            mine = [length for length in lens[starts[k]:starts[k + 1]] if length]
            both = p // PAGE * PAGE
            read += (both if mine else 0) + sum(length - both for length in mine)
        seen = sum(length - n + 1 + t for length in lens if length for t in range(n))
        rows = case["batch"] * n * heads
        return {"bytes": rows * (2 * D + 2 * D_C + 4) + read * ROW_BYTES["fp8" if case["fp8"]
                                                                         else "bf16"],
                "flops": seen * heads * 2 * (D + D_C)}
    if op == "rope":
        moved = case["width"] if case["split"] else case["rot"]
        values = case["tokens"] * case["heads"]
        return {"bytes": values * moved * 4 + 4 * case["tokens"], "flops": values * case["rot"] * 3}
    if op == "store":
        t = sum(_ragged(case)[0])
        return {"bytes": t * (2 * (case["q_lora"] + D) + 2 * case["q_lora"] +
                              2 * ROW_BYTES["fp4"] + 2 * D),
                "flops": t * 4 * (case["q_lora"] + D)}
    rows = sum(n for _, n in _spans(case))
    return {"bytes": rows * (ROW_BYTES[case["kind"]] + 2 * D), "flops": 0}


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.7e12, w["flops"] / 1.5e15)


# ------------------------------------------------------------------------- rotation's plan

SCALINGS = {
    # theta, and what the scaling takes: factor, original context, and the bounds of its ramp
    "none": dict(theta=10000.0),
    "linear": dict(theta=10000.0, factor=4.0),
    "ntk": dict(theta=10000.0, factor=8.0),
    "yarn": dict(theta=10000.0, factor=40.0, original=4096, fast=32.0, slow=1.0),
    "bands": dict(theta=500000.0, factor=8.0, original=8192, fast=4.0, slow=1.0),
}


def _frequencies(rot, scaling):
    """(radians a position of each pair, magnitude), in Python's 64 bits."""
    s = SCALINGS[scaling]
    theta, factor = s["theta"], s.get("factor", 1.0)
    if scaling == "ntk" and rot > 2:
        theta *= factor ** (rot / (rot - 2))
    plain = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling in ("none", "ntk"):
        return plain, 1.0
    if scaling == "linear":
        return [f / factor for f in plain], 1.0
    keep = []  # how much of the plain frequency stays
    if scaling == "yarn":
        def index(turns):  # the pair that makes so many turns over the original context
            return rot * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
        low = max(math.floor(index(s["fast"])), 0)
        high = min(math.ceil(index(s["slow"])), rot - 1)
        for i in range(rot // 2):
            keep.append(1.0 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001))))
    else:
        for f in plain:
            turns = s["original"] * f / (2 * math.pi)
            keep.append(min(1.0, max(0.0, (turns - s["slow"]) / (s["fast"] - s["slow"]))))
    mixed = [f * k + f / factor * (1.0 - k) for f, k in zip(plain, keep)]
    return mixed, 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0


# ------------------------------------------------------------------------------- inputs

def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(gen, blocks, kind):
    """Latent rows of unit size, or codes, scales and exponents that stand for such rows."""
    if kind == "bf16":
        return dict(cache=torch.randn(blocks, PAGE, D, device="cuda", generator=gen,
                                      dtype=torch.float32).to(torch.bfloat16))
    if kind == "fp8":
        x = torch.randn(blocks, PAGE, D, device="cuda", generator=gen) * 64.0
        exps = torch.randint(-7, -4, (blocks, PAGE), device="cuda", generator=gen).to(torch.int8)
        return dict(codes=x.to(torch.float8_e4m3fn).view(torch.uint8), exps=exps)
    codes = torch.randint(0, 256, (blocks, PAGE, D_C // 2), device="cuda", generator=gen,
                          dtype=torch.uint8)
    scales = torch.rand(blocks, PAGE, D_C // GROUP, device="cuda", generator=gen) * 440 + 8
    exps = torch.randint(-10, -7, (blocks, PAGE), device="cuda", generator=gen).to(torch.int8)
    keys = torch.randn(blocks, PAGE, D_R, device="cuda", generator=gen)
    return dict(codes=codes, scales=scales.to(torch.float8_e4m3fn).view(torch.uint8), exps=exps,
                keys=keys.to(torch.bfloat16))


def _tables(gen, held):
    """A block table over pages in random order, -1 where a sequence holds none, and their number."""
    pool = int(held.sum())
    table = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
    table[held] = torch.randperm(pool, device="cuda", generator=gen).to(torch.int32)
    return table, max(1, pool)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = dict(case)
    if op == "shared":
        starts, prefix, lens = _shared_shape(case)
        b, n, heads = case["batch"], case["tokens"], case["heads"]
        ctx = max(max(lens), 1)
        st.update(ctx=ctx, lens=_int(lens), starts=_int(starts), prefix=_int(prefix))
        both = torch.zeros(b, dtype=torch.int64, device="cuda")  # pages in common
        first = torch.zeros(b, dtype=torch.int64, device="cuda")  # and who comes first in them
        for k, p in enumerate(prefix):
            live = [i for i in range(starts[k], starts[k + 1]) if lens[i]]
            both[starts[k]:starts[k + 1]] = p // PAGE
            first[starts[k]:starts[k + 1]] = live[0] if live else starts[k]
        page = torch.arange(-(-ctx // PAGE), device="cuda")
        held = page < ((st["lens"] + PAGE - 1) // PAGE)[:, None]
        shared = held & (page < both[:, None])
        owner = first == torch.arange(b, device="cuda")
        table, pool = _tables(gen, held & (~shared | owner[:, None]))
        st["table"] = torch.where(shared, table[first], table)
        st.update(_cache(gen, pool, "fp8" if case["fp8"] else "bf16"))
        shape = (b, heads) if n == 1 else (b, n, heads)
        q = (0.6 * torch.randn(*shape, D, device="cuda", generator=gen)).to(torch.bfloat16)
        st["q_lat"], st["q_rope"] = q[..., :D_C].contiguous(), q[..., D_C:].contiguous()
        st["out"] = torch.zeros(*shape, D_C, device="cuda", dtype=torch.bfloat16)
        st["lse"] = torch.zeros(*shape, device="cuda")
        return st
    if op == "rope":
        t, heads, width = case["tokens"], case["heads"], case["width"]
        st["x"] = torch.randn(t, heads, width, device="cuda", generator=gen).to(torch.bfloat16)
        st["pos"] = torch.randint(0, case["far"], (t,), device="cuda", generator=gen,
                                  dtype=torch.int32)
        if case["split"]:
            st["out"] = torch.zeros(t, heads, case["rot"], device="cuda", dtype=torch.bfloat16)
            st["rest"] = torch.zeros(t, heads, width - case["rot"], device="cuda",
                                     dtype=torch.bfloat16)
        st["freq"], st["magnitude"] = _frequencies(case["rot"], case["scaling"])
        st["freq"] = torch.tensor(st["freq"], dtype=torch.float64, device="cuda")
        return st
    if op == "store":
        counts, lens = _ragged(case)
        pad, total, ql = case["pad"], sum(counts), case["q_lora"]
        st.update(total=total, lens=_int(lens),
                  starts=_int([sum(counts[:b]) for b in range(len(counts) + 1)]),
                  first=_int([length - n for n, length in zip(counts, lens)]))
        page = torch.arange(-(-case["ctx"] // PAGE), device="cuda")
        # only the pages that this step writes are there
        held = (page < ((st["lens"] + PAGE - 1) // PAGE)[:, None]) & (
            page >= (st["first"] // PAGE)[:, None])
        st["table"], pool = _tables(gen, held)
        st.update(_cache(gen, pool, "fp4"))
        # projections of hidden states: unit size with a scale of its own for each token
        x = torch.randn(total + pad, ql + D, device="cuda", generator=gen)
        x *= torch.rand(total + pad, 1, device="cuda", generator=gen) * 4 + 0.05
        st["x"] = x.to(torch.bfloat16)
        for k, n in (("w_q", ql), ("w_kv", D_C)):
            st[k] = (1 + 0.2 * torch.randn(n, device="cuda", generator=gen)).to(torch.bfloat16)
        st["c_q"] = torch.zeros(total + pad, ql, device="cuda", dtype=torch.bfloat16)
        st["rows"] = torch.zeros(total, D, device="cuda", dtype=torch.bfloat16)
        st["freq"], st["magnitude"] = _frequencies(D_R, case["scaling"])
        st["freq"] = torch.tensor(st["freq"], dtype=torch.float64, device="cuda")
        return st
    spans = _spans(case)
    ends = [first + n for first, n in spans]
    page = torch.arange(-(-max(ends) // PAGE), device="cuda")
    st["first"] = _int([first for first, _ in spans])
    st["starts"] = _int([sum(n for _, n in spans[:b]) for b in range(len(spans) + 1)])
    held = (page * PAGE < _int(ends)[:, None]) & (page >= (st["first"] // PAGE)[:, None])
    st["table"], pool = _tables(gen, held)
    st.update(_cache(gen, pool, case["kind"]))
    st["total"] = sum(n for _, n in spans)
    st["rows"] = torch.zeros(st["total"], D, device="cuda", dtype=torch.bfloat16)
    return st


# -------------------------------------------------------------------------- plain forms

def _read_rows(st, page, slot):
    """Cached rows in 32 bits."""
    if "cache" in st:
        return st["cache"][page, slot].float()
    e = torch.exp2(st["exps"][page, slot].float())[..., None]
    if "scales" not in st:
        return st["codes"].view(torch.float8_e4m3fn)[page, slot].float() * e
    byte = st["codes"][page, slot].int()
    code = torch.stack([byte & 15, byte >> 4], -1).reshape(*byte.shape[:-1], D_C // GROUP, GROUP)
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda")
    c = level[code] * st["scales"].view(torch.float8_e4m3fn)[page, slot].float()[..., None]
    c = c.reshape(*byte.shape[:-1], D_C) * e
    return torch.cat([c, st["keys"][page, slot].float()], -1)


def _attend(st):
    """Attention of all sequences at once, padded to the most rows of one."""
    b, n, heads = st["batch"], st["tokens"], st["heads"]
    lens = st["lens"].long()
    j = torch.arange(st["ctx"], device="cuda")
    live = j < lens[:, None]
    page = st["table"].long()[:, j // PAGE].clamp(min=0)
    kv = torch.where(live[..., None], _read_rows(st, page, j % PAGE), 0.0)
    q = torch.cat([st["q_lat"], st["q_rope"]], -1).float().reshape(b, n * heads, D)
    s = torch.matmul(q, kv.transpose(1, 2)).mul_(SCALE).reshape(b, n, heads, -1)
    pos = lens[:, None] - n + torch.arange(n, device="cuda")
    s.masked_fill_((j > pos[..., None])[:, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    st["lse"].copy_((torch.log(total) + top).reshape(st["lse"].shape))
    out = torch.matmul(s.reshape(b, n * heads, -1), kv[..., :D_C]).reshape(b, n, heads, D_C)
    st["out"].copy_(torch.where(total > 0, out / total, 0.0).reshape(st["out"].shape))
    return dict(out=st["out"], lse=st["lse"])


def _turned(x, st, pos):
    """The pairs of x [tokens, heads, rot], turned, in 32 bits."""
    angle = pos.double()[:, None, None] * st["freq"]
    co, si = angle.cos().float() * st["magnitude"], angle.sin().float() * st["magnitude"]
    if st["layout"] == "half":
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * co - b * si, a * si + b * co], -1)
    a, b = x.float().reshape(*x.shape[:-1], -1, 2).unbind(-1)
    return torch.stack([a * co - b * si, a * si + b * co], -1).reshape(x.shape)


def _rope(st):
    x, o, r = st["x"], st["offset"], st["rot"]
    y = _turned(x[..., o:o + r], st, st["pos"]).to(torch.bfloat16)
    if not st["split"]:
        # where it lies: the same buffer is turned by every pass
        x[..., o:o + r] = y
        return dict(x=x)
    st["out"].copy_(y)
    st["rest"][..., :o] = x[..., :o]
    st["rest"][..., o:] = x[..., o + r:]
    return dict(out=st["out"], rest=st["rest"])


def _nearest_bf16(x):
    """64-bit values to the nearest with 8 significant bits, ties to even, in one rounding."""
    bits = x.view(torch.int64)
    bits = (bits + ((1 << 44) - 1) + ((bits >> 45) & 1)) & ~((1 << 45) - 1)
    return bits.view(torch.float64).float()


def _store(st):
    """Both norms, the rotation, the quantised write of all tokens, and the rows that it left."""
    ql, total = st["q_lora"], st["total"]
    starts, lens = st["starts"].long(), st["lens"].long()
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[b] - starts[b + 1] + t
    x = st["x"][:total]
    if ql:
        c = x[:, :ql].float()
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * st["w_q"].float()
        st["c_q"][:total] = c.to(torch.bfloat16)
    # a value next to the border of two codes shows every rounding: the norm in 64 bits
    c = x[:, ql:ql + D_C].double()
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * st["w_kv"].double()
    c = _nearest_bf16(c).reshape(total, D_C // GROUP, GROUP)
    most = c.abs().amax((1, 2))
    # the smallest e with max |x| <= 6 * 448 * 2^e = 1.3125 * 2^(11 + e)
    f, k = torch.frexp(most)
    e = torch.where(f <= 0.65625, k - 12, k - 11).clamp(min=-120)
    e = torch.where(most > 0, e, 0)
    c = c * torch.exp2(-e.float())[:, None, None]
    scale = (c.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    step = scale.float()[..., None]
    q = torch.where(step > 0, c.abs() / step, 0.0)
    code = ((q > 0.25).int() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) +
            (q > 5.0))
    code = (code + 8 * (c < 0)).reshape(total, D_C)
    r = _turned(x[:, None, ql + D_C:], st, pos).reshape(total, D_R)
    page, slot = st["table"].long()[b, pos // PAGE], pos % PAGE
    st["codes"][page, slot] = (code[:, ::2] + 16 * code[:, 1::2]).to(torch.uint8)
    st["scales"][page, slot] = scale.view(torch.uint8)
    st["exps"][page, slot] = e.to(torch.int8)
    st["keys"][page, slot] = r.to(torch.bfloat16)
    st["rows"].copy_(_read_rows(st, page, slot))
    return dict(c_q=st["c_q"], rows=st["rows"])


def _read(st):
    starts = st["starts"].long()
    t = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = st["first"].long()[b] + t - starts[b]
    st["rows"].copy_(_read_rows(st, st["table"].long()[b, pos // PAGE], pos % PAGE))
    return dict(rows=st["rows"])


# ------------------------------------------------------------------- the framework's calls

def _kept(st, size):
    """The workspace that a program keeps for a shape."""
    if "workspace" not in st:
        from mla_latent_kv_13_gb300 import mla
        st["workspace"] = mla.alloc_workspace(size(mla))
    return st["workspace"]


def _plan(st, rot):
    """The rotation's plan, which a program makes once for a model."""
    if "plan" not in st:
        from mla_latent_kv_13_gb300 import mla
        st["plan"] = mla.rope_plan(rot, scaling=st["scaling"], layout=st["layout"],
                                   **SCALINGS[st["scaling"]])
    return st["plan"]


def _read_own(st, ws):
    from mla_latent_kv_13_gb300 import mla
    if "cache" in st:
        call, cache = mla.read_kv, (st["cache"],)
    elif "scales" in st:
        call, cache = mla.read_kv_fp4, (st["codes"], st["scales"], st["exps"], st["keys"])
    else:
        call, cache = mla.read_kv_fp8, (st["codes"], st["exps"])
    call(*cache, st["table"], st["first"], st["starts"], out=st["rows"], workspace=ws)


def _own(st):
    from mla_latent_kv_13_gb300 import mla
    op = st["op"]
    if op == "shared":
        b, n, h, g = st["batch"], st["tokens"], st["heads"], st["groups"]
        ws = _kept(st, lambda m: m.decode_shared_workspace_size(b, n, h, st["ctx"], g))
        cache = (st["codes"], st["exps"]) if st["fp8"] else (st["cache"],)
        call = mla.decode_attention_shared_fp8 if st["fp8"] else mla.decode_attention_shared
        call(st["q_lat"], st["q_rope"], *cache, st["table"], st["lens"], st["starts"],
             st["prefix"], st["ctx"], SCALE, out=st["out"], lse=st["lse"], workspace=ws)
        return dict(out=st["out"], lse=st["lse"])
    if op == "rope":
        plan, o, r = _plan(st, st["rot"]), st["offset"], st["rot"]
        if not st["split"]:
            mla.rope(st["x"], st["pos"], plan, offset=o, out=st["x"][..., o:o + r])
            return dict(x=st["x"])
        mla.rope(st["x"], st["pos"], plan, offset=o, out=st["out"], rest=st["rest"])
        return dict(out=st["out"], rest=st["rest"])
    ws = _kept(st, lambda m: m.WS_HEADER_BYTES)
    if op == "store":
        mla.norm_rope_append_fp4(st["x"], st["w_q"], st["w_kv"], st["starts"], st["lens"],
                                 st["table"], st["codes"], st["scales"], st["exps"], st["keys"],
                                 _plan(st, D_R), EPS, c_q=st["c_q"], workspace=ws)
        _read_own(st, ws)
        return dict(c_q=st["c_q"], rows=st["rows"])
    _read_own(st, ws)
    return dict(rows=st["rows"])


def run(state):
    if own:
        return _own(state)
    return {"shared": _attend, "rope": _rope, "store": _store, "read": _read}[state["op"]](state)


# ----------------------------------------------------------------------------- in 64 bits

def _pool64(st):
    """The whole cache in 64 bits, [pages, 64, 576]."""
    if "cache" in st:
        return st["cache"].double()
    e = 2.0 ** st["exps"].double()[..., None]
    if "scales" not in st:
        return st["codes"].view(torch.float8_e4m3fn).double() * e
    c = torch.empty(*st["codes"].shape[:2], D_C, dtype=torch.float64, device="cuda")
    for half, nibble in ((0, st["codes"] & 15), (1, st["codes"] >> 4)):
        m, two = (nibble & 1).double(), ((nibble >> 1) & 3).double()
        v = torch.where(two == 0, m / 2, (1 + m / 2) * 2.0 ** (two - 1))
        c[..., half::2] = torch.where(nibble >= 8, -v, v)
    c *= st["scales"].view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, -1)
    return torch.cat([c * e, st["keys"].double()], -1)


def _spin64(x, case, pos):
    """x [tokens, .., rot] turned at its positions, by complex products."""
    rot = x.shape[-1]
    freq, size = _frequencies(rot, case["scaling"])
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    angle = pos.double()[:, None] * freq
    z = torch.polar(torch.full_like(angle, size), angle)[:, None]
    x = x.double()
    if case["layout"] == "half":
        w = torch.complex(x[..., :rot // 2], x[..., rot // 2:]) * z
        return torch.cat([w.real, w.imag], -1)
    w = torch.complex(x[..., 0::2], x[..., 1::2]) * z
    return torch.view_as_real(w).reshape(x.shape)


def exact(case, seed):
    op = case["op"]
    if op == "shared" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    if op == "rope":
        x, o, r = st["x"], case["offset"], case["rot"]
        y = _spin64(x[..., o:o + r], case, st["pos"])
        if case["split"]:
            return dict(out=y, rest=torch.cat([x[..., :o], x[..., o + r:]], -1).double())
        return dict(x=torch.cat([x[..., :o].double(), y, x[..., o + r:].double()], -1))
    table = st["table"].long()
    if op == "shared":
        _, _, lens = _shared_shape(case)
        n, heads = case["tokens"], case["heads"]
        q = torch.cat([st["q_lat"], st["q_rope"]], -1).reshape(-1, n, heads, D).double()
        out = torch.zeros(*q.shape[:3], D_C, dtype=torch.float64, device="cuda")
        lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
        pool = _pool64(st)
        for b, length in enumerate(lens):
            kv = pool[table[b]].reshape(-1, D)[:length]
            for t in range(n):
                seen = kv[:max(0, length - n + 1 + t)]
                if len(seen):
                    s = q[b, t] @ seen.T * SCALE
                    lse[b, t] = torch.logsumexp(s, -1)
                    out[b, t] = torch.exp(s - lse[b, t, :, None]) @ seen[:, :D_C]
        return dict(out=out.reshape(st["out"].shape), lse=lse.reshape(st["lse"].shape))
    if op == "read":
        pool = _pool64(st)
        rows = []
        for b, (first, n) in enumerate(_spans(case)):
            p = torch.arange(first, first + n, device="cuda")
            rows.append(pool[table[b, p // PAGE], p % PAGE])
        return dict(rows=torch.cat(rows))
    return _exact_store(case, st)


def _exact_store(case, st):
    counts, lens = _ragged(case)
    ql = case["q_lora"]
    c_q = st["c_q"].double()
    w_q, w_kv = st["w_q"].double(), st["w_kv"].double()
    levels = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    rows, base = [], 0
    for n, length in zip(counts, lens):
        x = st["x"][base:base + n].double()
        if ql:
            q = x[:, :ql]
            c_q[base:base + n] = q / torch.sqrt((q * q).sum(-1, keepdim=True) / ql + EPS) * w_q
        c = x[:, ql:ql + D_C]
        c = c / torch.sqrt((c * c).sum(-1, keepdim=True) / D_C + EPS) * w_kv
        # to 8 significant bits
        unit = 2.0 ** (torch.floor(torch.log2(c.abs().clamp(min=1e-300))) - 7)
        c = (torch.round(c / unit) * unit).reshape(n, -1, GROUP)
        e = torch.ceil(torch.log2(c.abs().amax((1, 2)) / (6 * 448.0))).clamp(min=-120)
        c = c / 2.0 ** e[:, None, None]
        step = (c.abs().amax(-1, keepdim=True) / 6.0).to(torch.float8_e4m3fn).double()
        # the nearest level, the one of even index where two are equally near
        far = (c.abs() / step.clamp(min=2.0 ** -20))[..., None] - levels
        far = far.abs() + torch.arange(8, device="cuda") % 2 * 1e-9
        v = levels[far.argmin(-1)] * step * torch.sign(c) * 2.0 ** e[:, None, None]
        r = _spin64(x[:, None, ql + D_C:], case, torch.arange(length - n, length, device="cuda"))
        rows.append(torch.cat([v.reshape(n, D_C), r.reshape(n, D_R)], -1))
        base += n
    return dict(c_q=c_q, rows=torch.cat(rows))
