"""Workloads of the operators that serve ragged batches from a paged latent cache: attention of
chunks of new tokens, decode attention with a sliding window and sinks, the latent norms with the
rotation and the cache write, and the pages' turnover and compaction.

Each case runs in two forms: elementary torch operations in 32 bits (`own` false), or the calls a
program makes of this framework (`own` true).

Attention (window and chunk): query token i of sequence b stands at position
p = lens[b] - count[b] + i and sees the cached rows j <= p that are among the first `sinks` or
nearer than `window` (0: no window):
  s_j = scale (q_lat . c_j + q_rope . r_j), out = sum_j softmax(s)_j c_j, lse = ln sum_j exp(s_j);
a token that sees no row gets out = 0, lse = -inf.
"""
import math
import random

import torch

own = False

D_C, D_R, D = 512, 64, 576
PAGE = 64
SCALE = 1.0 / math.sqrt(192.0)
THETA = 10000.0
EPS = 1e-6


def listed():
    return [
        # one user far into a long stream: a single call's latency
        dict(name="window one user", op="window", batch=1, heads=128, tokens=1, ctx=5000,
             window=512, sinks=4, fp8=False, lens=1),
        # a head shard with two draft tokens to verify, FP8 cache, odd window
        dict(name="window draft fp8", op="window", batch=64, heads=16, tokens=2, ctx=8192,
             window=1000, sinks=4, fp8=True, lens=2),
        # a full decode batch with a wide window over long streams
        dict(name="window full batch", op="window", batch=128, heads=128, tokens=1, ctx=32768,
             window=4096, sinks=64, fp8=False, lens=3),
        # short turns of a few users, windowed, FP8 cache, padded batch
        dict(name="chunk short turns", op="chunk", batch=3, heads=16, ctx=700, chunk=9,
             singles=0.3, window=300, sinks=5, fp8=True, pad=5, lens=4),
        # continuous batching: decode tokens together with pieces of new prompts
        dict(name="chunk mixed batch", op="chunk", batch=64, heads=64, ctx=8192, chunk=63,
             singles=0.85, window=0, sinks=0, fp8=False, pad=0, lens=5),
        # follow-up questions on two long documents, every head
        dict(name="chunk long prefix", op="chunk", batch=2, heads=128, ctx=16500, chunk=300,
             singles=0.0, window=0, sinks=0, fp8=False, pad=0, lens=6),
        # the new tokens of a decode batch
        dict(name="norm decode batch", op="norm", batch=128, chunk=1, singles=1.0, q_lora=1536,
             ctx=8192, fp8=False, pad=0, lens=7),
        # a prefill step's tokens into an FP8 cache
        dict(name="norm prefill fp8", op="norm", batch=37, chunk=500, singles=0.2, q_lora=1536,
             ctx=4096, fp8=True, pad=3, lens=8),
        # one finished request makes room for a prompt and its three samples, FP8 pages
        dict(name="turnover small", op="turnover", layers=2, pages=300, seqs=8, done=1, forks=3,
             length=1500, fp8=True, lens=9),
        # many requests end, prompts come in, each is sampled several times
        dict(name="turnover large", op="turnover", layers=8, pages=2000, seqs=256, done=24,
             forks=140, length=2500, fp8=False, lens=10),
        # a small pool with holes
        dict(name="compact small", op="compact", layers=2, pages=301, seqs=9, live=0.5,
             fp8=True, lens=11),
        # a large pool of which a good half is live
        dict(name="compact large", op="compact", layers=8, pages=2000, seqs=250, live=0.6,
             fp8=False, lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo..hi."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9))))


def draw(rng):
    largest = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["window", "chunk", "norm", "turnover", "compact"])
        c = dict(op=op, fp8=rng.random() < 0.4, lens=rng.randrange(1 << 30))
        if op == "window":
            heads = rng.choice([16, 32, 64, 128])
            c.update(batch=_log(rng, 1, 160), heads=heads,
                     tokens=rng.randint(1, min(4, 128 // heads)), ctx=_log(rng, 40, 32768),
                     window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, rng.randint(2, 200)]))
        elif op == "chunk":
            c.update(batch=_log(rng, 1, 80), heads=rng.choice([16, 32, 64, 128]),
                     ctx=_log(rng, 40, 16500), chunk=_log(rng, 1, 300),
                     singles=round(rng.random(), 2),
                     window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                     sinks=rng.choice([0, 4, rng.randint(1, 200)]), pad=rng.choice([0, 0, 7]))
        elif op == "norm":
            c.update(batch=_log(rng, 1, 200), chunk=_log(rng, 1, 500),
                     singles=round(rng.random(), 2), q_lora=64 * rng.randint(0, 28),
                     ctx=_log(rng, 600, 16000), pad=rng.choice([0, 5]))
        elif op == "turnover":
            pages, seqs = _log(rng, 60, 3000), _log(rng, 2, 300)
            c.update(layers=_log(rng, 1, 9), pages=pages, seqs=seqs,
                     done=rng.randint(1, max(1, seqs // 6)), forks=rng.randint(0, seqs),
                     length=_log(rng, 1, 3000))
        else:
            c.update(layers=_log(rng, 1, 9), pages=_log(rng, 20, 3000), seqs=_log(rng, 1, 300),
                     live=round(rng.uniform(0.05, 1.0), 2))
        if _cost(c) <= largest:
            return c


# ------------------------------------------------------------------ shapes from the case alone

def _ragged(case):
    """(new tokens, length after them) of every sequence."""
    rng = random.Random(case["lens"])
    if case["op"] == "window":
        n = case["tokens"]
        lens = [_log(rng, 1, case["ctx"]) if rng.random() < 0.3 else
                rng.randint(max(1, case["ctx"] // 2), case["ctx"]) for _ in range(case["batch"])]
        return [n] * case["batch"], lens
    counts, lens = [], []
    for _ in range(case["batch"]):
        n = 1 if rng.random() < case["singles"] else rng.randint(
            max(1, case["chunk"] // 3), case["chunk"])
        n = min(n, case["ctx"])
        counts.append(n)
        lens.append(rng.randint(max(n, case["ctx"] // 3), case["ctx"]))
    return counts, lens


def _visible(p, window, sinks):
    """How many rows a token at position p sees."""
    if p < 0:
        return 0
    if not window or window > p:
        return p + 1
    return window + min(sinks, p + 1 - window)


def _rows_read(count, length, window, sinks):
    """How many cached rows the tokens of one sequence see between them."""
    if not window:
        return length
    first = max(0, length - count - window + 1)
    return length - first + min(sinks, first)


def _turnover_plan(case):
    """Lengths of the sequences that stay, and the finished rows', prompts' and forks' plan, so
    that everything fits the pool."""
    rng = random.Random(case["lens"])
    room = case["pages"]
    stay, done = case["seqs"], case["done"]
    forks = case["forks"]
    prompts = []
    for _ in range(done):
        n = rng.randint(max(1, case["length"] // 2), case["length"])
        n = min(n, max(1, room // (2 * done)) * PAGE)
        prompts.append(n)
        room -= -(-n // PAGE)
    forks = min(forks, max(0, room // 2))
    room -= forks
    kept = []
    for _ in range(stay):
        n = min(rng.randint(0, case["length"]), max(0, room) * PAGE)
        kept.append(n)
        room -= -(-n // PAGE)
    parents = [rng.randrange(done) for _ in range(forks)]
    return kept, prompts, parents


def _compact_plan(case):
    """Lengths of the sequences; together they hold about the live share of the pool."""
    rng = random.Random(case["lens"])
    goal = int(case["pages"] * case["live"])
    lens, used = [], 0
    for k in range(case["seqs"]):
        share = max(0, goal - used) / (case["seqs"] - k)
        pages = min(goal - used, round(share * rng.uniform(0.3, 1.7)))
        lens.append(max(0, pages * PAGE - rng.randint(0, PAGE - 1)) if pages > 0 else 0)
        used += -(-lens[-1] // PAGE)
    return lens


def _page_bytes(fp8):
    return PAGE * D + PAGE if fp8 else PAGE * D * 2


def work(case):
    row = D + 1 if case["fp8"] else 2 * D
    op = case["op"]
    if op in ("window", "chunk"):
        counts, lens = _ragged(case)
        w, s = case["window"], case["sinks"]
        seen = sum(_visible(n - c + i, w, s) for c, n in zip(counts, lens) for i in range(c))
        rows = sum(counts) * case["heads"]
        read = sum(_rows_read(c, n, w, s) for c, n in zip(counts, lens))
        return {"bytes": rows * (2 * D + 2 * D_C + 4) + read * row,
                "flops": seen * case["heads"] * 2 * (D + D_C)}
    if op == "norm":
        t = sum(_ragged(case)[0])
        return {"bytes": t * (2 * (case["q_lora"] + D) + 2 * case["q_lora"] + row),
                "flops": t * 4 * (case["q_lora"] + D)}
    if op == "turnover":
        kept, prompts, parents = _turnover_plan(case)
        copied = sum(1 for p in parents if prompts[p] % PAGE)
        held = sum(-(-prompts[p] // PAGE) for p in parents) + sum(-(-n // PAGE) for n in prompts)
        return {"bytes": 2 * copied * case["layers"] * _page_bytes(case["fp8"]) + 12 * held +
                4 * case["pages"], "flops": 0}
    lens = _compact_plan(case)
    used = sum(-(-n // PAGE) for n in lens)
    # pages held at random places of the pool: those past the first `used` move
    moved = used * (case["pages"] - used) / case["pages"]
    return {"bytes": 2 * moved * case["layers"] * _page_bytes(case["fp8"]) + 8 * used +
            8 * case["pages"], "flops": 0}


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.7e12, w["flops"] / 1.5e15)


# ------------------------------------------------------------------------------- inputs

def _cache(gen, blocks, fp8):
    """Latent rows of unit size; FP8: codes and exponents that stand for such rows."""
    if not fp8:
        return dict(cache=torch.randn(blocks, PAGE, D, device="cuda", generator=gen,
                                      dtype=torch.float32).to(torch.bfloat16))
    x = torch.randn(blocks, PAGE, D, device="cuda", generator=gen) * 64.0
    exps = torch.randint(-7, -4, (blocks, PAGE), device="cuda", generator=gen).to(torch.int8)
    return dict(codes=x.to(torch.float8_e4m3fn).view(torch.uint8), exps=exps)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, fp8 = case["op"], case["fp8"]
    st = dict(op=op, fp8=fp8)
    if op in ("window", "chunk", "norm"):
        counts, lens = _ragged(case)
        pad = case.get("pad", 0)
        total = sum(counts)
        st.update(batch=case["batch"], most=max(counts), ctx=case["ctx"], total=total,
                  lens=_int(lens),
                  starts=_int([sum(counts[:b]) for b in range(len(counts) + 1)]))
        blocks = -(-case["ctx"] // PAGE)
        tile = torch.arange(blocks, device="cuda")
        last = (st["lens"] + PAGE - 1) // PAGE
        held = tile < last[:, None]
        if op == "norm":
            st.update(q_lora=case["q_lora"])
            width = case["q_lora"] + D
            # projections of hidden states: unit size with a scale of its own for each token
            x = torch.randn(total + pad, width, device="cuda", generator=gen)
            x *= torch.rand(total + pad, 1, device="cuda", generator=gen) * 4 + 0.05
            st["x"] = x.to(torch.bfloat16)
            for k, n in (("w_q", case["q_lora"]), ("w_kv", D_C)):
                st[k] = (1 + 0.2 * torch.randn(n, device="cuda", generator=gen)).to(torch.bfloat16)
            st["c_q"] = torch.zeros(total + pad, case["q_lora"], device="cuda",
                                    dtype=torch.bfloat16)
            # only the pages that this step writes are there
            first = (st["lens"] - (st["starts"][1:] - st["starts"][:-1])) // PAGE
            held &= tile >= first[:, None]
        else:
            st.update(heads=case["heads"], window=case["window"], sinks=case["sinks"])
            q = torch.randn(total + pad, case["heads"], D, device="cuda", generator=gen)
            q = (0.6 * q).to(torch.bfloat16)
            shape = (total + pad, case["heads"])
            if op == "window":
                shape = (case["batch"], case["tokens"], case["heads"])
            st["q_lat"] = q[..., :D_C].reshape(*shape, D_C).contiguous()
            st["q_rope"] = q[..., D_C:].reshape(*shape, D_R).contiguous()
            st["out"] = torch.zeros(*shape, D_C, device="cuda", dtype=torch.bfloat16)
            st["lse"] = torch.zeros(*shape, device="cuda")
            if case["window"]:
                # pages that no token sees any more were given back
                first = st["lens"] - (st["starts"][1:] - st["starts"][:-1]) - case["window"] + 1
                held &= ((tile + 1) * PAGE > first[:, None]) | (tile * PAGE < case["sinks"])
        pool = int(held.sum())
        table = torch.full((case["batch"], blocks), -1, dtype=torch.int32, device="cuda")
        table[held] = torch.randperm(pool, device="cuda", generator=gen).to(torch.int32)
        st["table"] = table
        st.update(_cache(gen, max(1, pool), fp8))
        return st
    layers, pages = case["layers"], case["pages"]
    if fp8:
        st["pools"] = [torch.randint(0, 256, (layers, pages, PAGE, D), device="cuda",
                                     generator=gen, dtype=torch.uint8),
                       torch.randint(-9, 9, (layers, pages, PAGE), device="cuda", generator=gen,
                                     dtype=torch.int8)]
    else:
        st["pools"] = [torch.randint(-32768, 32767, (layers, pages, PAGE, D), device="cuda",
                                     generator=gen, dtype=torch.int16)]
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    if op == "compact":
        lens = _compact_plan(case)
        rows = len(lens)
    else:
        kept, prompts, parents = _turnover_plan(case)
        # a finished row held a sequence as long as the prompt that follows it
        rng = random.Random(seed)
        lens = kept + [rng.randint(max(0, n - PAGE), n) for n in prompts] + [0] * len(parents)
        rows = len(lens)
        first, child = len(kept), len(kept) + len(prompts)
        st.update(done=_int(list(range(first, rows))),
                  fresh=_int(list(range(first, child))), prompts=_int(prompts),
                  parents=_int([first + p for p in parents]),
                  children=_int(list(range(child, rows))))
    most = max(1, -(-max(lens + [case.get("length", 0)]) // PAGE))
    st["lens"] = _int(lens)
    held = torch.arange(most, device="cuda") < ((st["lens"] + PAGE - 1) // PAGE)[:, None]
    table = torch.full((rows, most), -1, dtype=torch.int32, device="cuda")
    table[held] = order[:int(held.sum())]
    st["table"] = table
    st["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    st["refs"][table[held].long()] = 1
    if op == "compact":
        st["refs_out"] = torch.zeros_like(st["refs"])
        st["table_out"] = torch.zeros_like(table)
        st["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


# -------------------------------------------------------------------------- plain forms

def _read_rows(st, page, slot):
    """Cached rows in 32 bits."""
    if not st["fp8"]:
        return st["cache"][page, slot].float()
    e = st["exps"][page, slot].float()
    return st["codes"].view(torch.float8_e4m3fn)[page, slot].float() * torch.exp2(e)[..., None]


def _attend(st):
    """Attention of all sequences at once, padded to the most tokens and rows of one."""
    dev, b, n, heads = "cuda", st["batch"], st["most"], st["heads"]
    window, sinks = st["window"], st["sinks"]
    starts, lens = st["starts"].long(), st["lens"].long()
    counts = starts[1:] - starts[:-1]
    i = torch.arange(n, device=dev)
    token = starts[:-1, None] + i
    live = i < counts[:, None]
    pos = (lens - counts)[:, None] + i
    if window:
        span = min(window + n - 1, st["ctx"])
        front = torch.arange(min(sinks, st["ctx"]), device=dev).expand(b, -1)
        near = (lens - counts - window + 1).clamp(min=0)[:, None] + torch.arange(span, device=dev)
        rows = torch.cat([front, near], 1)
        once = torch.cat([torch.ones_like(front, dtype=torch.bool), near >= sinks], 1)
    else:
        rows = torch.arange(st["ctx"], device=dev).expand(b, -1)
        once = torch.ones_like(rows, dtype=torch.bool)
    once &= rows < lens[:, None]
    sees = live[:, :, None] & once[:, None, :] & (rows[:, None, :] <= pos[:, :, None])
    if window:
        sees &= (rows[:, None, :] < sinks) | (rows[:, None, :] > pos[:, :, None] - window)
    safe = torch.where(once, rows, 0)
    page = torch.gather(st["table"].long(), 1, safe // PAGE).clamp(min=0)
    kv = torch.where(once[..., None], _read_rows(st, page, safe % PAGE), 0.0)
    q = torch.cat([st["q_lat"].reshape(-1, heads, D_C), st["q_rope"].reshape(-1, heads, D_R)], -1)
    q = q[torch.where(live, token, 0)].float().reshape(b, n * heads, D)
    s = torch.matmul(q, kv.transpose(1, 2)).mul_(SCALE).reshape(b, n, heads, -1)
    s.masked_fill_(~sees[:, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    out = torch.matmul(s.reshape(b, n * heads, -1), kv[..., :D_C]).reshape(b, n, heads, D_C)
    out = torch.where(total > 0, out / total, 0.0).to(torch.bfloat16)
    st["out"].view(-1, heads, D_C)[token[live]] = out[live]
    st["lse"].view(-1, heads)[token[live]] = lse[..., 0][live]
    return dict(out=st["out"], lse=st["lse"])


def _norm(st):
    """Both norms, the rotation and the write of all tokens."""
    ql = st["q_lora"]
    starts, lens = st["starts"].long(), st["lens"].long()
    total = st["total"]
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[b] - starts[b + 1] + t
    x = st["x"][:total].float()
    if ql:
        c = x[:, :ql]
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * st["w_q"].float()
        st["c_q"][:total] = c.to(torch.bfloat16)
    c = x[:, ql:ql + D_C]
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * st["w_kv"].float()
    i = torch.arange(D_R // 2, device="cuda", dtype=torch.float64)
    turn = pos.double()[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64,
                                                          device="cuda"), -2.0 * i / D_R)
    co, si = turn.cos().float(), turn.sin().float()
    r = x[:, ql + D_C:].reshape(total, D_R // 2, 2)
    r = torch.stack([r[..., 0] * co - r[..., 1] * si, r[..., 0] * si + r[..., 1] * co], -1)
    row = torch.cat([c, r.reshape(total, D_R)], -1)
    page, slot = st["table"].long()[b, pos // PAGE], pos % PAGE
    if not st["fp8"]:
        st["cache"][page, slot] = row.to(torch.bfloat16)
        return dict(c_q=st["c_q"], cache=st["cache"])
    # the smallest e with max |x| 2^-e <= 448 = 1.75 * 2^8
    f, k = torch.frexp(row.abs().amax(-1))
    e = torch.where(f <= 0.875, k - 9, k - 8).clamp(min=-126)
    e = torch.where(row.abs().amax(-1) > 0, e, 0)
    st["codes"][page, slot] = (row * torch.exp2(-e.float())[:, None]).to(
        torch.float8_e4m3fn).view(torch.uint8)
    st["exps"][page, slot] = e.to(torch.int8)
    return dict(c_q=st["c_q"], codes=st["codes"].view(torch.float8_e4m3fn), exps=st["exps"])


def _turnover(st):
    """Finished rows release their pages, prompts take the lowest free ones, forks share them."""
    refs, table, lens = st["refs"], st["table"], st["lens"]
    tile = torch.arange(table.shape[1], device="cuda")
    # release
    rows = st["done"].long()
    held = tile < ((lens[rows] + PAGE - 1) // PAGE)[:, None]
    ids = torch.where(held, table[rows], 0).long()
    refs.index_add_(0, ids.reshape(-1), -held.reshape(-1).to(torch.int32))
    table[rows] = torch.where(held, -1, table[rows])
    lens[rows] = 0
    # prompts: the lowest free pages, in the order of the list
    free = torch.sort((refs > 0).to(torch.int8), stable=True).indices.to(torch.int32)
    rows, new = st["fresh"].long(), st["prompts"]
    need = (new + PAGE - 1) // PAGE
    place = torch.cumsum(need, 0) - need
    held = tile < need[:, None]
    ids = free[torch.where(held, place[:, None] + tile, 0).clamp(max=len(free) - 1)]
    table[rows] = torch.where(held, ids, table[rows])
    refs.index_add_(0, torch.where(held, ids, 0).long().reshape(-1),
                    held.reshape(-1).to(torch.int32))
    lens[rows] = new
    if st["parents"].numel():
        # forks: full pages shared, the last partial one copied to the lowest free page
        par, child = st["parents"].long(), st["children"].long()
        length = lens[par]
        part = length % PAGE > 0
        free = torch.sort((refs > 0).to(torch.int8), stable=True).indices.to(torch.int32)
        place = torch.cumsum(part.to(torch.int32), 0) - 1
        taken = free[place.clamp(min=0)]
        full = tile < (length // PAGE)[:, None]
        ids = table[par]
        refs.index_add_(0, torch.where(full, ids, 0).long().reshape(-1),
                        full.reshape(-1).to(torch.int32))
        refs.index_add_(0, torch.where(part, taken, 0).long(), part.to(torch.int32))
        src = torch.gather(ids, 1, (length // PAGE).clamp(max=len(tile) - 1).long()[:, None])[:, 0]
        edge = part[:, None] & (tile == (length // PAGE)[:, None])
        table[child] = torch.where(full, ids, torch.where(edge, taken[:, None], table[child]))
        lens[child] = length
        for p in st["pools"]:
            p[:, taken[part].long()] = p[:, src[part].long()]
    return dict(refs=refs, table=table, lens=lens, pools=st["pools"])


def _compact(st):
    """Live pages past the number of live pages move into the holes before it."""
    refs, table, lens = st["refs"], st["table"], st["lens"]
    is_live = refs > 0
    count = is_live.sum()
    ids = torch.arange(len(refs), device="cuda")
    moves = ids[is_live & (ids >= count)]
    holes = ids[~is_live & (ids < count)]
    to = ids.clone()
    to[moves] = holes
    held = torch.arange(table.shape[1], device="cuda") < ((lens + PAGE - 1) // PAGE)[:, None]
    st["table_out"].copy_(torch.where(held, to[table.long().clamp(min=0)].to(torch.int32), table))
    st["refs_out"].zero_()
    st["refs_out"][to[is_live]] = refs[is_live]
    st["live"].copy_(count.reshape(1))
    for p in st["pools"]:
        p[:, holes] = p[:, moves]
    return dict(refs=st["refs_out"], table=st["table_out"], live=st["live"], pools=st["pools"])


# ------------------------------------------------------------------- the framework's calls

def _kept(st, size):
    """The workspace that a program keeps for a shape."""
    if "workspace" not in st:
        from mla_latent_kv_13_gb300 import mla
        st["workspace"] = mla.alloc_workspace(size(mla))
    return st["workspace"]


def _own(st):
    from mla_latent_kv_13_gb300 import mla
    op, fp8 = st["op"], st["fp8"]
    if op == "window":
        b, n, h, _ = st["q_lat"].shape
        ws = _kept(st, lambda m: m.decode_window_workspace_size(b, n, h, st["ctx"], st["window"],
                                                                st["sinks"]))
        cache = (st["codes"], st["exps"]) if fp8 else (st["cache"],)
        call = mla.decode_attention_window_fp8 if fp8 else mla.decode_attention_window
        call(st["q_lat"], st["q_rope"], *cache, st["table"], st["lens"], st["ctx"], st["window"],
             st["sinks"], SCALE, out=st["out"], lse=st["lse"], workspace=ws)
        return dict(out=st["out"], lse=st["lse"])
    if op == "chunk":
        t, h, _ = st["q_lat"].shape
        ws = _kept(st, lambda m: m.chunk_workspace_size(st["batch"], t, h, st["ctx"],
                                                        st["window"], st["sinks"]))
        cache = (st["codes"], st["exps"]) if fp8 else (st["cache"],)
        call = mla.chunk_attention_fp8 if fp8 else mla.chunk_attention
        call(st["q_lat"], st["q_rope"], *cache, st["table"], st["starts"], st["lens"], st["ctx"],
             SCALE, window=st["window"], sinks=st["sinks"], out=st["out"], lse=st["lse"],
             workspace=ws)
        return dict(out=st["out"], lse=st["lse"])
    if op == "norm":
        ws = _kept(st, lambda m: m.WS_HEADER_BYTES)
        if fp8:
            mla.norm_rope_append_fp8(st["x"], st["w_q"], st["w_kv"], st["starts"], st["lens"],
                                     st["table"], st["codes"], st["exps"], THETA, EPS,
                                     c_q=st["c_q"], workspace=ws)
            return dict(c_q=st["c_q"], codes=st["codes"].view(torch.float8_e4m3fn),
                        exps=st["exps"])
        mla.norm_rope_append(st["x"], st["w_q"], st["w_kv"], st["starts"], st["lens"],
                             st["table"], st["cache"], THETA, EPS, c_q=st["c_q"], workspace=ws)
        return dict(c_q=st["c_q"], cache=st["cache"])
    rows, pages = len(st["lens"]), len(st["refs"])
    ws = _kept(st, lambda m: m.pages_workspace_size(pages, rows))
    if op == "turnover":
        mla.pages_free(st["refs"], st["table"], st["lens"], st["done"], ws)
        mla.pages_extend(st["refs"], st["table"], st["lens"], st["fresh"], st["prompts"], ws)
        if st["parents"].numel():
            mla.pages_fork(st["refs"], st["table"], st["lens"], st["parents"], st["children"],
                           st["pools"], ws)
        return dict(refs=st["refs"], table=st["table"], lens=st["lens"], pools=st["pools"])
    mla.pages_compact(st["refs"], st["table"], st["lens"], st["pools"], refs_out=st["refs_out"],
                      table_out=st["table_out"], live=st["live"], workspace=ws)
    return dict(refs=st["refs_out"], table=st["table_out"], live=st["live"], pools=st["pools"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op in ("window", "chunk"):
        return _attend(state)
    return {"norm": _norm, "turnover": _turnover, "compact": _compact}[op](state)


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("turnover", "compact") or work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    counts, lens = _ragged(case)
    table = st["table"].long()
    if st["fp8"]:
        pool = st["codes"].view(torch.float8_e4m3fn).double()
        pool = pool * 2.0 ** st["exps"].double()[..., None]
    else:
        pool = st["cache"].double()
    if op == "norm":
        return _exact_norm(st, counts, lens, table, pool)
    heads = case["heads"]
    q_lat = st["q_lat"].reshape(-1, heads, D_C)
    q_rope = st["q_rope"].reshape(-1, heads, D_R)
    out = torch.zeros(q_lat.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q_lat.shape[:2], dtype=torch.float64, device="cuda")
    base = 0
    for b, (n, length) in enumerate(zip(counts, lens)):
        j = torch.arange(length, device="cuda")
        for i in range(0, n, 32):
            at = torch.arange(i, min(n, i + 32), device="cuda")
            p = length - n + at
            seen = j[None, :] <= p[:, None]
            if case["window"]:
                seen = seen & ((j < case["sinks"]) | (j[None, :] > p[:, None] - case["window"]))
            js = j[seen.any(0)]
            seen = seen[:, seen.any(0)]
            kv = pool[table[b, js // PAGE], js % PAGE]
            s = torch.einsum("nhd,kd->nhk", q_lat[base + at].double(), kv[:, :D_C])
            s += torch.einsum("nhd,kd->nhk", q_rope[base + at].double(), kv[:, D_C:])
            s = torch.where(seen[:, None, :], s * SCALE, -math.inf)
            total = torch.logsumexp(s, -1)
            p_ = torch.where(seen[:, None, :], torch.exp(s - total[..., None]), 0.0)
            out[base + at] = torch.einsum("nhk,kd->nhd", p_, kv[:, :D_C])
            lse[base + at] = total
        base += n
    return dict(out=out.reshape(st["out"].shape), lse=lse.reshape(st["lse"].shape))


def _exact_norm(st, counts, lens, table, pool):
    ql = st["q_lora"]
    c_q = st["c_q"].double()
    if st["fp8"]:
        codes, exps = st["codes"].view(torch.float8_e4m3fn).double(), st["exps"].clone()
    w_q, w_kv = st["w_q"].double(), st["w_kv"].double()
    freq = torch.tensor([THETA ** (-2.0 * i / D_R) for i in range(D_R // 2)],
                        dtype=torch.float64, device="cuda")
    base = 0
    for b, (n, length) in enumerate(zip(counts, lens)):
        x = st["x"][base:base + n].double()
        if ql:
            q = x[:, :ql]
            c_q[base:base + n] = q / torch.sqrt((q * q).sum(-1, keepdim=True) / ql + EPS) * w_q
        kv, r = x[:, ql:ql + D_C], x[:, ql + D_C:]
        kv = kv / torch.sqrt((kv * kv).sum(-1, keepdim=True) / D_C + EPS) * w_kv
        p = torch.arange(length - n, length, device="cuda")
        z = torch.polar(torch.ones(n, D_R // 2, dtype=torch.float64, device="cuda"),
                        p.double()[:, None] * freq)
        r = torch.view_as_real(torch.complex(r[:, 0::2], r[:, 1::2]) * z).reshape(n, D_R)
        row = torch.cat([kv, r], 1)
        at = (table[b, p // PAGE], p % PAGE)
        if st["fp8"]:
            e = torch.ceil(torch.log2(row.abs().amax(1) / 448.0)).clamp(min=-126)
            codes[at] = (row / 2.0 ** e[:, None]).to(torch.float8_e4m3fn).double()
            exps[at] = e.to(torch.int8)
        else:
            pool[at] = row
        base += n
    if st["fp8"]:
        return dict(c_q=c_q, codes=codes, exps=exps)
    return dict(c_q=c_q, cache=pool)
