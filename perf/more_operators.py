"""Cases that measure the operators of a ragged serving step: pages given back and taken with every token's place,
rotation tables stretched for long contexts, the norm, rotation and append of a packed batch, and the attention of
its new tokens over a paged cache.

``run`` computes an operator in elementary torch operations in 32 bits (``own`` false) or calls the library
(``own`` true) on the same state; ``exact`` is the definition in 64 bits, written apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # every sequence of the repository's contiguous decode batch goes on by a token: the smallest plan
        {"name": "plan-decode", "kind": "plan", "batch": 32, "page": 64, "low": 512, "high": 8192, "prompts": 0, "longest": 1,
         "released": 0, "tokens": 32},
        # a busy server's step: most requests decode, some bring prompts, some have ended and give their pages back
        {"name": "plan-mixed", "kind": "plan", "batch": 256, "page": 16, "low": 1, "high": 8192, "prompts": 16, "longest": 2048,
         "released": 16, "tokens": 16640},
        # the tables of a model as it was trained
        {"name": "tables-short", "kind": "tables", "first": 0, "positions": 8192, "dim": 128, "base": 10000.0, "scaling": "plain",
         "factor": 1.0, "trained": 8192, "magnitude": 1.0},
        # the same for a context sixteen times as long, slow frequencies stretched, fast ones kept
        {"name": "tables-long", "kind": "tables", "first": 0, "positions": 131072, "dim": 128, "base": 500000.0, "scaling": "parts",
         "factor": 16.0, "trained": 8192, "magnitude": 1.2772588722239782},
        # the decode batch's projections: latency counts
        {"name": "append-decode", "kind": "append", "tokens": 32, "padding": 0, "q_heads": 32, "kv_heads": 8, "dim": 128, "turned": 128,
         "pairs": "halves", "norm": True, "page": 64, "far": 8192, "dtype": "bf16"},
        # a chunk of 2048 tokens of each of 8 prompts
        {"name": "append-chunk", "kind": "append", "tokens": 16384, "padding": 0, "q_heads": 32, "kv_heads": 8, "dim": 128, "turned": 128,
         "pairs": "halves", "norm": True, "page": 64, "far": 8192, "dtype": "bf16"},
        # odd sizes, half of each head turned in neighbouring pairs, a padded buffer
        {"name": "append-odd", "kind": "append", "tokens": 1543, "padding": 57, "q_heads": 64, "kv_heads": 8, "dim": 64, "turned": 32,
         "pairs": "neighbours", "norm": True, "page": 16, "far": 20000, "dtype": "fp16"},
        # the decode batch through the ragged call
        {"name": "attend-decode", "kind": "attend", "batch": 32, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "low": 511,
         "high": 8191, "prompts": 0, "longest": 1, "window": 0, "dtype": "bf16"},
        # one user's next sentence: latency counts
        {"name": "attend-one", "kind": "attend", "batch": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "low": 700,
         "high": 700, "prompts": 1, "longest": 17, "window": 0, "dtype": "fp16"},
        # a chunk of up to 2048 tokens of each of 8 prompts over what their caches hold
        {"name": "attend-chunk", "kind": "attend", "batch": 8, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "low": 0,
         "high": 6144, "prompts": 8, "longest": 2048, "window": 0, "dtype": "bf16"},
        # decoding requests and a few prompts in one call, small pages, a local window, many heads of 64
        {"name": "attend-mixed", "kind": "attend", "batch": 48, "q_heads": 64, "kv_heads": 8, "dim": 64, "page": 16, "low": 1,
         "high": 4000, "prompts": 4, "longest": 512, "window": 1000, "dtype": "fp16"},
        # the repository's windowed prompt chunks, their cache paged
        {"name": "attend-window", "kind": "attend", "batch": 8, "q_heads": 16, "kv_heads": 8, "dim": 256, "page": 128, "low": 0,
         "high": 20000, "prompts": 8, "longest": 2048, "window": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "tables", "append", "append", "attend", "attend", "attend"])
    if kind == "plan":
        c = {"kind": kind, "batch": _log(rng, 1, 512), "page": rng.choice([16, 32, 48, 64, 128, 256]), "low": rng.choice([0, 1, 100])}
        c["high"] = _log(rng, 101, 16384)
        c["prompts"] = rng.randrange(0, min(16, c["batch"]) + 1)
        c["released"] = rng.randrange(0, (c["batch"] - c["prompts"]) // 2 + 1)
        c["longest"] = _log(rng, 1, 2048)
        # the buffer holds all of them, some padding behind
        c["tokens"] = c["batch"] + c["prompts"] * c["longest"] + rng.randrange(0, 64)
        return c
    if kind == "tables":
        c = {"kind": kind, "first": rng.choice([0, 0, rng.randrange(1, 1 << 20)]), "positions": _log(rng, 1, 131072)}
        c["dim"], c["base"] = rng.choice([16, 32, 48, 64, 80, 96, 128]), rng.choice([10000.0, 500000.0, 1000000.0])
        c["scaling"] = rng.choice(["plain", "linear", "base", "parts"])
        c["factor"] = 1.0 if c["scaling"] == "plain" else rng.choice([2.0, 4.0, 8.0, 2.5, 32.0])
        c["trained"], c["magnitude"] = rng.choice([2048, 4096, 8192]), rng.choice([1.0, 1.0 + rng.random() / 2])
        return c
    c = {"kind": kind, "kv_heads": rng.choice([1, 2, 3, 4, 8]), "dtype": rng.choice(["bf16", "fp16"])}
    c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if kind == "append":
        c["dim"] = rng.choice([64, 80, 96, 128, 128, 192, 256])
        c["turned"] = rng.choice([c["dim"], 16 * rng.randrange(1, c["dim"] // 16 + 1)])
        c["pairs"], c["norm"] = rng.choice(["halves", "neighbours"]), rng.random() < 0.7
        c["page"], c["far"] = rng.choice([16, 32, 64, 128, 192]), _log(rng, 64, 65536)
        rows = c["q_heads"] + 2 * c["kv_heads"]
        c["tokens"] = _log(rng, 1, max(1, 16384 * 48 * 128 // (rows * c["dim"])))
        c["padding"] = rng.choice([0, rng.randrange(0, 100)])
        return c
    c["dim"], c["page"] = rng.choice([64, 128, 256]), rng.choice([16, 32, 48, 64, 128, 192])
    c["high"] = _log(rng, 1, 16384)
    c["low"] = rng.randrange(0, c["high"] + 1)
    c["longest"] = _log(rng, 1, 2048)
    c["window"] = rng.choice([0, 0, rng.randrange(1, c["high"] + c["longest"] + 1)])
    # no more keys, scores (the plain form pads them) and products than the largest listed
    span = c["high"] + c["longest"] + c["page"]
    most = min(64, 550000000 // (4 * c["dim"] * (c["kv_heads"] * span + c["q_heads"] * c["longest"])),
               8 * 32 * 2048 * 8192 * 128 // 2 // (c["q_heads"] * c["longest"] * span * c["dim"]))
    c["batch"] = _log(rng, 1, max(1, most))
    c["prompts"] = rng.randrange(0, c["batch"] + 1)
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 6151 + 29)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _whole(g, lo, hi, shape):
    """int32 in [lo, hi]"""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)


def _pages(tokens, page):
    return -(-tokens // page)


def _held(g, counts, page, most, spare):
    """A block table whose rows hold the pages of counts[b] tokens, scattered over a pool (-1: none), and the other
    pages of the pool as a stack of free ones with their number."""
    B = len(counts)
    n = B * most + spare
    order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    table = order[:B * most].reshape(B, most).clone()
    there = torch.arange(most, device=DEV) < _pages(counts.to(DEV), page)[:, None]
    free = torch.cat([order[B * most:], table[~there]])
    table[~there] = -1
    stack = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    stack[:len(free)] = free
    return table, stack, torch.tensor([len(free)], dtype=torch.int32, device=DEV)


def _rope(positions, dim):
    i = torch.arange(dim // 2, device=DEV, dtype=torch.float64)
    at = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / dim)
    return at.cos().float(), at.sin().float()


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": case}
    if c["kind"] == "plan":
        B, page = c["batch"], c["page"]
        cached = _whole(g, c["low"], c["high"], (B,))
        new = torch.ones_like(cached)
        order = torch.randperm(B, generator=g, device=DEV)
        prompts, ended = order[:c["prompts"]], order[c["prompts"]:c["prompts"] + c["released"]]
        new[prompts] = _whole(g, (c["longest"] + 1) // 2, c["longest"], (B,))[:len(prompts)]
        cached[prompts[::2]] = 0  # (the others go on with their prompts)
        most = _pages(c["high"] + c["longest"], page) + 1
        s["table"], s["free"], s["count"] = _held(g, cached, page, most, 16)
        s["released"] = torch.zeros_like(cached)
        s["released"][ended] = cached[ended]
        cached[ended], new[ended] = 0, 0
        s["cached"], s["new"] = cached, new
        s["between"], s["left"] = torch.zeros_like(s["count"]), torch.zeros_like(s["count"])
        s["max_pages"] = most
    elif c["kind"] == "tables":
        # (an inference program makes them when it starts, or when a longer request comes)
        s["cos"], s["sin"] = torch.zeros((2, c["positions"], c["dim"] // 2), device=DEV)
        s["magnitude"] = c["magnitude"] * (1.0 + float(torch.rand((), generator=g, device=DEV)) / 64)
    elif c["kind"] == "append":
        T, n, D, Hq, H, page = c["tokens"], c["tokens"] + c["padding"], c["dim"], c["q_heads"], c["kv_heads"], c["page"]
        dtype = DTYPES[c["dtype"]]
        qkv = _normal(g, (n, (Hq + 2 * H) * D), dtype)  # one projection's output
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], 1))
        s["q_weight"], s["k_weight"] = (1 + 0.25 * _normal(g, (2, D), dtype)).unbind(0) if c["norm"] else (None, None)
        s["positions"] = _whole(g, 0, c["far"] - 1, (n,))
        pool = _pages(T, page) + 3
        s["slots"] = torch.randperm(pool * page, generator=g, device=DEV)[:n].to(torch.int32)
        s["slots"] = torch.cat([s["slots"], s["slots"].new_full((max(0, n - pool * page),), -1)])
        s["positions"][T:], s["slots"][T:] = -1, -1
        s["k_pool"], s["v_pool"] = _normal(g, (2, pool, H, page, D), dtype)
        s["q_out"] = torch.zeros((n, Hq, D), dtype=dtype, device=DEV)
        s["rope"] = _rope(c["far"], c["turned"])
    else:
        B, page, D, Hq, H = c["batch"], c["page"], c["dim"], c["q_heads"], c["kv_heads"]
        dtype = DTYPES[c["dtype"]]
        past = _whole(g, c["low"], c["high"], (B,))
        new = torch.ones_like(past)
        prompts = torch.randperm(B, generator=g, device=DEV)[:c["prompts"]]
        new[prompts] = _whole(g, (c["longest"] + 1) // 2, c["longest"], (B,))[:c["prompts"]]
        most = _pages(c["high"] + c["longest"], page)
        s["table"], _, _ = _held(g, past + new, page, most, 3)
        total = past + new
        s["offsets"] = torch.cat([new.new_zeros(1), new.cumsum(0).to(torch.int32)])
        s["lens"] = torch.stack([past, total, past, total, torch.zeros_like(past)])
        # a buffer for the longest prompts: the rows behind the last request's stay as they are
        s["tokens"] = int(s["offsets"][-1])
        s["k"], s["v"] = _normal(g, (2, B * most + 3, H, page, D), dtype)
        s["q"] = _normal(g, (B + c["prompts"] * (c["longest"] - 1), Hq, D), dtype)
        s["out"] = torch.zeros_like(s["q"])
        s["new_most"], s["seen_most"] = int(new.max()), int(total.max())
        if c["window"]:
            s["seen_most"] = min(s["seen_most"], c["window"] - 1 + s["new_most"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"plan": _own_plan, "tables": _own_tables, "append": _own_append, "attend": _own_attend}[kind](s)
    return {"plan": _plan, "tables": _tables, "append": _append, "attend": _attend}[kind](s)


def _kept(s, make):
    """Lengths, plans and workspaces that a program makes once and keeps."""
    if "kept" not in s:
        from persistent_kv_cache_gb300 import kvc
        s["kept"] = (kvc,) + tuple(make(kvc))
    return s["kept"]


def _own_plan(s):
    c = s["case"]
    # room for the longest prompts: a request whose tokens find no row is rejected
    K, plan = _kept(s, lambda K: [K.RaggedPlan(c["batch"], max(c["tokens"], c["batch"] + c["prompts"] * c["longest"]), DEV)])
    K.kvc_page_release(s["released"], s["table"], c["page"], s["free"], s["count"], s["between"])
    K.kvc_ragged_plan(s["cached"], s["new"], s["table"], c["page"], s["free"], s["between"], s["left"], plan)
    return [plan.offsets, plan.positions[:c["tokens"]], plan.slots[:c["tokens"]], plan.lengths.buf, s["table"], s["free"], s["left"]]


def _own_tables(s):
    c = s["case"]
    K, = _kept(s, lambda K: [])
    scaling = {"plain": K.KVC_ROPE_PLAIN, "linear": K.KVC_ROPE_LINEAR, "base": K.KVC_ROPE_BASE, "parts": K.KVC_ROPE_PARTS}[c["scaling"]]
    K.kvc_rope_tables(s["cos"], s["sin"], first=c["first"], base=c["base"], scaling=scaling, factor=c["factor"],
                      trained=c["trained"], low=1.0, high=4.0, magnitude=s["magnitude"])
    return [s["cos"], s["sin"]]


def _own_append(s):
    c = s["case"]
    K, = _kept(s, lambda K: [])
    K.kvc_ragged_append(s["q_out"], s["k_pool"], s["v_pool"], s["q"], s["k"], s["v"], s["positions"], s["slots"], rope=s["rope"],
                        interleaved=c["pairs"] == "neighbours", q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)
    return [s["q_out"], s["k_pool"], s["v_pool"]]


def _own_attend(s):
    c = s["case"]

    def make(K):
        lengths = K.Lengths(c["batch"], DEV)
        lengths.buf.copy_(s["lens"])
        return [lengths, K.ragged_workspace(s["q"], s["k"], c["batch"])]
    K, lengths, ws = _kept(s, make)
    return [K.kvc_gqa_ragged(s["out"], s["q"], s["k"], s["v"], s["table"], s["offsets"], lengths,
                             local_window_size=c["window"], workspace=ws)]


# ---------------------------------------------------------------- the plain form

def _plan(s):
    c = s["case"]
    B, page, most, T = c["batch"], c["page"], s["max_pages"], c["tokens"]
    j, lines = torch.arange(most, device=DEV), torch.arange(B, device=DEV)
    # the pages of the requests that have ended go onto the stack, row by row
    back = _pages(s["released"].long(), page)
    at = s["count"] + (back.cumsum(0) - back)[:, None] + j
    gone = j < back[:, None]
    s["free"][at[gone]] = s["table"][gone]
    s["between"].copy_(s["count"] + back.sum())
    # each row takes the pages that its new tokens need from the top of the stack
    past, new = s["cached"].long(), s["new"].long()
    total = past + new
    held, need = _pages(past, page), _pages(total, page)
    want = need - held
    at = s["between"] - 1 - ((want.cumsum(0) - want)[:, None] + j - held[:, None])
    fresh = (j >= held[:, None]) & (j < need[:, None])
    s["table"][fresh] = s["free"][at[fresh]]
    s["left"].copy_(s["between"] - want.sum())
    # every token's request, position and slot
    ends = new.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(T, device=DEV)
    row = torch.searchsorted(ends, t, right=True)
    there = row < B
    row = row.clamp(max=B - 1)
    position = past[row] + t - offsets[row]
    slot = s["table"][row, (position // page).clamp(0, most - 1)].long() * page + position % page
    none = torch.full_like(t, -1)
    lens = torch.stack([past, total, past, total, torch.zeros_like(past)])
    return [offsets.int(), torch.where(there, position, none).int(), torch.where(there, slot, none).int(), lens.int(),
            s["table"], s["free"], s["left"]]


def _tables(s):
    c = s["case"]
    half = c["dim"] // 2
    i = torch.arange(half, device=DEV, dtype=torch.float64)
    base = c["base"]
    if c["scaling"] == "base":
        base = base * c["factor"] ** (c["dim"] / (c["dim"] - 2))
    speed = base ** (-i / half)
    if c["scaling"] == "linear":
        speed = speed / c["factor"]
    if c["scaling"] == "parts":
        # by how often a frequency has gone round within the trained length
        kept = ((c["trained"] * speed / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        speed = speed * kept + speed / c["factor"] * (1 - kept)
    at = torch.arange(c["first"], c["first"] + c["positions"], device=DEV, dtype=torch.float64)[:, None] * speed
    s["cos"].copy_(at.cos() * s["magnitude"])
    s["sin"].copy_(at.sin() * s["magnitude"])
    return [s["cos"], s["sin"]]


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()


def _turned(x, cos, sin, pairs):
    """the first 2 * cos.shape[-1] columns of rows x [T, heads, D] rotated"""
    r = 2 * cos.shape[-1]
    a, b = x[..., :r].chunk(2, -1) if pairs == "halves" else (x[..., 0:r:2], x[..., 1:r:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([a, b], -1) if pairs == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _append(s):
    c = s["case"]
    page = c["page"]
    there = s["slots"] >= 0
    at = s["positions"].clamp(min=0).long()
    cos, sin = s["rope"][0][at][:, None], s["rope"][1][at][:, None]
    q = _turned(_normed(s["q"], s["q_weight"]), cos, sin, c["pairs"]).to(s["q"].dtype)
    k = _turned(_normed(s["k"], s["k_weight"]), cos, sin, c["pairs"]).to(s["q"].dtype)
    s["q_out"].copy_(torch.where(there[:, None, None], q, s["q_out"]))
    slot = s["slots"][there].long()
    s["k_pool"][slot // page, :, slot % page] = k[there]
    s["v_pool"][slot // page, :, slot % page] = s["v"][there]
    return [s["q_out"], s["k_pool"], s["v_pool"]]


def _attend(s):
    c = s["case"]
    B, Hq, H, D, page, W = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["window"]
    n, keys = s["new_most"], s["seen_most"]
    offsets, past = s["offsets"].long(), s["lens"][0].long()[:, None]
    new = (offsets[1:] - offsets[:-1])[:, None]
    # queries padded to the longest request, keys from the first one that is seen
    i = torch.arange(n, device=DEV)
    token = (offsets[:-1, None] + i).clamp(max=len(s["q"]) - 1)
    q = s["q"][token].float().reshape(B, n, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * n, D)
    first = (past - W + 1).clamp(min=0) if W else torch.zeros_like(past)
    r = first + torch.arange(keys, device=DEV)
    there = r < past + new
    row = torch.where(there, r, torch.zeros_like(r))
    id = torch.gather(s["table"].long(), 1, row // page)
    k, v = (torch.where(there[..., None, None], x[id, :, row % page].float(), torch.zeros((), device=DEV)).transpose(1, 2)
            for x in (s["k"], s["v"]))
    seen = there[:, None] & (r[:, None] <= (past + i)[..., None])
    if W:
        seen &= (past + i)[..., None] - r[:, None] < W
    scores = torch.matmul(q, k.transpose(-1, -2)).div_(math.sqrt(D)).reshape(B, H, Hq // H, n, keys)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.reshape(B, H, -1, keys), v).reshape(B, H, Hq // H, n, D) / total.masked_fill(total == 0, 1.0)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(s["q"].dtype)
    s["out"][:s["tokens"]] = out[i < new]
    return [s["out"]]


# ---------------------------------------------------------------- work

def _mean_new(c):
    """mean number of new tokens of a request that brings a prompt"""
    return ((c["longest"] + 1) // 2 + c["longest"]) / 2


def work(case):
    c = case
    if c["kind"] == "plan":
        tokens = c["batch"] - c["prompts"] - c["released"] + c["prompts"] * _mean_new(c)
        pages = (tokens + c["released"] * (c["low"] + c["high"]) / 2) / c["page"]
        return {"bytes": c["batch"] * 4 * (3 + 1 + 5 + 1) + c["tokens"] * 8 + pages * 8, "flops": c["tokens"] * 4}
    if c["kind"] == "tables":
        return {"bytes": c["positions"] * c["dim"] * 4, "flops": c["positions"] * c["dim"] * 10}
    if c["kind"] == "append":
        rows = c["tokens"] * (c["q_heads"] + 2 * c["kv_heads"])
        tables = min(c["tokens"], c["far"]) * c["turned"] * 4
        return {"bytes": rows * c["dim"] * 2 * 2 + c["tokens"] * 8 + tables,
                "flops": c["tokens"] * (c["q_heads"] + c["kv_heads"]) * (3 * c["turned"] + (4 * c["dim"] if c["norm"] else 0))}
    past, D, W = (c["low"] + c["high"]) / 2, c["dim"], c["window"] or 1 << 40
    rows = scores = tokens = 0
    for count, new in ((c["batch"] - c["prompts"], 1), (c["prompts"], _mean_new(c))):
        rows += count * min(past + new, W - 1 + new)
        tokens += count * new
        # a token at position p sees min(p + 1, W) keys
        a, b = past, past + new
        grow = max(0, min(b, W) - min(a, W))
        scores += count * ((min(a, W) + min(b, W) + 1) / 2 * grow + (new - grow) * min(W, b))
    return {"bytes": rows * c["kv_heads"] * D * 2 * 2 + 2 * tokens * c["q_heads"] * D * 2, "flops": 4 * D * c["q_heads"] * scores}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "plan":
        B, page, T = c["batch"], c["page"], c["tokens"]
        table, stack = s["table"].cpu(), s["free"].cpu()
        n = int(s["count"])
        for b, gone in enumerate(s["released"].tolist()):
            for j in range(-(-gone // page)):
                stack[n] = table[b, j]
                n += 1
        offsets, positions, slots, past, total = [0], [], [], [], []
        for b, (P, S) in enumerate(zip(s["cached"].tolist(), s["new"].tolist())):
            for p in range(P, P + S):
                if p % page == 0:
                    n -= 1
                    table[b, p // page] = stack[n]
                positions.append(p)
                slots.append(int(table[b, p // page]) * page + p % page)
            offsets.append(len(positions))
            past.append(P)
            total.append(P + S)
        pad = [-1] * (T - len(positions))
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        return [t(offsets), t(positions + pad), t(slots + pad), t([past, total, past, total, [0] * B]), table.to(DEV), stack.to(DEV), t([n])]
    if c["kind"] == "tables":
        D, f, outs = c["dim"], c["factor"], []
        base = c["base"] * (f ** (D / (D - 2)) if c["scaling"] == "base" else 1.0)
        for i in range(D // 2):
            speed = math.exp(-2 * i / D * math.log(base))
            if c["scaling"] == "linear":
                speed /= f
            elif c["scaling"] == "parts":
                rounds = c["trained"] * speed / (2 * math.pi)
                g = 1.0 if rounds >= 4 else 0.0 if rounds <= 1 else (rounds - 1) / 3
                speed = (1 - g) * speed / f + g * speed
            outs.append(speed)
        p = torch.arange(c["positions"], dtype=torch.float64, device=DEV) + c["first"]
        angle = torch.outer(p, torch.tensor(outs, dtype=torch.float64, device=DEV))
        return [torch.cos(angle) * s["magnitude"], torch.sin(angle) * s["magnitude"]]
    if c["kind"] == "append":
        T, page, r = c["tokens"], c["page"], c["turned"]
        at = s["positions"][:T].long()
        angle = [x[at].double()[:, None, :] for x in s["rope"]]

        def done(x, w):
            x = x[:T].double()
            if w is not None:
                x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
            z = x.clone()
            lo = slice(0, r // 2) if c["pairs"] == "halves" else slice(0, r, 2)
            hi = slice(r // 2, r) if c["pairs"] == "halves" else slice(1, r, 2)
            z[..., lo] = x[..., lo] * angle[0] - x[..., hi] * angle[1]
            z[..., hi] = x[..., lo] * angle[1] + x[..., hi] * angle[0]
            return z
        q, k, v = s["q_out"].double(), s["k_pool"].double(), s["v_pool"].double()
        slot = s["slots"][:T].long()
        keep = slot >= 0
        q[:T][keep] = done(s["q"], s["q_weight"])[keep]
        k[slot[keep] // page, :, slot[keep] % page] = done(s["k"], s["k_weight"])[keep]
        v[slot[keep] // page, :, slot[keep] % page] = s["v"][:T].double()[keep]
        return [q, k, v]
    H, D, page, W = c["kv_heads"], c["dim"], c["page"], c["window"]
    G = c["q_heads"] // H
    if work(case)["flops"] > 3e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    offsets, past = s["offsets"].tolist(), s["lens"][0].tolist()
    for b, P in enumerate(past):
        t0, t1 = offsets[b], offsets[b + 1]
        for a in range(t0, t1, 256):
            z = min(t1, a + 256)
            p0, p1 = P + a - t0, P + z - t0
            lo = max(0, p0 - W + 1) if W else 0
            r = torch.arange(lo, p1, device=DEV)
            id = s["table"][b, r // page].long()
            k, v = (x[id, :, r % page].double() for x in (s["k"], s["v"]))
            q = s["q"][a:z].double().reshape(z - a, H, G, D)
            w = torch.einsum("thgd,rhd->htgr", q, k) / math.sqrt(D)
            back = torch.arange(p0, p1, device=DEV)[:, None] - r
            hide = (back < 0) | (back >= W) if W else back < 0
            w = torch.softmax(w.masked_fill(hide[None, :, None], -math.inf), -1)
            out[a:z] = torch.einsum("htgr,rhd->thgd", w, v).reshape(z - a, H * G, D)
    return [out]
