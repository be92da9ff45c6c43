"""Cases that measure the cache operators: rows quantised as they are written and attention over them, attention
for a tree of drafted tokens, and attention over the pages that a cheap score selects.

``run`` computes an operator in elementary torch operations in 32 bits (``own`` false) or calls the library
(``own`` true) on the same state; ``exact`` is the definition in 64 bits, written apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


def listed():
    return [
        # one prompt chunk of 8 sequences goes into an int8 cache, which the next chunk's attention reads back in 16 bits
        {"name": "quant-write-chunk", "kind": "quant_write", "batch": 8, "kv_heads": 8, "dim": 128, "cap": 4096, "new": 2048,
         "past": 2048, "ring": False, "codes": "int8", "dtype": "bf16"},
        # one token of 4 sequences into a ring of 128 slots: the smallest call
        {"name": "quant-write-token", "kind": "quant_write", "batch": 4, "kv_heads": 8, "dim": 64, "cap": 128, "new": 1,
         "past": 5000, "ring": True, "codes": "e4m3", "dtype": "fp16"},
        # the repository's contiguous decode workload with the cache held in int8
        {"name": "quant-decode-contiguous", "kind": "quant_decode", "batch": 32, "q_heads": 32, "kv_heads": 8, "dim": 128, "cap": 8192,
         "low": 512, "high": 8192, "ring": False, "window": 0, "codes": "int8", "dtype": "bf16"},
        # the repository's head_dim-256 ring workload in e4m3
        {"name": "quant-decode-ring", "kind": "quant_decode", "batch": 8, "q_heads": 16, "kv_heads": 8, "dim": 256, "cap": 4096,
         "low": 1, "high": 20000, "ring": True, "window": 4096, "codes": "e4m3", "dtype": "bf16"},
        # one user's short conversation: latency counts
        {"name": "quant-decode-one", "kind": "quant_decode", "batch": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "cap": 1024,
         "low": 577, "high": 577, "ring": False, "window": 0, "codes": "e4m3", "dtype": "fp16"},
        # 32 drafts a sequence verified over the contiguous decode workload's cache
        {"name": "tree-batch", "kind": "tree", "batch": 32, "q_heads": 32, "kv_heads": 8, "dim": 128, "cap": 8192, "nodes": 32,
         "low": 512, "high": 8160, "page": 0, "window": 0, "ragged": False, "dtype": "bf16"},
        # one user, 8 drafts: latency counts
        {"name": "tree-one", "kind": "tree", "batch": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "cap": 1024, "nodes": 8,
         "low": 700, "high": 700, "page": 0, "window": 0, "ragged": False, "dtype": "bf16"},
        # trees of different sizes over a paged cache with a local window
        {"name": "tree-paged-ragged", "kind": "tree", "batch": 6, "q_heads": 64, "kv_heads": 8, "dim": 64, "cap": 4096, "nodes": 61,
         "low": 1, "high": 4000, "page": 64, "window": 1000, "ragged": True, "dtype": "fp16"},
        # the bounds of every page that a long prompt filled
        {"name": "page-bounds-prompt", "kind": "page_bounds", "batch": 8, "kv_heads": 8, "dim": 128, "page": 64, "new": 16384,
         "past": 0, "dtype": "bf16"},
        # those of one chunk over larger pages
        {"name": "page-bounds-chunk", "kind": "page_bounds", "batch": 2, "kv_heads": 8, "dim": 64, "page": 128, "new": 500,
         "past": 5000, "dtype": "fp16"},
        # eight long documents, 64 of up to 2048 pages read for each head
        {"name": "sparse-long", "kind": "sparse", "batch": 8, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "low": 16384,
         "high": 131072, "select": 64, "sink": 1, "recent": 2, "dtype": "bf16"},
        # one shorter document: latency counts
        {"name": "sparse-one", "kind": "sparse", "batch": 1, "q_heads": 16, "kv_heads": 8, "dim": 64, "page": 64, "low": 4097,
         "high": 4097, "select": 16, "sink": 1, "recent": 1, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quant_write", "quant_decode", "quant_decode", "tree", "tree", "page_bounds", "sparse"])
    dim = rng.choice([64, 128, 256])
    c = {"kind": kind, "kv_heads": rng.choice([1, 2, 3, 4, 8]), "dim": dim, "dtype": rng.choice(["bf16", "fp16"])}
    if kind == "quant_write":
        c["codes"], c["ring"] = rng.choice(["int8", "e4m3"]), rng.random() < 0.5
        c["new"], c["past"] = _log(rng, 1, 2048), _log(rng, 1, 6000) - 1
        c["cap"] = max(c["new"], _log(rng, 64, 4096)) if c["ring"] else c["new"] + c["past"] + rng.randrange(64)
        c["batch"] = _log(rng, 1, max(1, min(32, 8 * 8 * 4096 * 128 // (c["kv_heads"] * c["cap"] * dim))))
    elif kind == "quant_decode":
        c["codes"], c["ring"] = rng.choice(["int8", "e4m3"]), rng.random() < 0.5
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
        c["cap"] = _log(rng, 17, 32768)
        c["high"] = 4 * c["cap"] if c["ring"] else c["cap"]
        c["low"] = rng.randrange(1, c["high"] + 1)
        c["window"] = rng.choice([0, rng.randrange(1, c["cap"] + 1)])
        c["batch"] = _log(rng, 1, max(1, min(64, 32 * 8 * 4096 * 128 // (c["kv_heads"] * c["cap"] * dim))))
    elif kind == "tree":
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8, 16])
        c["nodes"], c["page"] = _log(rng, 1, 96), rng.choice([0, 64, 128, 192])
        c["cap"] = _log(rng, 256, 16384)
        if c["page"]:
            c["cap"] = -(-c["cap"] // c["page"]) * c["page"]
        c["high"] = c["cap"] - c["nodes"]
        c["low"] = rng.randrange(0, c["high"] + 1)
        c["window"] = rng.choice([0, 0, rng.randrange(1, c["cap"] + 1)])
        c["ragged"] = rng.random() < 0.5
        rows = c["kv_heads"] * c["cap"] * dim * max(128, c["nodes"] * c["q_heads"] // c["kv_heads"]) // 128
        c["batch"] = _log(rng, 1, max(1, min(48, 32 * 8 * 8192 * 128 // 2 // rows)))
    elif kind == "page_bounds":
        c["page"], c["new"], c["past"] = rng.choice([64, 128, 256]), _log(rng, 64, 16384), _log(rng, 1, 8192) - 1
        c["batch"] = _log(rng, 1, max(1, min(16, 8 * 8 * 16384 * 128 // (c["kv_heads"] * (c["new"] + c["past"]) * dim))))
    else:
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 5, 8, 16])
        c["page"] = rng.choice([64, 128, 256])
        c["high"] = _log(rng, 512, 131072)
        c["low"] = rng.randrange(1, c["high"] + 1)
        c["sink"], c["recent"] = rng.randrange(3), rng.randrange(1, 4)
        c["select"] = max(c["sink"] + c["recent"], _log(rng, 2, 8192 // c["page"]))
        c["batch"] = _log(rng, 1, max(1, min(16, 8 * 8 * 131072 * 128 // (c["kv_heads"] * c["high"] * dim))))
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _whole(g, lo, hi, shape):
    """int32 in [lo, hi]"""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)


def _rope(positions, dim):
    i = torch.arange(dim // 2, device=DEV, dtype=torch.float64)
    at = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / dim)
    return at.cos().float(), at.sin().float()


def _codes(g, shape, codes):
    """What a quantised cache of normal rows holds: codes and one scale a row."""
    top = TOP[codes]
    x = (_normal(g, shape, torch.float16) * (top / 3.5)).clamp_(-top, top)
    x = x.round_().to(torch.int8) if codes == "int8" else x.to(CODES[codes])
    scale = torch.exp(0.5 * _normal(g, shape[:-1], torch.float32)) * (3.5 / top)
    return x, scale


def _tree_of(case, g):
    """parents [B, N] (-1: follows the cache, -2: absent), an accepted path [B, N] from the root with its length [B]"""
    B, N = case["batch"], case["nodes"]
    u = torch.rand((2, B, N), generator=g, device=DEV).tolist()
    size = _whole(g, (N + 1) // 2 if case["ragged"] else N, N, (B,)).tolist()
    parents, path, count = [], [], []
    for b in range(B):
        p = [-2] * N
        for i in range(size[b]):
            p[i] = -1 if i == 0 else max(-1, i - 1 - int(u[0][b][i] ** 2 * (i + 1)))
        at, line = int(u[1][b][0] * size[b]), []
        while at >= 0:
            line.append(at)
            at = p[at]
        parents.append(p)
        path.append((line[::-1] + [-1] * N)[:N])
        count.append(len(line))
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return t(parents), t(path), t(count)


def _pool(g, shape, dtype, per_page):
    """keys whose pages differ, as those of a text's passages do"""
    k = _normal(g, shape, dtype)
    return k.add_(per_page * _normal(g, shape[:2] + (1,) + shape[3:], dtype))


def _bounds_of(k_pool):
    """The bounds of every page of a pool, as a program that has decoded so far holds them."""
    hi, lo = k_pool.amax(2).float(), k_pool.amin(2).float()
    scale = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    scale = scale / torch.full_like(scale, 127.0)
    code = lambda x, f: f(x / scale[..., None]).clamp_(-127, 127).to(torch.int8)  # noqa: E731
    return torch.stack([code(hi, torch.ceil), code(lo, torch.floor)], 2), scale


def prepare(case, seed):
    g, c = _gen(seed), case
    B, H, D = c["batch"], c["kv_heads"], c["dim"]
    dtype = DTYPES[c["dtype"]]
    s = {"case": case}
    if c["kind"] == "quant_write":
        C, S = c["cap"], c["new"]
        past = _whole(g, 0, c["past"], (B,))
        s["seqlens"] = past + (S - 1)
        s["kq"], s["ks"] = _codes(g, (B, H, C, D), c["codes"])
        s["vq"], s["vs"] = _codes(g, (B, H, C, D), c["codes"])
        s["new_k"], s["new_v"] = _normal(g, (B, H, S, D), dtype), _normal(g, (B, H, S, D), dtype)
        s["k_rows"], s["v_rows"] = torch.zeros((2, B, H, C, D), dtype=dtype, device=DEV)
        s["rope"] = _rope(c["past"] + S, D)
    elif c["kind"] == "quant_decode":
        s["seqlens"] = _whole(g, c["low"], c["high"], (B,)) - 1
        s["kq"], s["ks"] = _codes(g, (B, H, c["cap"], D), c["codes"])
        s["vq"], s["vs"] = _codes(g, (B, H, c["cap"], D), c["codes"])
        s["q"] = _normal(g, (B, c["q_heads"], 1, D), dtype)
        s["out"] = torch.zeros_like(s["q"])
        s["rope"] = _rope(c["high"], D)
    elif c["kind"] == "tree":
        N, C, page = c["nodes"], c["cap"], c["page"]
        s["seqlens"] = _whole(g, c["low"], c["high"], (B,)) + (N - 1)
        s["parents"], s["path"], s["accepted"] = _tree_of(case, g)
        s["table"] = None
        shape = (B, H, C, D)
        if page:
            n = B * (C // page)
            s["table"] = torch.randperm(n + 3, generator=g, device=DEV)[:n].to(torch.int32).reshape(B, C // page)
            shape = (n + 3, H, page, D)
        s["k"], s["v"] = _normal(g, shape, dtype), _normal(g, shape, dtype)
        s["new_k"], s["new_v"] = _normal(g, (B, H, N, D), dtype), _normal(g, (B, H, N, D), dtype)
        s["q"] = _normal(g, (B, c["q_heads"], N, D), dtype)
        s["out"] = torch.zeros_like(s["q"])
        s["next"] = torch.zeros_like(s["seqlens"])
        s["rope"] = _rope(C, D)
    elif c["kind"] == "page_bounds":
        page = c["page"]
        past = _whole(g, 0, c["past"], (B,))
        s["seqlens"] = past + (c["new"] - 1)
        m = -(-(c["past"] + c["new"]) // page)
        s["table"] = torch.randperm(B * m, generator=g, device=DEV).to(torch.int32).reshape(B, m)
        s["k"] = _pool(g, (B * m, H, page, D), dtype, 0.5)
        s["bounds"] = _whole(g, -127, 127, (B * m, H, 2, D)).to(torch.int8)
        s["bscale"] = torch.rand((B * m, H), generator=g, device=DEV) + 0.5
    else:
        page = c["page"]
        s["seqlens"] = _whole(g, c["low"], c["high"], (B,)) - 1
        m = -(-c["high"] // page)
        s["table"] = torch.randperm(B * m, generator=g, device=DEV).to(torch.int32).reshape(B, m)
        s["k"], s["v"] = _pool(g, (B * m, H, page, D), dtype, 0.5), _normal(g, (B * m, H, page, D), dtype)
        s["bounds"], s["bscale"] = _bounds_of(s["k"])
        s["q"] = _normal(g, (B, c["q_heads"], 1, D), dtype)
        s["out"] = torch.zeros_like(s["q"])
        s["selected"] = torch.zeros((B, H, c["select"]), dtype=torch.int32, device=DEV)
        s["rope"] = _rope(c["high"], D)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"quant_write": _own_quant_write, "quant_decode": _own_quant_decode, "tree": _own_tree,
                "page_bounds": _own_page_bounds, "sparse": _own_sparse}[kind](s)
    return {"quant_write": _quant_write, "quant_decode": _quant_decode, "tree": _tree, "page_bounds": _page_bounds,
            "sparse": _sparse}[kind](s)


def _kept(s, make):
    """Lengths and workspaces that a program makes once and keeps."""
    if "kept" not in s:
        from persistent_kv_cache_gb300 import kvc
        s["kept"] = (kvc,) + tuple(make(kvc))
    return s["kept"]


def _own_quant_write(s):
    c = s["case"]
    K, L = _kept(s, lambda K: [K.Lengths(c["batch"], DEV)])
    policy = K.KVC_RING if c["ring"] else K.KVC_CONTIGUOUS
    K.kvc_seq_lengths(s["seqlens"], c["new"], c["cap"], policy, c["cap"], out=L)
    K.kvc_quant_append(s["kq"], s["vq"], s["ks"], s["vs"], s["new_k"], s["new_v"], L, policy, rope=s["rope"])
    K.kvc_dequant_rows(s["k_rows"], s["v_rows"], s["kq"], s["vq"], s["ks"], s["vs"], L, policy)
    return [s["k_rows"], s["v_rows"], s["ks"], s["vs"]]


def _own_quant_decode(s):
    c = s["case"]
    K, L, ws = _kept(s, lambda K: [K.Lengths(c["batch"], DEV), K.quant_decode_workspace(s["q"], s["kq"])])
    policy = K.KVC_RING if c["ring"] else K.KVC_CONTIGUOUS
    K.kvc_seq_lengths(s["seqlens"], 1, c["cap"], policy, c["cap"], out=L)
    return [K.kvc_gqa_decode_quant(s["out"], s["q"], s["kq"], s["vq"], s["ks"], s["vs"], L, policy,
                                   local_window_size=c["window"], rope=s["rope"], workspace=ws)]


def _own_tree(s):
    c = s["case"]
    K, L, mask, depth, ws = _kept(s, lambda K: [K.Lengths(c["batch"], DEV), *K.tree_buffers(s["parents"]),
                                                K.tree_workspace(s["q"], s["k"])])
    K.kvc_seq_lengths(s["seqlens"], c["nodes"], c["cap"], K.KVC_CONTIGUOUS, out=L)
    K.kvc_tree_mask(s["parents"], mask, depth)
    K.kvc_tree_append(s["k"], s["v"], s["new_k"], s["new_v"], depth, L, block_table=s["table"], rope=s["rope"])
    K.kvc_gqa_tree(s["out"], s["q"], s["k"], s["v"], mask, depth, L, block_table=s["table"],
                   local_window_size=c["window"], rope=s["rope"], workspace=ws)
    K.kvc_tree_commit(s["k"], s["v"], s["path"], s["accepted"], L, s["next"], c["nodes"], block_table=s["table"])
    return [s["out"], s["k"], s["v"], s["next"]]


def _own_page_bounds(s):
    c = s["case"]
    K, L = _kept(s, lambda K: [K.Lengths(c["batch"], DEV)])
    K.kvc_seq_lengths(s["seqlens"], c["new"], s["table"].shape[1] * c["page"], K.KVC_CONTIGUOUS, out=L)
    K.kvc_page_bounds(s["bounds"], s["bscale"], s["k"], s["table"], L, c["new"])
    return [s["bounds"].float() * s["bscale"][:, :, None, None], s["bscale"]]


def _own_sparse(s):
    c = s["case"]
    K, L, ws = _kept(s, lambda K: [K.Lengths(c["batch"], DEV), K.sparse_workspace(s["q"], s["k"], s["selected"])])
    K.kvc_seq_lengths(s["seqlens"], 1, s["table"].shape[1] * c["page"], K.KVC_CONTIGUOUS, out=L)
    K.kvc_gqa_decode_sparse(s["out"], s["q"], s["k"], s["v"], s["bounds"], s["bscale"], s["table"], L, s["selected"],
                            sink_pages=c["sink"], recent_pages=c["recent"], rope=s["rope"], workspace=ws)
    return [s["out"], s["selected"]]


# ---------------------------------------------------------------- the plain form

def _rotated(x, positions, rope):
    """rows x [B, H, S, D] rotated (halves paired) at positions [B, S], in 32 bits"""
    cos, sin = rope[0][positions][:, None], rope[1][positions][:, None]
    lo, hi = x.float().chunk(2, -1)
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)


def _attend(scores, values, visible, dtype):
    """softmax over the visible keys; a row that sees none gives zeros"""
    scores = scores.masked_fill(~visible, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return (torch.matmul(p, values) / torch.where(total == 0, torch.ones_like(total), total)).to(dtype)


def _quantised(x, codes):
    top = x.abs().amax(-1)
    scale = top / torch.full_like(top, TOP[codes])
    code = x / torch.where(scale == 0, torch.ones_like(scale), scale)[..., None]
    code = code.round().clamp(-127, 127).to(torch.int8) if codes == "int8" else code.to(CODES[codes])
    return code, scale


def _quant_write(s):
    c = s["case"]
    B, S, C = c["batch"], c["new"], c["cap"]
    total = s["seqlens"].long() + 1
    at = total[:, None] - S + torch.arange(S, device=DEV)
    b, slot = torch.arange(B, device=DEV)[:, None], at % C
    kc, ks = _quantised(_rotated(s["new_k"], at, s["rope"]), c["codes"])
    vc, vs = _quantised(s["new_v"].float(), c["codes"])
    s["kq"].view(torch.uint8)[b, :, slot] = kc.view(torch.uint8).transpose(1, 2)
    s["vq"].view(torch.uint8)[b, :, slot] = vc.view(torch.uint8).transpose(1, 2)
    s["ks"][b, :, slot], s["vs"][b, :, slot] = ks.transpose(1, 2), vs.transpose(1, 2)
    # back in 16 bits: row r of a ring is its r-th oldest
    held = total.clamp(max=C)
    r = torch.arange(C, device=DEV)
    row = (total[:, None] - held[:, None] + r) % C
    there = (r < held[:, None])[:, None, :, None]
    back = lambda q, x: (q.view(torch.uint8)[b, :, row].view(q.dtype).float() * x[b, :, row][..., None]).transpose(1, 2)  # noqa: E731
    s["k_rows"].copy_(torch.where(there, back(s["kq"], s["ks"]).to(s["k_rows"].dtype), s["k_rows"]))
    s["v_rows"].copy_(torch.where(there, back(s["vq"], s["vs"]).to(s["v_rows"].dtype), s["v_rows"]))
    return [s["k_rows"], s["v_rows"], s["ks"], s["vs"]]


def _quant_decode(s):
    c = s["case"]
    B, Hq, H, D, C = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["cap"]
    last = s["seqlens"].long()[:, None]
    q = _rotated(s["q"], last, s["rope"]).reshape(B, H, Hq // H, D)
    slot = torch.arange(C, device=DEV)
    pos = last - (last - slot) % C if c["ring"] else slot.expand(B, C)
    visible = (pos >= 0) & (pos <= last)
    if c["window"]:
        visible &= last - pos < c["window"]
    scores = torch.matmul(q, (s["kq"].float() * s["ks"][..., None]).transpose(-1, -2)) / math.sqrt(D)
    out = _attend(scores, s["vq"].float() * s["vs"][..., None], visible[:, None, None], s["q"].dtype)
    s["out"].copy_(out.reshape(B, Hq, 1, D))
    return [s["out"]]


def _logical(pool, table):
    """the rows of a paged cache in order: [B, H, rows, D]"""
    x = pool[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _tree(s):
    c = s["case"]
    B, Hq, H, D, N, C, page = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["nodes"], c["cap"], c["page"]
    parents = s["parents"].long()
    there = parents > -2
    up = torch.zeros((B, N, N + 2), dtype=torch.float64, device=DEV).scatter_(2, (parents % (N + 2))[..., None], 1.0)[..., :N]
    above = torch.linalg.matrix_power(up + torch.eye(N, dtype=torch.float64, device=DEV), N) > 0
    above &= there[..., None]
    depth = above.sum(-1) - 1
    past = s["seqlens"].long()[:, None] + 1 - N
    at = torch.where(there, past + depth, torch.zeros_like(depth))
    # the drafts' rows go behind the cache
    b, row = torch.arange(B, device=DEV)[:, None].expand(B, N), past + torch.arange(N, device=DEV)
    place = (lambda b, r: (s["table"].long()[b, r // page], r % page)) if page else (lambda b, r: (b, r))
    first, second = place(b[there], row[there])
    s["k"][first, :, second] = _rotated(s["new_k"], at, s["rope"]).to(s["k"].dtype).transpose(1, 2)[there]
    s["v"][first, :, second] = s["new_v"].transpose(1, 2)[there]
    k, v = (_logical(s["k"], s["table"]), _logical(s["v"], s["table"])) if page else (s["k"], s["v"])
    # each draft sees the cache and its own line
    r = torch.arange(C, device=DEV)
    draft = (r - past).clamp(0, N - 1)
    mine = torch.gather(above, 2, draft[:, None].expand(B, N, C)) & (r < past + N)[:, None] & (r >= past)[:, None]
    visible = ((r < past)[:, None] | mine) & there[..., None]
    if c["window"]:
        pos = torch.where(r < past, r, past + torch.gather(depth, 1, draft))
        visible &= at[..., None] - pos[:, None] < c["window"]
    q = _rotated(s["q"], at, s["rope"]).reshape(B, H, Hq // H * N, D)
    scores = torch.matmul(q, k.float().transpose(-1, -2)) / math.sqrt(D)
    visible = visible[:, None, None].expand(B, 1, Hq // H, N, C).reshape(B, 1, -1, C)
    # rows behind the last sequence are not read
    v = torch.where((r < past + N)[:, None, :, None], v.float(), torch.zeros((), device=DEV))
    s["out"].copy_(_attend(scores, v, visible, s["q"].dtype).reshape(B, Hq, N, D))
    # the accepted line's rows move to the front of the drafts'
    n = torch.arange(N, device=DEV)
    taken = n < s["accepted"][:, None]
    to, frm = place(b[taken], (past + n)[taken]), place(b[taken], (past + s["path"].long())[taken])
    s["k"][to[0], :, to[1]], s["v"][to[0], :, to[1]] = s["k"][frm[0], :, frm[1]], s["v"][frm[0], :, frm[1]]
    s["next"].copy_(past[:, 0] + s["accepted"] - 1)
    return [s["out"], s["k"], s["v"], s["next"]]


def _page_bounds(s):
    c = s["case"]
    page = c["page"]
    total = s["seqlens"].long()[:, None] + 1
    j = torch.arange(s["table"].shape[1], device=DEV)
    filled = s["table"].long()[((total - c["new"]) // page <= j) & (j < total // page)]
    k = s["k"][filled]
    hi, lo = k.amax(2).float(), k.amin(2).float()
    scale = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    scale = scale / torch.full_like(scale, 127.0)
    by = torch.where(scale == 0, torch.ones_like(scale), scale)[..., None]
    s["bounds"][filled] = torch.stack([torch.ceil(hi / by), torch.floor(lo / by)], 2).clamp(-127, 127).to(torch.int8)
    s["bscale"][filled] = scale
    return [s["bounds"].float() * s["bscale"][:, :, None, None], s["bscale"]]


def _sparse(s):
    c = s["case"]
    B, Hq, H, D, page, n = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["select"]
    last = s["seqlens"].long()[:, None]
    q = _rotated(s["q"], last, s["rope"]).reshape(B, H, Hq // H, D)
    # sums over a group's heads in 64 bits (a page's rank may hang on the last bit), rounded once
    side = torch.stack([q.double().clamp(min=0).sum(2), q.double().clamp(max=0).sum(2)], 2).float()
    by = side.abs().amax((-1, -2))
    by = by / torch.full_like(by, 127.0)
    code = (side / torch.where(by == 0, torch.ones_like(by), by)[..., None, None]).round()
    table = s["table"].long()
    m = table.shape[1]
    # whole numbers below 2^24: exact in 32 bits
    score = torch.matmul(s["bounds"][table].float().reshape(B, m, H, 1, 2 * D), code.reshape(B, 1, H, 2 * D, 1)).reshape(B, m, H)
    score = (s["bscale"][table] * score).transpose(1, 2)
    pages = last // page + 1
    j = torch.arange(m, device=DEV)
    always = (j < pages) & ((j < c["sink"]) | (j >= pages - c["recent"]))
    score = score.masked_fill(always[:, None], math.inf).masked_fill((j >= pages)[:, None], -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = torch.cat([order, order.new_full((B, H, max(0, n - m)), m)], -1)[..., :n]
    order = torch.where(torch.arange(n, device=DEV) < pages[:, None], order, m).sort(-1).values
    s["selected"].copy_(torch.where(order < m, order, -1))
    chosen = torch.where(order < m, order, 0)
    where, head = table[torch.arange(B, device=DEV)[:, None, None], chosen], torch.arange(H, device=DEV)[:, None]
    k, v = (s[x][where, head].reshape(B, H, n * page, D).float() for x in ("k", "v"))
    row = chosen[..., None] * page + torch.arange(page, device=DEV)
    visible = ((order < m)[..., None] & (row <= last[..., None, None])).reshape(B, H, 1, n * page)
    scores = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    s["out"].copy_(_attend(scores, v, visible, s["q"].dtype).reshape(B, Hq, 1, D))
    return [s["out"], s["selected"]]


# ---------------------------------------------------------------- work

def _seen(case):
    """rows of the cache that a call reads for one sequence and kv head, on average"""
    lo, hi = case["low"], case["high"]
    most = case["cap"] if "cap" in case else hi
    if case.get("window"):
        most = min(most, case["window"])
    # the mean of min(T, most) for T even over [lo, hi]
    if hi <= most:
        return (lo + hi) / 2
    if lo >= most:
        return most
    return ((most - lo + 1) * (lo + most) / 2 + (hi - most) * most) / (hi - lo + 1)


def work(case):
    c = case
    B, H, D = c["batch"], c["kv_heads"], c["dim"]
    if c["kind"] == "quant_write":
        S, past = c["new"], c["past"] / 2
        held = min(c["cap"], past + S)
        rows = B * H
        moved = rows * S * D * 2 * 2 + rows * S * 2 * (D + 4)           # new rows in, their codes out
        moved += rows * max(0, held - S) * 2 * (D + 4) + rows * held * D * 2 * 2  # the others' codes in, 16-bit rows out
        return {"bytes": moved, "flops": rows * D * (S * 2 * 4 + held * 2)}
    if c["kind"] == "quant_decode":
        n = B * H * _seen(c)
        return {"bytes": n * 2 * (D + 4) + 2 * B * c["q_heads"] * D * 2, "flops": 4 * D * B * c["q_heads"] * _seen(c)}
    if c["kind"] == "tree":
        N, n = c["nodes"], _seen(c)
        moved = B * H * (n + N) * D * 2 * 2 + 2 * B * c["q_heads"] * N * D * 2 + B * H * N * D * 2 * 2 * 2
        return {"bytes": moved, "flops": 4 * D * B * c["q_heads"] * N * (n + N / 2)}
    if c["kind"] == "page_bounds":
        pages = B * H * (c["new"] // c["page"])
        everything = 2 * D * 4 * B * H * -(-(c["past"] + c["new"]) // c["page"])
        return {"bytes": pages * (c["page"] * D * 2 + 2 * D + 4) + everything, "flops": pages * c["page"] * D * 2}
    pages = _seen(c) / c["page"]
    taken = min(c["select"], pages + 1) * c["page"]
    return {"bytes": B * H * (pages * (2 * D + 4) + taken * D * 2 * 2) + 2 * B * c["q_heads"] * D * 2,
            "flops": B * (H * pages * 4 * D + 4 * D * c["q_heads"] * taken)}


# ---------------------------------------------------------------- the definition in 64 bits

def _turn(x, positions, rope):
    """one batch row's x [H, S, D] at positions [S]"""
    c, n = rope[0].double()[positions], rope[1].double()[positions]
    h = x.shape[-1] // 2
    a, b = x.double()[..., :h], x.double()[..., h:]
    return torch.cat([a * c - b * n, a * n + b * c], -1)


def _softmax(q, k, v, see):
    """q [H, G, D], k and v [H, R, D], see [G, R] -> [H, G, D]; zeros where nothing is seen"""
    z = torch.einsum("hgd,hrd->hgr", q, k) / math.sqrt(q.shape[-1])
    z = torch.where(see, z, torch.full_like(z, -math.inf))
    w = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
    return torch.einsum("hgr,hrd->hgd", w, v)


def _coded(x, codes):
    """(codes, scales): scale in 32 bits, then the nearest code"""
    s = (x.abs().amax(-1) / TOP[codes]).float().double()
    y = x / torch.where(s == 0, torch.ones_like(s), s)[..., None]
    return (torch.round(y) if codes == "int8" else y.float().to(CODES[codes]).double()), s


def exact(case, seed):
    c, s = case, prepare(case, seed)
    B, H, D = c["batch"], c["kv_heads"], c["dim"]
    total = (s["seqlens"].long() + 1).tolist()
    if c["kind"] == "quant_write":
        C, S = c["cap"], c["new"]
        ks, vs = s["ks"].double(), s["vs"].double()
        outs = []
        for name, sc in (("k", ks), ("v", vs)):
            code, rows = s[name + "q"].float().double(), s[name + "_rows"].double()
            for b, T in enumerate(total):
                new, at = s["new_" + name][b], torch.arange(T - S, T, device=DEV)
                x = _turn(new, at, s["rope"]) if name == "k" else new.double()
                code[b][:, at % C], sc[b][:, at % C] = _coded(x, c["codes"])
                old = torch.arange(max(0, T - C), T, device=DEV) % C
                rows[b, :, :len(old)] = code[b][:, old] * sc[b][:, old][..., None]
            outs.append(rows)
        return outs + [ks, vs]
    if c["kind"] == "quant_decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for b, T in enumerate(total):
            n = min(T, c["cap"], c["window"] or T)
            at = torch.arange(T - n, T, device=DEV) % c["cap"]
            k, v = (s[x + "q"][b].float()[:, at].double() * s[x + "s"][b][:, at].double()[..., None] for x in ("k", "v"))
            q = _turn(s["q"][b], torch.tensor([T - 1], device=DEV), s["rope"]).reshape(H, -1, D)
            out[b] = _softmax(q, k, v, torch.ones((1, n), dtype=torch.bool, device=DEV)).reshape(-1, 1, D)
        return [out]
    if c["kind"] == "tree":
        N, page = c["nodes"], c["page"]
        if 4 * D * B * c["q_heads"] * N * c["cap"] > 1.5e12:
            return None
        k, v = s["k"].double(), s["v"].double()
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        parents, path, taken = s["parents"].tolist(), s["path"].tolist(), s["accepted"].tolist()
        for b, T in enumerate(total):
            P = T - N
            lines = []
            for i in range(N):
                p = parents[b][i]
                lines.append([] if p == -2 else ([] if p == -1 else lines[p]) + [i])
            there = [i for i in range(N) if lines[i]]
            r = torch.arange(T, device=DEV)
            first, second = (s["table"][b].long()[r // page], r % page) if page else (torch.full_like(r, b), r)
            kb, vb = k[first, :, second].transpose(0, 1).clone(), v[first, :, second].transpose(0, 1).clone()
            pos = torch.tensor([P + len(x) - 1 if x else 0 for x in lines], device=DEV)
            new = _turn(s["new_k"][b], pos, s["rope"])
            kb[:, [P + i for i in there]], vb[:, [P + i for i in there]] = new[:, there], s["new_v"][b].double()[:, there]
            k[first, :, second], v[first, :, second] = kb.transpose(0, 1), vb.transpose(0, 1)
            see = torch.zeros((N, T), dtype=torch.bool)
            for i in there:
                see[i, :P] = True
                see[i, [P + x for x in lines[i]]] = True
            see = see.to(DEV)
            if c["window"]:
                see &= pos[:, None] - torch.cat([r[:P], pos])[None] < c["window"]
            # what an absent draft's row holds is not looked at: it may be anything
            q = _turn(s["q"][b], pos, s["rope"]).reshape(H, -1, D)
            out[b] = _softmax(q, kb, vb, see.repeat(c["q_heads"] // H, 1)).reshape(-1, N, D)
            n = taken[b]
            k[first[P:P + n], :, second[P:P + n]] = kb[:, [P + x for x in path[b][:n]]].transpose(0, 1)
            v[first[P:P + n], :, second[P:P + n]] = vb[:, [P + x for x in path[b][:n]]].transpose(0, 1)
        return [out, k, v, torch.tensor([T - N + n - 1 for T, n in zip(total, taken)], dtype=torch.int32, device=DEV)]
    if c["kind"] == "page_bounds":
        value = s["bounds"].double() * s["bscale"].double()[:, :, None, None]
        scale = s["bscale"].double()
        for b, T in enumerate(total):
            for j in range((T - c["new"]) // c["page"], T // c["page"]):
                p = int(s["table"][b, j])
                x = s["k"][p].double()
                sc = (x.abs().amax((1, 2)) / 127).float().double()
                by = torch.where(sc == 0, torch.ones_like(sc), sc)[:, None]
                value[p, :, 0] = torch.ceil((x.amax(1) / by).float().double()).clamp(-127, 127) * sc[:, None]
                value[p, :, 1] = torch.floor((x.amin(1) / by).float().double()).clamp(-127, 127) * sc[:, None]
                scale[p] = sc
        return [value, scale]
    page, n = c["page"], c["select"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    picked = torch.full_like(s["selected"], -1)
    for b, T in enumerate(total):
        q = _turn(s["q"][b], torch.tensor([T - 1], device=DEV), s["rope"]).reshape(H, -1, D)
        m = -(-T // page)
        phys = s["table"][b, :m].long()
        # the ranks go by the query as it is rotated in 32 bits, each product and sum rounded
        cos, sin = s["rope"][0][T - 1], s["rope"][1][T - 1]
        a, z = s["q"][b, :, 0].float().chunk(2, -1)
        turned = torch.cat([a * cos - z * sin, z * cos + a * sin], -1).double().reshape(H, -1, D)
        plus, minus = turned.clamp(min=0).sum(1).float(), turned.clamp(max=0).sum(1).float()
        by = (torch.maximum(plus.amax(-1), -minus.amin(-1)).double() / 127).float().double()
        by = torch.where(by == 0, torch.ones_like(by), by)[:, None]
        p, q8 = (torch.round((x.double() / by).float().double()) for x in (plus, minus))
        bounds = s["bounds"][phys].double()
        score = torch.einsum("mhd,hd->hm", bounds[:, :, 0], p) + torch.einsum("mhd,hd->hm", bounds[:, :, 1], q8)
        score = (score * s["bscale"][phys].double().T).float().cpu().tolist()
        forced = set(range(min(c["sink"], m))) | set(range(max(0, m - c["recent"]), m))
        for h in range(H):
            rest = sorted((j for j in range(m) if j not in forced), key=lambda j: (-score[h][j], j))
            mine = sorted(forced | set(rest[:max(0, n - len(forced))]))
            picked[b, h, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            at = torch.cat([torch.arange(j * page, min(T, (j + 1) * page), device=DEV) for j in mine])
            k, v = (s[x][s["table"][b].long()[at // page], h, at % page].double()[None] for x in ("k", "v"))
            see = torch.ones((1, len(at)), dtype=torch.bool, device=DEV)
            out[b].reshape(H, -1, D)[h] = _softmax(q[h:h + 1], k, v, see)[0]
    return [out, picked]
