"""Attention over selected pages: the pages' bounds (kvc_page_bounds) and the pages taken
(kvc_gqa_decode_sparse) equal bit for bit to the header's formulas, the attention over them within
the bound that attention() of _ops_reference.py derives (query and weights with the digits of two
numbers of the cache's type)."""
import math

import pytest
import torch

import _ops_reference as R

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make(g, B, H, D, page, max_pages, dtype, spare=3):
    n = B * max_pages + spare
    table = torch.randperm(n, generator=g)[:B * max_pages].to(torch.int32).reshape(B, max_pages)
    k = (torch.randn((n, H, page, D), generator=g) + 0.7 * torch.randn((n, H, 1, D), generator=g)).to(dtype)
    v = torch.randn((n, H, page, D), generator=g).to(dtype)
    return table, k, v


def bounds_of(k):
    """one page's bounds, per head: codes [H, 2, D] and scale [H]"""
    x = k.float()
    hi, lo = x.amax(1), x.amin(1)
    top = x.abs().amax((1, 2))
    s = top / torch.full_like(top, 127.0)
    by = torch.where(s == 0, torch.ones_like(s), s)[:, None]
    code = torch.stack([torch.ceil(hi / by), torch.floor(lo / by)], 1).clamp(-127, 127)
    bad = ~torch.isfinite(x).all(-1).all(-1)
    code = torch.where((bad | (s == 0))[:, None, None], torch.zeros_like(code), code)
    return code.to(torch.int8), torch.where(bad, torch.full_like(s, math.inf), s)


def all_bounds(k):
    made = [bounds_of(x) for x in k]
    return torch.stack([c for c, _ in made]), torch.stack([s for _, s in made])


def choose(q, bounds, scale, pages, n, sink, recent):
    """q [G, D] float32 rotated; bounds [pages, 2, D], scale [pages] of one head"""
    u, w = (q.double().clamp(min=0).sum(0).float(), q.double().clamp(max=0).sum(0).float())
    top = torch.maximum(u.max(), -w.min())
    sq = top / torch.full_like(top, 127.0)
    code = torch.zeros(2, q.shape[1], dtype=torch.int64) if sq == 0 else torch.round(torch.stack([u, w]) / sq).long()
    score = (scale * (bounds.long() * code).sum((1, 2)).float()).tolist()
    score = [math.inf if math.isinf(s) else x for x, s in zip(score, scale.tolist())]
    forced = set(range(min(sink, pages))) | set(range(max(0, pages - recent), pages))
    rest = sorted((j for j in range(pages) if j not in forced), key=lambda j: (-score[j], j))
    return sorted(forced | set(rest[:max(0, min(n, pages) - len(forced))]))


def lengths(K, totals, S, C, st=None):
    sk = torch.tensor([t - 1 for t in totals], dtype=torch.int32, device="cuda")
    return K.kvc_seq_lengths(sk, S, C, K.KVC_CONTIGUOUS, status=st)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 64, 100, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_bounds_of_the_pages_that_a_step_filled(K, D, page, dtype):
    B, H, m, S = 4, 3, 5, page + page // 2 + 1
    g = gen(D + page)
    table, k, v = make(g, B, H, D, page, m, dtype)
    k[table[0, 1], 1] = 0
    k[table[0, 0], 0, page // 2, 3] = math.nan
    k[table[3, 0], 2, 0, D - 1] = -math.inf
    k[table[1, m - 1], 0] *= 1e-4
    totals = [2 * page, m * page, S, 0]  # from a page's start on; to the table's end; inside a page; refused
    totals[3] = S - 1
    have = [torch.randint(-127, 128, (len(k), H, 2, D), generator=g).to(torch.int8), torch.rand((len(k), H), generator=g)]
    got = [x.cuda() for x in have]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lengths(K, totals, S, m * page, st)
    K.kvc_page_bounds(*got, k.cuda(), table.cuda(), L, S, status=st)
    for b, T in enumerate(totals[:3]):
        for j in range((T - S) // page, T // page):
            have[0][table[b, j]], have[1][table[b, j]] = bounds_of(k[table[b, j]])
    assert torch.equal(got[0].cpu(), have[0]) and torch.equal(got[1].cpu(), have[1])
    assert st.item() == K.KVC_DEV_SEQLEN_RANGE


def run(K, dtype, B, H, G, D, page, m, n, sink, recent, totals, rope=True, seed=0, edit=None, scale=0.0):
    g = gen(seed + D + page)
    table, k, v = make(g, B, H, D, page, m, dtype)
    q = torch.randn((B, H * G, 1, D), generator=g).to(dtype)
    if edit:
        edit(q, k, v, table)
    bounds, bscale = all_bounds(k)
    tables = R.rope_tables(m * page, D) if rope else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lengths(K, totals, 1, m * page, st)
    out = torch.full_like(q, 7.0, device="cuda")
    selected = torch.full((B, H, n), -7, dtype=torch.int32, device="cuda")
    d = [x.cuda() for x in (q, k, v, bounds, bscale, table)]
    K.kvc_gqa_decode_sparse(out, *d, L, selected, sink, recent, scale=scale, rope=tables and [x.cuda() for x in tables], status=st)
    step = R.half_step(dtype)  # (query and weights are sums of two numbers of the type)
    for b, T in enumerate(totals):
        if T < 1 or T > m * page:
            assert (out[b] == 7).all() and (selected[b] == -7).all()
            continue
        pages = -(-T // page)
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            at = torch.tensor([T - 1])
            q32 = R.rotate32(q[b, heads], at, tables)[:, 0]
            phys = table[b, :pages].long()
            mine = choose(q32, bounds[phys, h], bscale[phys, h], pages, n, sink, recent)
            assert selected[b, h].tolist() == mine + [-1] * (n - len(mine)), f"row {b} head {h}"
            rows = torch.cat([torch.arange(j * page, min(T, (j + 1) * page)) for j in mine])
            kk, vv = (x[table[b, rows // page].long(), h, rows % page].double() for x in (k, v))
            want, bound = R.attention(R.rotate64(q[b, heads], at, tables)[:, 0], kk, vv, torch.ones((G, len(rows)), dtype=torch.bool),
                                      scale or D ** -0.5, step ** 2 if rope else 0.0, step ** 2, dtype,
                                      half_weights=torch.ones(len(rows)) if dtype == F16 else None)
            R.assert_within(out[b, heads, 0], want, bound, f"row {b} head {h}")
    return out, selected, st.item()


@pytest.mark.parametrize("dtype,D,G", [(BF16, 64, 1), (F16, 64, 16), (BF16, 128, 5), (F16, 128, 8), (BF16, 256, 16), (F16, 256, 2)])
@pytest.mark.parametrize("page,n,sink,recent", [(64, 1, 0, 1), (64, 9, 1, 2), (128, 4, 0, 3), (64, 40, 3, 1), (192, 6, 2, 2)])
def test_selection_and_attention(K, dtype, D, G, page, n, sink, recent):
    m = 23
    totals = [m * page, 0, 1, 11 * page + 1, 12 * page, 9 * page - 1, n * page, m * page + 1]
    _, _, st = run(K, dtype, 8, 2, G, D, page, m, n, sink, recent, totals)
    assert st == K.KVC_DEV_SEQLEN_RANGE | K.KVC_DEV_CAPACITY


def test_many_pages(K):
    """more pages than the block has threads, and a choice that is most of them"""
    run(K, BF16, 2, 1, 4, 64, 64, 1500, 37, 1, 1, [1500 * 64, 1031 * 64 + 5])
    run(K, F16, 1, 2, 2, 64, 64, 700, 600, 0, 1, [700 * 64 - 3])


def test_ties_go_to_the_lower_page(K):
    def alike(q, k, v, table):
        k[:] = k[0, :, :1]
    _, sel, _ = run(K, BF16, 1, 2, 4, 128, 64, 30, 8, 0, 2, [30 * 64], edit=alike)
    assert sel[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 28, 29]

    def no_query(q, k, v, table):
        q.zero_()
    _, sel, _ = run(K, BF16, 1, 2, 4, 128, 64, 600, 5, 1, 1, [600 * 64], edit=no_query, rope=False)
    assert sel[0, 1].tolist() == [0, 1, 2, 3, 599]


def test_a_page_that_is_not_finite_is_taken(K):
    def edit(q, k, v, table):
        k[table[0, 13], 1, 5, 7] = math.inf
        k[table[0, 17], 0, 9, 1] = math.nan
    g = gen(1)
    table, k, v = make(g, 1, 2, 64, 64, 20, BF16)
    edit(None, k, v, table)
    bounds, bscale = all_bounds(k)
    sel = torch.zeros((1, 2, 3), dtype=torch.int32, device="cuda")
    q = torch.randn((1, 4, 1, 64), generator=g).to(BF16).cuda()
    out = torch.zeros_like(q)
    K.kvc_gqa_decode_sparse(out, q, *[x.cuda() for x in (k, v, bounds, bscale, table)], lengths(K, [20 * 64], 1, 20 * 64), sel, 0, 1)
    assert 17 in sel[0, 0].tolist() and 13 in sel[0, 1].tolist()
    assert torch.isnan(out[0, :2].float()).all()


def test_every_page_taken(K):
    for dtype, D, G in ((BF16, 128, 4), (F16, 256, 16), (F16, 64, 12)):
        _, sel, _ = run(K, dtype, 5, 2, G, D, 64, 33, 33, 0, 1, [33 * 64, 1, 700, 64, 65])
        assert sel[2, 1].tolist() == list(range(11)) + [-1] * 22


@pytest.mark.parametrize("B,H,D", [(1, 1, 128), (1, 3, 64), (40, 8, 64), (70, 2, 256), (3, 1, 128)])
def test_shares_of_few_and_of_many_rows(K, B, H, D):
    """rows that many CTAs join, and CTAs with many rows; again into the same workspace"""
    g = gen(B)
    m, n = 60 if B < 10 else 7, 50 if B < 10 else 4
    totals = [int(torch.randint(0, m * 64 + 1, (), generator=g)) for _ in range(B)]
    totals[0] = m * 64
    a = run(K, F16, B, H, 3, D, 64, m, n, 1, 1, totals)
    b = run(K, F16, B, H, 3, D, 64, m, n, 1, 1, totals)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_past_the_newest_token_hold_anything(K):
    def edit(q, k, v, table):
        for x in (k, v):
            x[table[0, 12], :, 10:] = math.nan
            x[table[1, 3], :, 63] = math.inf
    run(K, BF16, 2, 2, 4, 128, 64, 13, 4, 0, 1, [12 * 64 + 10, 4 * 64 - 1], edit=edit)


def test_bad_pages(K):
    B, H, D, page, m = 2, 2, 64, 64, 9
    g = gen(2)
    table, k, v = make(g, B, H, D, page, m, BF16)
    bounds, bscale = all_bounds(k)
    table[0, 4] = len(k)
    table[0, 7] = -1
    d = [x.cuda() for x in (k, v, bounds, bscale, table)]
    q = torch.randn((B, 4, 1, D), generator=g).to(BF16).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L = lengths(K, [m * page, m * page], 1, m * page)
    sel = torch.zeros((B, H, 5), dtype=torch.int32, device="cuda")
    out = K.kvc_gqa_decode_sparse(torch.zeros_like(q), q, *d, L, sel, status=st)
    assert st.item() == K.KVC_DEV_INDEX_OOB and torch.isfinite(out[1]).all()
    # the step of the whole prompt: the good pages' bounds are written, the bad ones skipped
    st.zero_()
    got = [torch.zeros_like(d[2]), torch.zeros_like(d[3])]
    L = lengths(K, [m * page, m * page], m * page, m * page)
    K.kvc_page_bounds(*got, d[0], d[4], L, m * page, status=st)
    assert st.item() == K.KVC_DEV_INDEX_OOB
    named = torch.zeros(len(k), dtype=torch.bool)
    for b in range(B):
        for j in range(m):
            if 0 <= table[b, j] < len(k):
                named[table[b, j]] = True
    assert torch.equal(got[0][named].cpu(), bounds[named]) and not got[1][~named].any()


def test_rope_range(K):
    g = gen(2)
    table, k, v = make(g, 2, 2, 64, 64, 4, BF16)
    bounds, bscale = all_bounds(k)
    q = torch.randn((2, 4, 1, 64), generator=g).to(BF16).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sel = torch.full((2, 2, 2), -7, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    K.kvc_gqa_decode_sparse(out, q, *[x.cuda() for x in (k, v, bounds, bscale, table)], lengths(K, [201, 200], 1, 256), sel,
                            rope=[x.cuda() for x in R.rope_tables(200, 64)], status=st)
    assert st.item() == K.KVC_DEV_ROPE_RANGE and (out[0] == 7).all() and (sel[0] == -7).all() and (sel[1] >= 0).all()


def test_prompt_then_steps(K):
    """As a server runs it: a prompt appended to pages with their bounds, then 70 one-token steps, captured in a
    graph and replayed on another stream; the bounds of every full page are those of its rows."""
    B, H, G, D, page, m, P, n = 2, 2, 4, 128, 64, 12, 500, 5
    g = gen(4)
    table, k, v = make(g, B, H, D, page, m, BF16)
    rope = [x.cuda() for x in R.rope_tables(m * page, D)]
    bounds = torch.zeros((len(k), H, 2, D), dtype=torch.int8, device="cuda")
    bscale = torch.zeros((len(k), H), device="cuda")
    k, v, table = k.cuda(), v.cuda(), table.cuda()
    nk, nv = (torch.randn((B, H, P + 70, D), generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn((B, H * G, 70, D), generator=g).to(BF16).cuda()
    sk = torch.tensor([P - 1, P - 1], dtype=torch.int32, device="cuda")

    def append(i, S):
        L = K.kvc_seq_lengths(sk, S, m * page, K.KVC_CONTIGUOUS)
        K.kvc_paged_append(k, v, nk[:, :, i:i + S].contiguous(), nv[:, :, i:i + S].contiguous(), table, L, rope=rope)
        K.kvc_page_bounds(bounds, bscale, k, table, L, S)
        return L

    def steps():
        outs, sels = [], []
        append(0, P)
        for i in range(70):
            sk.add_(1)
            L = append(P + i, 1)
            out = torch.zeros((B, H * G, 1, D), dtype=BF16, device="cuda")
            sel = torch.zeros((B, H, n), dtype=torch.int32, device="cuda")
            K.kvc_gqa_decode_sparse(out, q[:, :, i:i + 1].contiguous(), k, v, bounds, bscale, table, L, sel, rope=rope)
            outs.append(out)
            sels.append(sel)
        return torch.cat(outs, 2), torch.stack(sels)

    want = steps()
    full, scale = all_bounds(k.cpu())
    for b in range(B):
        for j in range((P + 70) // page):
            i = int(table[b, j])
            assert torch.equal(bounds[i].cpu(), full[i]) and torch.equal(bscale[i].cpu(), scale[i])
    sk.fill_(P - 1)
    bounds.zero_()
    bscale.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps()
    sk.fill_(P - 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_smallest_cache(K, D):
    _, sel, _ = run(K, F16, 1, 1, 1, D, 64, 1, 1, 0, 1, [1])
    assert sel.tolist() == [[[0]]]
    run(K, BF16, 2, 1, 2, D, 64, 1, 3, 1, 1, [64, 63])
