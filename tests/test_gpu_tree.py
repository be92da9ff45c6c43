"""A tree of drafted tokens over a cache: masks, depths, appended and kept rows equal bit for bit to
the header's statement, the attention (kvc_gqa_tree) within the bound that attention() of
_ops_reference.py derives (of query and weights one rounded to the cache's type, the other a sum of
two numbers of it)."""
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


def a_tree(g, N, absent=0.1):
    p = []
    for i in range(N):
        u = float(torch.rand((), generator=g))
        p.append(-2 if u < absent else int(torch.randint(-1, i, (), generator=g)) if i else -1)
    return p


def lines_of(parents):
    """for each node its line from the root on, [] for an absent one"""
    lines = []
    for i, p in enumerate(parents):
        ok = -1 <= p < i and (p < 0 or lines[p])
        lines.append((lines[p] if p >= 0 else []) + [i] if ok else [])
    return lines


def words(rows, N):
    w = torch.zeros((len(rows), (N + 31) // 32), dtype=torch.int64)
    for i, row in enumerate(rows):
        for j in row:
            w[i, j // 32] |= 1 << (j % 32)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 100, 256])
def test_mask(K, N):
    g = gen(N)
    trees = [[i - 1 for i in range(N)], [-1] * N, [-2] * N] + [a_tree(g, N) for _ in range(5)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mask, depth = K.kvc_tree_mask(torch.tensor(trees, dtype=torch.int32, device="cuda"), status=st)
    assert st.item() == 0
    bad = [list(t) for t in trees]
    bad[3][N - 1], bad[4][0] = N - 1, -3
    mask2, depth2 = K.kvc_tree_mask(torch.tensor(bad, dtype=torch.int32, device="cuda"), status=st)
    assert st.item() == K.KVC_DEV_INDEX_OOB
    for some, m, d in ((trees, mask, depth), (bad, mask2, depth2)):
        for b, t in enumerate(some):
            lines = lines_of(t)
            assert d[b].tolist() == [len(x) - 1 for x in lines]
            assert torch.equal(m[b].cpu(), words(lines, N))


class Case:
    """A cache (contiguous or paged) with trees over it, on the CPU and on the GPU."""

    def __init__(self, K, g, B, H, G, D, C, N, totals, page=0, dtype=BF16, rope=True, trees=None):
        self.K, self.B, self.H, self.G, self.D, self.C, self.N, self.page, self.dtype = K, B, H, G, D, C, N, page, dtype
        self.past = totals
        shape, self.table = (B, H, C, D), None
        if page:
            n = B * (C // page) + 2
            self.table = torch.randperm(n, generator=g)[:n - 2].to(torch.int32).reshape(B, C // page)
            shape = (n, H, page, D)
        self.k, self.v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
        self.new_k, self.new_v = (torch.randn((B, H, N, D), generator=g).to(dtype) for _ in range(2))
        self.q = torch.randn((B, H * G, N, D), generator=g).to(dtype)
        self.trees = trees or [a_tree(g, N) for _ in range(B)]
        self.lines = [lines_of(t) for t in self.trees]
        self.rope = R.rope_tables(C, D) if rope else None
        self.gpu = {x: getattr(self, x).cuda() for x in ("k", "v", "new_k", "new_v", "q")}
        self.gpu_table = None if self.table is None else self.table.cuda()
        self.gpu_rope = self.rope and [x.cuda() for x in self.rope]
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sk = torch.tensor([p + N - 1 for p in totals], dtype=torch.int32, device="cuda")
        self.L = K.kvc_seq_lengths(sk, N, C, K.KVC_CONTIGUOUS, status=self.st)
        self.mask, self.depth = K.kvc_tree_mask(torch.tensor(self.trees, dtype=torch.int32, device="cuda"))

    def at(self, b, r):
        """index of rows r of batch row b: [first][:, head][second]"""
        r = torch.as_tensor(r, dtype=torch.long)
        return (self.table[b, r // self.page].long(), r % self.page) if self.page else (torch.full_like(r, b), r)

    def good(self):
        return [b for b, p in enumerate(self.past) if p >= 0 and p + self.N <= self.C]

    def append(self):
        self.K.kvc_tree_append(self.gpu["k"], self.gpu["v"], self.gpu["new_k"], self.gpu["new_v"], self.depth, self.L,
                               block_table=self.gpu_table, rope=self.gpu_rope, status=self.st)
        for b in self.good():
            P = self.past[b]
            for i, line in enumerate(self.lines[b]):
                if line:
                    x, y = self.at(b, [P + i])
                    pos = torch.tensor([P + len(line) - 1])
                    self.k[x, :, y] = R.rotate32(self.new_k[b, :, i:i + 1], pos, self.rope)[:, 0].to(self.dtype)
                    self.v[x, :, y] = self.new_v[b, :, i]
        assert torch.equal(self.gpu["k"].cpu(), self.k) and torch.equal(self.gpu["v"].cpu(), self.v)

    def attend(self, window=0, scale=0.0, mask=None, depth=None, sees=None, pos=None, workspace="auto", rows=None):
        out = torch.full_like(self.gpu["q"], 7.0)
        self.K.kvc_gqa_tree(out, self.gpu["q"], self.gpu["k"], self.gpu["v"], self.mask if mask is None else mask,
                            self.depth if depth is None else depth, self.L, block_table=self.gpu_table,
                            local_window_size=window, scale=scale, rope=self.gpu_rope, status=self.st, workspace=workspace)
        got, N, G = out.cpu(), self.N, self.G
        for b in range(self.B):
            if b not in self.good():
                assert (got[b] == 7).all()
                continue
            P = self.past[b]
            lines = self.lines[b] if sees is None else sees[b]
            d = torch.tensor([len(x) - 1 for x in lines]) if pos is None else pos[b]
            there = d >= 0
            see = torch.zeros((N, P + N), dtype=torch.bool)
            for i in range(N):
                if there[i]:
                    see[i, :P] = True
                    see[i, [P + j for j in lines[i] if there[j]]] = True
            at = P + d.clamp(min=0)
            if window > 0:
                see &= at[:, None] - torch.cat([torch.arange(P), at])[None] < window
            x, y = self.at(b, torch.arange(P + N))
            # the query (head_dim <= 128) or the weights (256) are sums of two numbers of the type
            step = R.half_step(self.dtype)
            q_step, w_step = (step ** 2, step) if self.D <= 128 else (step, step ** 2)
            for h in range(self.H) if rows is None else rows:
                kk, vv = (c[x, h, y].double() for c in (self.k, self.v))
                heads = slice(h * G, (h + 1) * G)
                qq = R.rotate64(self.q[b, heads], at, self.rope).reshape(G * N, self.D)
                want, bound = R.attention(qq, kk, vv, see.repeat(G, 1), scale or self.D ** -0.5, q_step if self.rope else 0.0, w_step,
                                          self.dtype, half_weights=torch.ones(P + N) if self.dtype == F16 else None)
                R.assert_within(got[b, heads].reshape(G * N, self.D), want, bound, f"row {b} head {h}")
                assert not got[b, heads][:, ~there].any()
        return out

    def commit(self, paths, counts, seqlens):
        B = self.B
        width = max(1, max(len(p) for p in paths))
        path = torch.tensor([p + [-5] * (width - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        self.K.kvc_tree_commit(self.gpu["k"], self.gpu["v"], path, torch.tensor(counts, dtype=torch.int32, device="cuda"), self.L,
                               seqlens, self.N, block_table=self.gpu_table, status=self.st)
        return B


@pytest.mark.parametrize("dtype,D,G", [(BF16, 64, 1), (F16, 64, 8), (BF16, 128, 4), (F16, 128, 7), (BF16, 256, 2), (F16, 256, 16)])
@pytest.mark.parametrize("N,C,page,window", [(1, 300, 0, 0), (8, 300, 0, 0), (33, 700, 0, 40), (64, 640, 64, 0), (61, 576, 192, 100),
                                             (5, 640, 128, 3), (130, 400, 0, 0)])
def test_append_and_attention(K, dtype, D, G, N, C, page, window):
    past = [0, C - N, 1, C // 2 + 3, C - N + 1, 127, 128 - min(N, 20)]
    c = Case(K, gen(D + N + G), 7, 2, G, D, C, N, past, page, dtype)
    assert c.st.item() == K.KVC_DEV_CAPACITY
    c.append()
    c.attend(window)
    assert c.st.item() == K.KVC_DEV_CAPACITY


def test_the_largest_tree(K):
    c = Case(K, gen(1), 2, 1, 16, 128, 1500, 256, [1244, 700])
    c.append()
    c.attend()


@pytest.mark.parametrize("B,H,page", [(1, 1, 0), (40, 5, 0), (3, 8, 64)])
def test_shares(K, B, H, page):
    """One row over all of the GPU; more rows than CTAs; shares that end inside rows of odd lengths."""
    past = [9000] if B == 1 else [(37 * b * b) % 900 for b in range(B)]
    C = -(-(max(past) + 6) // 64) * 64
    c = Case(K, gen(B), B, H, 4, 128, C, 6, past, page)
    c.append()
    c.attend(rows=range(0, H, 2))


@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("D,dtype,page", [(64, F16, 0), (64, BF16, 64), (128, F16, 192), (128, BF16, 0), (256, F16, 64), (256, BF16, 0)])
def test_many_tiles_of_a_row(K, D, dtype, page, rope):
    """rows of a few to dozens of tiles, several of them to a CTA"""
    c = Case(K, gen(D), 6, 8, 4, D, 3840, 40, [3800, 2011, 0, 1279, 600, 3583], page, dtype, rope=rope)
    c.append()
    c.attend(rows=[0, 3, 7])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("C,N,past", [(1, 1, [0, 1]), (3, 2, [1, 0]), (40, 7, [33, 5]), (129, 1, [128, 127])])
def test_the_smallest_caches(K, D, C, N, past):
    c = Case(K, gen(C), 2, 1, 2, D, C, N, past, 0, F16)
    c.append()
    c.attend()
    c.attend(2)


def test_without_rope_and_with_a_scale(K):
    for scale in (0.3, -0.05):
        c = Case(K, gen(3), 2, 2, 3, 64, 300, 20, [250, 31], dtype=F16, rope=False)
        c.append()
        c.attend(scale=scale)


def test_masks_of_the_callers_own(K):
    """Nodes that do not see themselves, or nothing at all (an empty cache or a window that leaves nothing), depths that are not
    those of a tree, nodes that are absent."""
    B, H, N = 3, 2, 40
    g = gen(11)
    c = Case(K, g, B, H, 4, 128, 400, N, [0, 200, 300], trees=[[-1] * N] * 3)
    sees = [[[j for j in range(N) if float(torch.rand((), generator=g)) < 0.3] if i % 5 else [] for i in range(N)] for _ in range(B)]
    pos = torch.randint(0, N, (B, N), generator=g)
    pos[:, 7] = -1
    mask = torch.stack([words(s, N) for s in sees]).cuda()
    c.append()
    for window in (0, 1, 30):
        out = c.attend(window, mask=mask, depth=pos.to(torch.int32).cuda(), sees=sees, pos=pos)
        assert not out[0, :, [0, 5, 10]].any()
    assert c.st.item() == 0
    deep = pos.clone()
    deep[1, 3] = N
    out = c.K.kvc_gqa_tree(torch.full_like(c.gpu["q"], 7.0), c.gpu["q"], c.gpu["k"], c.gpu["v"], mask, deep.to(torch.int32).cuda(), c.L,
                           rope=c.gpu_rope, status=c.st)
    assert c.st.item() == K.KVC_DEV_INDEX_OOB and not out[1, :, 3].any()


def test_what_no_node_sees_may_be_anything(K):
    """NaN behind the drafts, in absent drafts' rows and below the window: the outputs stay what they were."""
    N = 12
    trees = [[-1, 0, -2, 1, -2] + [3] * 7, [-1] * 12]
    for page in (0, 64):
        c = Case(K, gen(5), 2, 2, 4, 128, 640, N, [300, 77], page, trees=trees)
        c.append()
        want = c.attend(150)
        for b, P in enumerate(c.past):
            for rows in (torch.arange(P + N, 640), torch.arange(0, max(0, P + 1 - 150 - N)),
                         torch.tensor([P + i for i in range(N) if not c.lines[b][i]], dtype=torch.long)):
                x, y = c.at(b, rows)
                for n in ("k", "v"):
                    c.gpu[n][x.cuda(), :, y.cuda()] = float("nan")
        if page:
            free = torch.ones(len(c.k), dtype=torch.bool)
            free[c.table.long().reshape(-1)] = False
            c.gpu["k"][free.cuda()] = float("nan")
            c.gpu["v"][free.cuda()] = float("nan")
        out = torch.full_like(want, 7.0)
        K.kvc_gqa_tree(out, c.gpu["q"], c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, block_table=c.gpu_table, local_window_size=150,
                       rope=c.gpu_rope)
        assert torch.equal(out, want)


@pytest.mark.parametrize("page,dtype,D", [(0, BF16, 128), (64, F16, 64), (64, BF16, 128), (192, BF16, 256)])
def test_what_only_some_nodes_see(K, page, dtype, D):
    """NaN and infinities in the K and V of drafts, and of cache rows that the window leaves to the first nodes only: NaN for the
    nodes that see them, the others' results as they were."""
    N = 20
    trees = [[-1] + [i - 1 - (i % 3 == 0) for i in range(1, N)], [-1] * 5 + [0, 1, 2, 3, 4] * 3]
    c = Case(K, gen(D), 2, 2, 5, D, 576, N, [250, 126], page, dtype, trees=trees)
    c.append()
    window = 40
    want = c.attend(window).cpu()
    for kind, draft, value in (("v", 4, float("inf")), ("k", 7, float("nan")), ("v", 11, float("nan")), ("v", None, float("nan"))):
        kept = c.gpu[kind].clone()
        for b, P in enumerate(c.past):
            x, y = c.at(b, [P - window + 4 if draft is None else P + draft])
            c.gpu[kind][x.cuda(), :, y.cuda()] = value
        out = torch.full_like(c.gpu["q"], 7.0)
        K.kvc_gqa_tree(out, c.gpu["q"], c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, block_table=c.gpu_table,
                       local_window_size=window, rope=c.gpu_rope)
        out = out.cpu()
        for b in range(2):
            for i, line in enumerate(c.lines[b]):
                # a row at distance W - 4 from P is seen up to depth 3
                sees = len(line) - 1 <= 3 if draft is None else draft in line
                if sees:
                    assert torch.isnan(out[b, :, i]).all(), (kind, draft, b, i)
                else:
                    assert torch.equal(out[b, :, i], want[b, :, i]), (kind, draft, b, i)
        c.gpu[kind].copy_(kept)


@pytest.mark.parametrize("page,dtype,D", [(0, BF16, 128), (64, F16, 64), (192, BF16, 256)])
def test_commit(K, page, dtype, D):
    N, C = 70, 576
    past = [0, 130, C - N, 250, 60, 300, 20, C - N + 1]
    trees = [[-1] * N] * 8
    c = Case(K, gen(D), 8, 2, 1, D, C, N, past, page, dtype, trees=trees)
    c.append()
    paths = [list(range(N)), [0, 3, 4, 9, 30, 69], [5], [], list(range(1, N)), [0, 2, 2], [0, 70], [0]]
    counts = [N, 6, 1, 0, N - 1, 3, 2, 1]
    seqlens = torch.full((8,), -77, dtype=torch.int32, device="cuda")
    c.st.zero_()
    c.commit(paths, counts, seqlens)
    assert c.st.item() == K.KVC_DEV_INDEX_OOB
    assert seqlens.tolist() == [p + n - 1 for p, n in zip(past[:5], counts)] + [-77] * 3
    for b in range(5):
        x, y = c.at(b, [past[b] + j for j in range(counts[b])])
        u, w = c.at(b, [past[b] + j for j in paths[b]])
        c.k[x, :, y], c.v[x, :, y] = c.k[u, :, w].clone(), c.v[u, :, w].clone()
    assert torch.equal(c.gpu["k"].cpu(), c.k) and torch.equal(c.gpu["v"].cpu(), c.v)
    # counts that do not fit, a path that goes below its place
    for path, n in (([0, 1], 3), ([0, 1], -1), ([1, 0], 2)):
        c.st.zero_()
        c.commit([path] * 8, [n] * 8, seqlens)
        assert c.st.item() == K.KVC_DEV_INDEX_OOB
    assert torch.equal(c.gpu["k"].cpu(), c.k) and seqlens[0].item() == past[0] + N - 1


def test_bad_pages(K):
    N = 10
    c = Case(K, gen(2), 2, 2, 4, 64, 640, N, [300, 300], 64)
    c.table[0, 4] = -1          # a page of the new rows
    c.gpu_table.copy_(c.table)
    before = c.gpu["k"].clone()
    K.kvc_tree_append(c.gpu["k"], c.gpu["v"], c.gpu["new_k"], c.gpu["new_v"], c.depth, c.L, block_table=c.gpu_table, status=c.st)
    assert c.st.item() == K.KVC_DEV_INDEX_OOB
    changed = (c.gpu["k"] != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= set(c.table[1, 4:6].tolist()) and changed
    c.st.zero_()
    seqlens = torch.zeros(2, dtype=torch.int32, device="cuda")
    c.commit([[3], [3]], [1, 1], seqlens)
    assert c.st.item() == K.KVC_DEV_INDEX_OOB and seqlens.tolist() == [0, 300]
    c.table[1, 2] = len(c.k)    # a page of the cache
    c.gpu_table.copy_(c.table)
    c.st.zero_()
    K.kvc_gqa_tree(torch.zeros_like(c.gpu["q"]), c.gpu["q"], c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, block_table=c.gpu_table, status=c.st)
    assert c.st.item() == K.KVC_DEV_INDEX_OOB


def test_rope_range(K):
    c = Case(K, gen(2), 2, 2, 4, 64, 300, 10, [100, 91])
    c.gpu_rope = [x[:101].contiguous() for x in c.gpu_rope]
    before = c.gpu["k"].clone()
    K.kvc_tree_append(c.gpu["k"], c.gpu["v"], c.gpu["new_k"], c.gpu["new_v"], c.depth, c.L, rope=c.gpu_rope, status=c.st)
    assert c.st.item() == K.KVC_DEV_ROPE_RANGE
    assert torch.equal(c.gpu["k"][0], before[0]) and not torch.equal(c.gpu["k"][1], before[1])
    c.st.zero_()
    out = K.kvc_gqa_tree(torch.full_like(c.gpu["q"], 7.0), c.gpu["q"], c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, rope=c.gpu_rope,
                         status=c.st)
    assert c.st.item() == K.KVC_DEV_ROPE_RANGE and (out[0] == 7).all() and not (out[1] == 7).any()


@pytest.mark.parametrize("page", [0, 64])
def test_verified_steps_are_one_token_steps(K, page):
    """A line of a tree, kept, leaves the cache and gives the outputs that one-token steps give: three rounds of
    drafting, then the same tokens one at a time through the append and decode calls; the rounds captured in a graph and
    replayed on another stream."""
    B, H, G, D, C, N = 2, 2, 4, 128, 640, 12
    g = gen(21)
    c = Case(K, g, B, H, G, D, C, N, [200, 63], page, trees=[[-1, 0, 0, 1, 1, 2, 3, 3, 6, 6, 8, 9]] * B)
    line = [0, 1, 3, 6, 9, 11]
    paths = torch.tensor([line, line], dtype=torch.int32, device="cuda")
    counts = torch.tensor([6, 4], dtype=torch.int32, device="cuda")
    sk = torch.tensor([200 - 1, 63 - 1], dtype=torch.int32, device="cuda")
    rounds = 3
    nk, nv = (torch.randn((rounds, B, H, N, D), generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn((rounds, B, H * G, N, D), generator=g).to(BF16).cuda()
    parents = torch.tensor(c.trees, dtype=torch.int32, device="cuda")
    k0, v0 = c.gpu["k"].clone(), c.gpu["v"].clone()

    def verify(k, v):
        outs = []
        for r in range(rounds):
            sk.add_(N)
            L = K.kvc_seq_lengths(sk, N, C, K.KVC_CONTIGUOUS)
            mask, depth = K.kvc_tree_mask(parents)
            K.kvc_tree_append(k, v, nk[r], nv[r], depth, L, block_table=c.gpu_table, rope=c.gpu_rope)
            outs.append(K.kvc_gqa_tree(torch.zeros_like(q[r]), q[r], k, v, mask, depth, L, block_table=c.gpu_table, rope=c.gpu_rope))
            K.kvc_tree_commit(k, v, paths, counts, L, sk, N, block_table=c.gpu_table)
        return outs

    outs = verify(c.gpu["k"], c.gpu["v"])
    total = [200 + 3 * 6, 63 + 3 * 4]
    assert (sk + 1).tolist() == total
    k1, v1 = k0.clone(), v0.clone()
    for r in range(rounds):
        for j in range(6):
            # batch row 1 keeps four: its steps five and six are its step four again
            at = torch.tensor([200 + 6 * r + j, 63 + 4 * r + min(j, 3)], dtype=torch.int32, device="cuda")
            i = [line[j], line[min(j, 3)]]
            L = K.kvc_seq_lengths(at, 1, C, K.KVC_CONTIGUOUS)
            pick = lambda x: torch.stack([x[r, b, :, i[b]:i[b] + 1] for b in range(B)]).contiguous()  # noqa: E731
            out = torch.zeros((B, H * G, 1, D), dtype=BF16, device="cuda")
            if page:
                K.kvc_paged_append(k1, v1, pick(nk), pick(nv), c.gpu_table, L, rope=c.gpu_rope)
                K.kvc_gqa_decode_paged(out, pick(q), k1, v1, c.gpu_table, L, rope=c.gpu_rope)
            else:
                K.kvc_window_append(k1, v1, pick(nk), pick(nv), L, K.KVC_CONTIGUOUS, rope=c.gpu_rope)
                K.kvc_gqa_decode(out, pick(q), k1, v1, L, rope=c.gpu_rope)
            got = pick(outs[r][None].expand(rounds, -1, -1, -1, -1))
            # two kernels within 2 * 2^-8 (query, weights and result in bf16) of the same attention of N(0, 1) values
            assert (got.float() - out.float()).abs().max() < 0.05
    for b in range(B):
        x, y = (t.cuda() for t in c.at(b, torch.arange(total[b])))
        assert torch.equal(c.gpu["k"][x, :, y], k1[x, :, y]) and torch.equal(c.gpu["v"][x, :, y], v1[x, :, y])
    # the same, captured
    k2, v2 = k0.clone(), v0.clone()
    sk.copy_(torch.tensor([199, 62]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = verify(k2, v2)
    k2.copy_(k0)
    v2.copy_(v0)
    sk.copy_(torch.tensor([199, 62]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, again)) and torch.equal(k2, c.gpu["k"])


def test_two_streams_with_their_own_workspaces(K):
    c = Case(K, gen(4), 2, 4, 4, 128, 2000, 16, [1900, 700])
    c.append()
    qs = [c.gpu["q"], (c.gpu["q"] * 0.5).contiguous()]
    want = [K.kvc_gqa_tree(torch.zeros_like(x), x, c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, rope=c.gpu_rope) for x in qs]
    ws = [K.tree_workspace(x, c.gpu["k"]) for x in qs]
    got = [torch.zeros_like(x) for x in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, o, s in zip(qs, ws, got, streams):
            K.kvc_gqa_tree(o, x, c.gpu["k"], c.gpu["v"], c.mask, c.depth, c.L, rope=c.gpu_rope, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
