"""Attention of a packed batch over a paged cache (kvc_gqa_ragged) within the bound that attention() of
_ops_reference.py derives: the queries enter as they are, the weights are rounded to the cache's type once (fp16's as
halves, whose step below 2^-14 is fixed).

Rows that no token sees -- of pages that no request holds, of a page behind its request's last token -- are NaN."""
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


def ceil(a, b):
    return -(-a // b)


class Case:
    def __init__(self, K, seed, past, new, H, G, D, page, dtype=BF16, pad=3, spread=1.0, max_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.K, self.past, self.new, self.H, self.G, self.D, self.page, self.dtype = K, past, new, H, G, D, page, dtype
        B, self.T = len(past), sum(new)
        total = [p + n for p, n in zip(past, new)]
        most = max_pages or max(1, max(ceil(t, page) for t in total))
        held = sum(ceil(t, page) for t in total)
        self.pool = held + 2
        order = torch.randperm(self.pool, generator=g).tolist()
        self.table = torch.full((B, most), -1, dtype=torch.int32)
        self.k, self.v = torch.full((2, self.pool, H, page, D), math.nan).to(dtype)
        self.rows = []  # each request's (keys, values) [H, total, D]
        for b, t in enumerate(total):
            k, v = spread * torch.randn((H, t, D), generator=g), torch.randn((H, t, D), generator=g)
            self.rows.append((k.to(dtype), v.to(dtype)))
            for j in range(ceil(t, page)):
                id = self.table[b, j] = order.pop()
                z = min(page, t - j * page)
                self.k[id, :, :z] = self.rows[b][0][:, j * page:j * page + z]
                self.v[id, :, :z] = self.rows[b][1][:, j * page:j * page + z]
        self.q = torch.randn((self.T + pad, H * G, D), generator=g).to(dtype)
        self.offsets = torch.tensor([0] + new).cumsum(0).int()
        self.out = torch.randn((self.T + pad, H * G, D), generator=g).to(dtype)
        t = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
        self.lens = torch.stack([t(past), t(total), t(past), t(total), t([0] * B)])

    def set_row(self, b, r, k=None, v=None):
        """row r of request b (columns of every head) becomes k, v"""
        id, at = self.table[b, r // self.page], r % self.page
        for pool, rows, x in ((self.k, self.rows[b][0], k), (self.v, self.rows[b][1], v)):
            if x is not None:
                pool[id, :, at] = x
                rows[:, r] = x

    def gpu(self):
        self.L = self.K.Lengths(len(self.past), "cuda")
        self.L.buf.copy_(self.lens)
        return [x.cuda() for x in (self.out, self.q, self.k, self.v, self.table, self.offsets)]

    def run(self, **kw):
        out, q, k, v, table, offsets = self.gpu()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        self.K.kvc_gqa_ragged(out, q, k, v, table, offsets, self.L, status=st, **kw)
        torch.cuda.synchronize()
        return out.cpu(), st.item()

    def want(self, b, window=0, scale=0.0, some=None):
        """(values, bound) of request b's tokens [n, H * G, D], or of the tokens `some`"""
        k, v = (x.double() for x in self.rows[b])
        i = torch.arange(self.new[b]) if some is None else torch.tensor(some)
        o = int(self.offsets[b])
        q = self.q[o + i].double().reshape(len(i), self.H, self.G, self.D)
        back = (self.past[b] + i)[:, None] - torch.arange(k.shape[1])
        seen = (back >= 0) & (back < (window if window > 0 else 1 << 40))
        outs = []
        half = torch.ones(k.shape[1]) if self.dtype == F16 else None
        for h in range(self.H):
            outs.append(R.attention(q[:, h].reshape(-1, self.D), k[h], v[h], seen.repeat_interleave(self.G, 0),
                                    scale or 1 / math.sqrt(self.D), 0.0, R.half_step(self.dtype), self.dtype, half))
        return [torch.stack([x[j].reshape(len(i), self.G, self.D) for x in outs], 1).reshape(len(i), -1, self.D) for j in (0, 1)]

    def check(self, out, window=0, scale=0.0, skip=(), some=None):
        for b in range(len(self.past)):
            o, n = int(self.offsets[b]), self.new[b]
            if b in skip:
                assert torch.equal(out[o:o + n], self.out[o:o + n]), f"request {b}"
            elif n:
                i = None if some is None else [x for x in some if x < n] + [n - 1]
                want, bound = self.want(b, window, scale, i)
                got = out[o:o + n] if i is None else out[[o + x for x in i]]
                R.assert_within(got, want, bound, f"request {b}: {n} tokens after {self.past[b]}")
        assert torch.equal(out[self.T:], self.out[self.T:])


def ragged(seed, B, high, longest, zero=0.1):
    g = torch.Generator().manual_seed(seed)
    past = torch.randint(0, high + 1, (B,), generator=g).tolist()
    new = torch.randint(1, longest + 1, (B,), generator=g)
    new[torch.rand(B, generator=g) < 0.4] = 1
    new[torch.rand(B, generator=g) < zero] = 0
    return past, new.tolist()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,page,B,high,longest,window", [
    (1, 1, 16, 1, 0, 1, 0), (2, 4, 64, 3, 200, 40, 0), (1, 8, 16, 5, 300, 70, 0), (2, 1, 48, 4, 150, 300, 0), (1, 16, 128, 3, 260, 33, 0),
    (3, 3, 32, 4, 130, 90, 50), (1, 7, 192, 5, 400, 60, 129), (2, 5, 16, 6, 90, 20, 1), (1, 12, 64, 3, 500, 25, 300), (4, 2, 96, 9, 700, 150, 0),
    (8, 4, 64, 12, 300, 1, 0), (2, 4, 16, 40, 60, 5, 17)])
def test_ragged(K, H, G, page, B, high, longest, window, D, dtype):
    past, new = ragged(H * 100 + G + D + B, B, high, longest)
    if not sum(new):
        new[0] = 1
    c = Case(K, B + D, past, new, H, G, D, page, dtype)
    out, st = c.run(local_window_size=window)
    assert st == 0
    c.check(out, window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385])
def test_lengths_around_tiles(K, n, D):
    past = [0, 0, 1, 127, 128, 129, 255]
    c = Case(K, n + D, past, [n, 1, n, 1, n, n, 1], 1, 2, D, 16)
    out, st = c.run()
    assert st == 0
    c.check(out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 80, 112, 160, 256, 320])
def test_page_sizes(K, page, D):
    past, new = ragged(page + D, 6, 600, 200, 0)
    c = Case(K, page, past, new, 2, 4, D, page)
    for window in (0, 333):
        out, st = c.run(local_window_size=window)
        assert st == 0
        c.check(out, window)


def test_extreme_windows(K):
    """No window, the widest and the narrowest."""
    past, new = ragged(77, 5, 400, 150, 0)
    c = Case(K, 77, past, new, 2, 4, 128, 64)
    want, _ = c.run()
    for window in (-1, -2 ** 31, 2 ** 31 - 1, 100000):
        out, st = c.run(local_window_size=window)
        assert st == 0 and (out.float() - want.float()).abs().max() <= 2.0 ** -6  # (other shares of the keys, at most)
        c.check(out)
    out, _ = c.run(local_window_size=1)  # each token itself
    for b in range(5):
        o, n = int(c.offsets[b]), new[b]
        v = c.rows[b][1][:, past[b]:past[b] + n].transpose(0, 1).repeat_interleave(4, 1)
        assert torch.equal(out[o:o + n], v)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_beside_the_paged_decode(K, D):
    """One token a request: what kvc_gqa_decode_paged gives for the same cache, within both calls' roundings (either is
    within the bound of the definition)."""
    past = [0, 63, 64, 500, 1000, 127]
    c = Case(K, 90 + D, past, [1] * 6, 2, 4, D, 64, pad=0)
    c.k, c.v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    out, st = c.run()
    _, q, k, v, table, offsets = c.gpu()
    other = torch.empty((6, 8, 1, D), dtype=BF16, device="cuda")
    K.kvc_gqa_decode_paged(other, q.reshape(6, 8, 1, D), k, v, table, c.L)
    other = other.cpu().reshape(6, 8, D)
    for b in range(6):
        want, bound = c.want(b)
        R.assert_within(out[b:b + 1], want, bound, f"ragged {b}")
        assert ((other[b:b + 1].double() - want).abs() <= 2 * bound + 2.0 ** -7).all()


@pytest.mark.parametrize("D,G", [(64, 8), (128, 4), (128, 7), (256, 2)])
def test_long_rows(K, D, G):
    """Rows whose keys go to many blocks, beside short ones."""
    c = Case(K, D, [20000, 0, 9000, 130], [3, 200, 1, 1], 1, G, D, 64)
    out, st = c.run()
    assert st == 0
    c.check(out)
    out, st = c.run(local_window_size=7001)
    c.check(out, 7001)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_chunk(K, D):
    c = Case(K, 7 + D, [1500, 37], [1300, 900], 2, 4, D, 64)
    out, st = c.run()
    assert st == 0
    some = [0, 1, 31, 32, 63, 64, 100, 127, 128, 500, 511, 640, 899, 1023, 1200]
    c.check(out, some=some)
    out, _ = c.run(local_window_size=400)
    c.check(out, 400, some=some)


def test_shares_in_pieces(K):
    """head_dim 256 and more keys than L2 holds: the CTAs' shares are in two or three pieces (2.6 million units of the line,
    167 MB of keys and values), with and without a window."""
    c = Case(K, 60, [4096, 3900, 4200, 4096], [1024, 1000, 1100, 1], 8, 4, 256, 64)
    some = [0, 1, 31, 32, 63, 64, 500, 767, 999]
    out, st = c.run()
    assert st == 0
    c.check(out, some=some)
    again, _ = c.run()
    assert torch.equal(out, again)
    out, st = c.run(local_window_size=4000)
    c.check(out, 4000, some=some)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [1.0, 0.01, -0.3])
def test_scales(K, scale, D):
    """Sharp, flat and turned weights."""
    c = Case(K, D + 3, [300, 5, 0], [20, 1, 150], 2, 4, D, 32, F16)
    out, st = c.run(scale=scale)
    c.check(out, scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rising_scores(K, D):
    """Scores that rise from tile to tile by more than the reference may lag."""
    c = Case(K, D + 4, [900, 0], [130, 600], 1, 4, D, 64)
    for b in range(2):
        for r in range(c.rows[b][0].shape[1]):
            c.set_row(b, r, k=c.rows[b][0][:, r] * (0.05 + r / 64))
    out, st = c.run()
    c.check(out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_what_is_not_seen_may_hold_anything(K, D, dtype):
    """The rows of a request's later tokens, and those a window has left behind."""
    c = Case(K, D + 5, [300, 10, 129], [40, 200, 1], 1, 4, D, 16, dtype)
    W = 100
    c.set_row(0, 3, k=torch.full((1, D), math.nan).to(dtype), v=torch.full((1, D), math.inf).to(dtype))
    c.set_row(0, 200, v=torch.full((1, D), -math.inf).to(dtype))
    bad = torch.zeros((1, D), dtype=dtype)
    bad[:, 5] = math.nan
    c.set_row(1, 150, v=bad)     # seen by the tokens from position 150 to 249
    c.set_row(1, 205, k=torch.full((1, D), math.nan).to(dtype))
    out, st = c.run(local_window_size=W)
    assert st == 0
    o = int(c.offsets[1])
    for b in range(3):
        want, bound = c.want(b, W)
        n = c.new[b]
        got = out[int(c.offsets[b]):int(c.offsets[b]) + n]
        pos = c.past[b] + torch.arange(n)
        nan = torch.zeros_like(want, dtype=torch.bool)
        if b == 0:
            nan[(pos >= 200) & (pos - 200 < W)] = True
        if b == 1:
            nan[(pos >= 150) & (pos - 150 < W), :, 5] = True
            nan[(pos >= 205) & (pos - 205 < W)] = True
        assert torch.equal(torch.isnan(got), nan), f"request {b}"
        fine = ~nan
        off = (got.double() - clean(c, b, W)).abs()
        assert (off[fine] <= bound_of(c, b, W)[fine]).all()
    assert o == 40


def clean(c, b, W):
    return _clean(c, b, W)[0]


def bound_of(c, b, W):
    return _clean(c, b, W)[1]


def _clean(c, b, W):
    """want() with zeros for the values and keys that are not finite (their rows' outputs are looked at apart)"""
    rows = c.rows[b]
    c.rows[b] = tuple(torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in rows)
    got = c.want(b, W)
    c.rows[b] = rows
    return got


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinite_values_in_whole_tiles(K, D):
    """In a tile that every token sees a column with an infinity is NaN for all, the others are as they were."""
    c = Case(K, D + 6, [600], [70], 1, 2, D, 64)
    bad = c.rows[0][1][:, 40].clone()
    bad[:, 9] = math.inf
    c.set_row(0, 40, v=bad)
    out, st = c.run()
    nan = torch.isnan(out[:70])
    assert nan[:, :, 9].all() and int(nan.sum()) == 70 * 2
    want, bound = _clean(c, 0, 0)
    keep = [i for i in range(D) if i != 9]
    assert ((out[:70].double() - want).abs() <= bound)[:, :, keep].all()


def test_rejected_requests(K):
    c = Case(K, 11, [100, 30, 0, 64, 5], [10, 4, 20, 1, 3], 2, 4, 128, 64)
    good = c.lens.clone()
    c.lens[:, 1] = -1
    out, st = c.run()
    assert st == 0
    c.check(out, skip=(1,))
    c.lens = good.clone()
    c.lens[1, 2] += 1            # lengths and offsets that do not go together
    c.lens[0, 0] = -5
    out, st = c.run()
    assert st == K.KVC_DEV_SEQLEN_RANGE
    c.check(out, skip=(0, 2))
    c.lens = good.clone()
    c.lens[0, 4], c.lens[1, 4] = 64 * c.table.shape[1], 64 * c.table.shape[1] + 3
    out, st = c.run()
    assert st == K.KVC_DEV_CAPACITY
    c.check(out, skip=(4,))
    c.lens = good.clone()
    c.offsets[5] = c.T + 100     # past the buffer
    out, st = c.run()
    assert st == K.KVC_DEV_SEQLEN_RANGE
    c.offsets[5] = c.T
    c.check(out, skip=(4,))


def test_bad_pages(K):
    """An id outside the pool: the others' outputs are as they were."""
    c = Case(K, 12, [100, 300, 0], [10, 4, 20], 2, 4, 128, 64)
    c.table[1, 2], c.table[1, 4] = c.pool, -7
    out, st = c.run()
    assert st == K.KVC_DEV_INDEX_OOB
    for b in (0, 2):
        want, bound = c.want(b)
        o = int(c.offsets[b])
        R.assert_within(out[o:o + c.new[b]], want, bound, f"request {b}")


def test_nothing_to_do(K):
    c = Case(K, 13, [10, 0, 5], [0, 0, 0], 1, 4, 64, 16)
    out, st = c.run()
    assert st == 0 and torch.equal(out, c.out)


def test_many_requests(K):
    past, new = ragged(14, 700, 150, 3)
    c = Case(K, 14, past, new, 1, 4, 64, 16)
    out, st = c.run()
    assert st == 0
    c.check(out)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_same_bits_on_every_run_and_stream(K, D):
    past, new = ragged(15, 9, 900, 300, 0)
    c = Case(K, 15, past, new, 2, 4, D, 64)
    first, _ = c.run()
    s = torch.cuda.Stream()
    for i in range(6):
        out, st = c.run(stream=s if i % 2 else None)
        assert st == 0 and torch.equal(out, first)


def test_two_calls_at_once(K):
    """Two streams, a workspace each."""
    cases = [Case(K, 16 + i, *ragged(20 + i, 6, 2000, 400), 2, 4, 128, 64) for i in range(2)]
    alone = [c.run()[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    state = [c.gpu() + [c.L] for c in cases]
    ws = [K.ragged_workspace(s[1], s[2], len(c.past)) for s, c in zip(state, cases)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (out, q, k, v, table, offsets, L), w, st in zip(state, ws, streams):
            with torch.cuda.stream(st):
                K.kvc_gqa_ragged(out, q, k, v, table, offsets, L, workspace=w)
    torch.cuda.synchronize()
    for s, want in zip(state, alone):
        assert torch.equal(s[0].cpu(), want)


def test_graph_replay_with_other_lengths(K):
    """A captured call reads its lengths from the device: replayed after they changed."""
    c = Case(K, 17, [500, 3, 64, 0], [70, 1, 2, 130], 2, 4, 128, 64)
    d = Case(K, 18, [3, 700, 0, 100], [1, 150, 0, 2], 2, 4, 128, 64, pad=3 + 50, max_pages=c.table.shape[1] + 10)
    want = d.run()[0]
    out, q, k, v, table, offsets = d.gpu()
    L = d.L
    w = K.ragged_workspace(q, k, 4)
    graph = torch.cuda.CUDAGraph()
    L.buf.fill_(-1)
    K.kvc_gqa_ragged(out, q, k, v, table, offsets, L, workspace=w)
    with torch.cuda.graph(graph):
        K.kvc_gqa_ragged(out, q, k, v, table, offsets, L, workspace=w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), d.out)  # every request rejected
    L.buf.copy_(d.lens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)


def test_pool_past_32_bit_offsets(K):
    """Pages whose last element lies past 2^32."""
    D, H, page, G = 256, 8, 64, 2
    pages = (1 << 32) // (D * H * page) + 3
    kp = torch.full((pages, H, page, D), math.nan, dtype=F16, device="cuda")
    vp = torch.full_like(kp, math.nan)
    g = torch.Generator().manual_seed(1)
    c = Case(K, 30, [100], [9], H, G, D, page, F16)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    for j in range(2):
        kp[table[0, j]], vp[table[0, j]] = c.k[c.table[0, j]].cuda(), c.v[c.table[0, j]].cuda()
    out, q, _, _, _, offsets = c.gpu()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvc_gqa_ragged(out, q, kp, vp, table.cuda(), offsets, c.L, status=st)
    assert st.item() == 0 and g is not None
    c.check(out.cpu())


def test_a_whole_step(K):
    """Plan, append and attention of two steps: prompts, then their next tokens beside a new prompt; against the
    requests' whole histories in float64."""
    H, G, D, page, B = 2, 4, 128, 16, 4
    g = torch.Generator().manual_seed(40)
    pool, most = 60, 20
    kp, vp = torch.full((2, pool, H, page, D), math.nan, dtype=BF16, device="cuda")
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, generator=g).int().cuda()
    counts = [torch.tensor([pool], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")]
    cos, sin = torch.zeros((2, 512, D // 2), device="cuda")
    K.kvc_rope_tables(cos, sin, base=50000.0, scaling=K.KVC_ROPE_LINEAR, factor=2.0)
    rope = (cos, sin)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(BF16) for _ in range(2))
    cached, history = [0] * B, [[torch.zeros((0, H, D)), torch.zeros((0, H, D))] for _ in range(B)]
    for step, new in enumerate(([100, 0, 33, 1], [1, 0, 1, 1], [1, 70, 5, 1], [1, 1, 1, 1])):
        n = sum(new) + 2
        plan = K.RaggedPlan(B, n, "cuda")
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        K.kvc_page_release(t([0] * B), table, page, free, counts[0], counts[1], status=st)
        K.kvc_ragged_plan(t(cached), t(new), table, page, free, counts[1], counts[0], plan, status=st)
        qkv = torch.randn((n, (H * G + 2 * H) * D), generator=g).to(BF16)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.cuda().split([H * G * D, H * D, H * D], 1))
        q_out = torch.zeros((n, H * G, D), dtype=BF16, device="cuda")
        K.kvc_ragged_append(q_out, kp, vp, q, k, v, plan.positions, plan.slots, rope=rope, q_weight=wq.cuda(), k_weight=wk.cuda(),
                            status=st)
        out = torch.zeros_like(q_out)
        K.kvc_gqa_ragged(out, q_out, kp, vp, table, plan.offsets, plan.lengths, status=st)
        assert st.item() == 0
        out, qr = out.cpu(), q_out.cpu()
        rows = plan.slots.long()[:n - 2]
        kr, vr = (p[rows // page, :, rows % page].float().cpu() for p in (kp, vp))
        o = 0
        for b in range(B):
            z = new[b]
            history[b] = [torch.cat([history[b][0], kr[o:o + z]]), torch.cat([history[b][1], vr[o:o + z]])]
            total = cached[b] + z
            seen = torch.arange(total)[None] <= (cached[b] + torch.arange(z))[:, None]
            for h in range(H if z else 0):
                want, bound = R.attention(qr[o:o + z, h * G:(h + 1) * G].double().reshape(-1, D), history[b][0][:, h].double(),
                                          history[b][1][:, h].double(), seen.repeat_interleave(G, 0), D ** -0.5, 0.0,
                                          R.half_step(BF16), BF16)
                R.assert_within(out[o:o + z, h * G:(h + 1) * G].reshape(-1, D), want, bound, f"step {step} request {b}")
            cached[b], o = total, o + z
        assert torch.equal(out[o:], torch.zeros_like(out[o:]))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_requests_that_share_pages(K, D):
    """A prefix whose pages are in three rows of the table, and a page twice in one of them."""
    page, H = 32, 2
    c = Case(K, 50, [200, 220, 192, 64], [20, 1, 150, 1], H, 4, D, page)
    for b in (1, 2):
        c.table[b, :6] = c.table[0, :6]
        for x, y in zip(c.rows[b], c.rows[0]):
            x[:, :192] = y[:, :192]
    c.table[3, 1] = c.table[3, 0]
    for x in c.rows[3]:
        x[:, 32:64] = x[:, :32]
    out, st = c.run()
    assert st == 0
    c.check(out)


@pytest.mark.parametrize("D", [64, 256])
def test_positions_up_to_the_last(K, D):
    """Positions up to 2^31 - 512 in a window, the table's entries all one page; a request past that is rejected."""
    page, H, G, W, n = 112, 2, 4, 300, 5
    most, last = ((1 << 31) - 1) // page, (1 << 31) - 512
    c = Case(K, 51, [0], [page], H, G, D, page)
    c.new, c.past = [n, 1], [last - n, last]
    c.T = n + 1
    table = torch.full((2, most), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    c.offsets = torch.tensor([0, n, n + 1], dtype=torch.int32)
    t = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    total = [last, last + 1]
    c.lens = torch.stack([t(c.past), t(total), t(c.past), t(total), t([0, 0])])
    out, q, k, v, _, offsets = c.gpu()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kvc_gqa_ragged(out, q, k, v, table, offsets, c.L, local_window_size=W, status=st)
    assert st.item() == K.KVC_DEV_CAPACITY
    # the same window over the rows that the positions fall on
    first = last - n - W
    at = (torch.arange(first, last) % page)
    c.rows[0] = tuple(x[:, at] for x in c.rows[0])
    c.past[0] -= first
    got = out.cpu()
    want, bound = c.want(0, W)
    R.assert_within(got[:n], want, bound, "last positions")
    assert torch.equal(got[n:], c.out[n:])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("W", [0, 150])
def test_a_value_row_that_is_not_finite_anywhere(K, D, W):
    """One value that is no number in a V row, the row in each place of tiles that are cut, and of those beside them:
    its column is NaN for the tokens that see the row, and for no other."""
    places = [0, 31, 32, 62, 63, 64, 95, 96, 127, 128, 129, 159, 160, 161, 191, 192, 199, 200, 201, 220, 223, 224, 239]
    c = Case(K, D + W, [200] * len(places), [40] * len(places), 1, 4, D, 16)
    for b, r in enumerate(places):
        bad = c.rows[b][1][:, r].clone()
        bad[:, b % D] = (math.nan, math.inf, -math.inf)[b % 3]
        c.set_row(b, r, v=bad)
    out, st = c.run(local_window_size=W)
    assert st == 0
    for b, r in enumerate(places):
        got, pos = out[40 * b:40 * b + 40], 200 + torch.arange(40)
        nan = torch.zeros(got.shape, dtype=torch.bool)
        nan[(pos >= r) & (pos - r < (W or 1 << 30)), :, b % D] = True
        assert torch.equal(torch.isnan(got), nan), f"row {r}"
        want, bound = _clean(c, b, W)
        assert ((got.double() - want).abs() <= bound)[~nan].all(), f"row {r}"
