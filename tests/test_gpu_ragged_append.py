"""Norm, rotation and append of a packed batch (kvc_ragged_append) against float64, row by row.

A normed value is off by the sum of squares ((D + 1) / 2 roundings at most after the square root: D 2^-24 covers
them with the quotient, eps and the inverse root's 2 ulp) and two products; the rotation by three roundings of its
two products; the result by its own half step."""
import pytest
import torch

import _ops_reference as R

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def turned(x, cos, sin, inter):
    """rows [T, heads, D] in float64 -> (rotated, sum of the products' magnitudes)"""
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    c, s = cos[:, None], sin[:, None]
    z, m = x.clone(), x.abs()
    lo, hi = a * c - b * s, b * c + a * s
    ml, mh = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    if inter:
        z[..., 0:r:2], z[..., 1:r:2], m[..., 0:r:2], m[..., 1:r:2] = lo, hi, ml, mh
    else:
        z[..., :r // 2], z[..., r // 2:r], m[..., :r // 2], m[..., r // 2:r] = lo, hi, ml, mh
    return z, m


def reference(x, w, eps, rope, pos, inter):
    """(values, bound) of the rows x [T, heads, D] of a 16-bit type"""
    D, y = x.shape[-1], x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    z, m = y, y.abs()
    if rope is not None:
        z, m = turned(y, rope[0][pos].double(), rope[1][pos].double(), inter)
    steps = (D + 8 if w is not None else 0) + (4 if rope is not None else 0)
    bound = m * steps * 2.0 ** -24
    tiny = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps
    return z, bound + (z.abs() + bound) * R.half_step(x.dtype) + tiny


class Case:
    def __init__(self, K, seed, T, Hq, H, D, page, dtype, turned=None, inter=False, norm=(True, True), far=500, pad=0, packed=True, eps=1e-6):
        g = torch.Generator().manual_seed(seed)
        self.K, self.T, self.Hq, self.H, self.D, self.page, self.inter, self.eps = K, T, Hq, H, D, page, inter, eps
        n = T + pad
        rand = lambda *s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
        if packed:
            qkv = rand(n, (Hq + 2 * H) * D)
            self.qkv = qkv.cuda()
            cut = lambda t: [x.unflatten(1, (-1, D)) for x in t.split([Hq * D, H * D, H * D], 1)]  # noqa: E731
            (self.q, self.k, self.v), (self.gq, self.gk, self.gv) = cut(qkv), cut(self.qkv)
        else:
            self.q, self.k, self.v = rand(n, Hq, D), rand(n, H, D), rand(n, H, D)
            self.gq, self.gk, self.gv = self.q.cuda(), self.k.cuda(), self.v.cuda()
        self.qw = 1 + 0.3 * torch.randn(D, generator=g) if norm[0] else None
        self.kw = 1 + 0.3 * torch.randn(D, generator=g) if norm[1] else None
        self.qw, self.kw = (None if w is None else w.to(dtype) for w in (self.qw, self.kw))
        pages = -(-n // page) + 2
        self.pos = torch.randint(0, far, (n,), generator=g).int()
        self.slot = torch.randperm(pages * page, generator=g)[:n].int()
        self.slot[T:], self.pos[T:] = -1, -1
        self.rope = R.rope_tables(far, turned) if turned else None
        self.kp, self.vp = rand(pages, H, page, D), rand(pages, H, page, D)
        self.out = rand(n, Hq, D)

    def run(self, q_out=None, stream=None, **kw):
        self.gkp, self.gvp = self.kp.cuda(), self.vp.cuda()
        out = self.out.cuda() if q_out is None else q_out
        cu = lambda x: None if x is None else x.cuda()  # noqa: E731
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        rope = None if self.rope is None else tuple(x.cuda() for x in self.rope)
        self.args = dict(rope=rope, interleaved=self.inter, q_weight=cu(self.qw), k_weight=cu(self.kw), eps=self.eps, status=st)
        pos, slot = self.pos.cuda(), self.slot.cuda()
        torch.cuda.synchronize()
        self.K.kvc_ragged_append(out, self.gkp, self.gvp, self.gq, self.gk, self.gv, pos, slot, stream=stream, **{**self.args, **kw})
        torch.cuda.synchronize()
        return out, st.item()

    def check(self, out):
        keep = self.slot >= 0
        pos = self.pos.clamp(min=0).long()
        want, bound = reference(self.q, self.qw, self.eps, self.rope, pos, self.inter)
        R.assert_within(out[keep.cuda()], want[keep], bound[keep], "queries")
        assert torch.equal(out.cpu()[~keep], self.out[~keep])
        want, bound = reference(self.k, self.kw, self.eps, self.rope, pos, self.inter)
        slot = self.slot[keep].long()
        at = (slot // self.page, slice(None), slot % self.page)
        R.assert_within(self.gkp.cpu()[at], want[keep], bound[keep], "keys")
        assert torch.equal(self.gvp.cpu()[at], self.v[keep])
        # nothing else is written
        left = torch.ones(self.kp.shape[0], self.page, dtype=torch.bool)
        left[slot // self.page, slot % self.page] = False
        for pool, was in ((self.gkp, self.kp), (self.gvp, self.vp)):
            assert torch.equal(pool.cpu().transpose(1, 2)[left], was.transpose(1, 2)[left])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,Hq,H,D,page,turned,inter", [
    (1, 1, 1, 16, 16, 16, False), (1, 32, 8, 128, 64, 128, False), (3, 4, 2, 64, 16, 32, True), (5, 7, 1, 80, 48, 48, False),
    (17, 12, 4, 96, 16, 96, True), (33, 6, 3, 112, 1, 16, False), (40, 5, 5, 192, 192, 192, False), (9, 16, 2, 256, 128, 240, True),
    (200, 64, 8, 64, 64, 64, False), (700, 2, 1, 32, 7, 32, True), (64, 3, 1, 256, 64, 256, False), (7, 4, 2, 128, 64, 0, False),
    (1200, 32, 8, 128, 64, 64, False)])
@pytest.mark.parametrize("norm", [(True, True), (False, False), (True, False)])
def test_append(K, T, Hq, H, D, page, turned, inter, norm, dtype):
    c = Case(K, T + D, T, Hq, H, D, page, dtype, turned, inter, norm, pad=T % 5)
    out, st = c.run()
    assert st == 0
    c.check(out)


def test_dense_and_in_place(K):
    c = Case(K, 1, 50, 8, 2, 128, 64, BF16, 128, packed=False)
    out, st = c.run()
    c.check(out)
    out2, st = c.run(q_out=c.gq)  # the queries' own buffer
    assert st == 0 and torch.equal(out, out2)


def test_bits_of_the_paged_append(K):
    """Without a norm, all columns turned by halves: the rows of kvc_paged_append."""
    B, H, D, page, n = 3, 2, 128, 64, 5
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn((2, B, H, n, D), generator=g).to(BF16).cuda()
    past = torch.tensor([0, 62, 100], dtype=torch.int32)
    table = torch.randperm(8, generator=g)[:6].int().reshape(B, 2)
    rope = tuple(x.cuda() for x in R.rope_tables(200, D))
    pools = [torch.zeros((2, 8, H, page, D), dtype=BF16, device="cuda") for _ in range(2)]
    L = K.kvc_seq_lengths((past + n - 1).cuda(), n, 2 * page, K.KVC_CONTIGUOUS)
    K.kvc_paged_append(pools[0][0], pools[0][1], k, v, table.cuda(), L, rope=rope)
    pos = past[:, None] + torch.arange(n)
    slot = table[torch.arange(B)[:, None], pos // page] * page + pos % page
    rows = lambda x: x.transpose(1, 2).reshape(B * n, H, D).contiguous()  # noqa: E731
    q = rows(k)
    K.kvc_ragged_append(torch.empty_like(q), pools[1][0], pools[1][1], q, rows(k), rows(v), pos.reshape(-1).int().cuda(),
                        slot.reshape(-1).int().cuda(), rope=rope)
    assert torch.equal(pools[0], pools[1])


def test_refused_tokens(K):
    c = Case(K, 2, 12, 4, 2, 64, 16, F16, 64, far=100)
    rows = c.kp.shape[0] * c.page
    good = c.slot.clone()
    c.slot[3], c.slot[7] = rows, rows + 1000
    out, st = c.run()
    assert st == K.KVC_DEV_INDEX_OOB
    c.slot[3] = c.slot[7] = -1
    c.check(out)
    c.slot = good
    c.pos[2], c.pos[5] = 100, -1
    out, st = c.run()
    assert st == K.KVC_DEV_ROPE_RANGE
    c.slot[2] = c.slot[5] = c.pos[2] = -1
    c.check(out)


def test_values_that_are_not_finite_stay_in_their_row(K):
    c = Case(K, 4, 9, 4, 2, 128, 16, BF16, 64)
    c.gq[4, 1, 5], c.q[4, 1, 5] = float("nan"), float("nan")
    c.gv[2, 0, 3], c.v[2, 0, 3] = float("inf"), float("inf")
    out, st = c.run()
    assert st == 0
    got = out.cpu()
    assert torch.isnan(got[4, 1]).all()
    keep = torch.ones(9, 4, dtype=torch.bool)
    keep[4, 1] = False
    assert torch.isfinite(got[keep]).all()
    assert torch.equal(c.gvp.cpu()[c.slot.long() // 16, :, c.slot.long() % 16], c.v)


def test_zero_rows_and_large_ones(K):
    """eps keeps a row of zeros zero; squares of bf16 values up to 2^60 sum below 2^128."""
    c = Case(K, 6, 6, 2, 1, 64, 16, BF16, 64)
    c.gq[1], c.q[1] = 0, 0
    c.gq[3] *= 2.0 ** 58
    c.q[3] *= 2.0 ** 58
    c.gk[2] *= 2.0 ** -30
    c.k[2] *= 2.0 ** -30
    out, st = c.run()
    c.check(out)


def test_another_stream(K):
    c = Case(K, 8, 300, 8, 2, 128, 64, BF16, 128)
    s = torch.cuda.Stream()
    out, st = c.run(stream=s)
    c.check(out)


def test_graph_replay(K):
    c = Case(K, 9, 30, 8, 2, 128, 64, BF16, 128)
    want, _ = c.run()
    pools = c.gkp.clone(), c.gvp.clone()
    out, gk, gv = c.out.cuda(), c.kp.cuda(), c.vp.cuda()
    pos, slot = c.pos.cuda(), c.slot.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kvc_ragged_append(out, gk, gv, c.gq, c.gk, c.gv, pos, slot, **c.args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(gk, pools[0]) and torch.equal(gv, pools[1])


def test_pool_past_32_bit_offsets(K):
    """Rows of a pool whose last element lies past 2^32."""
    D, H, page = 256, 8, 64
    pages = (1 << 32) // (D * H * page) + 3
    kp = torch.zeros((pages, H, page, D), dtype=F16, device="cuda")
    vp = torch.zeros_like(kp)
    slot = torch.tensor([0, (pages - 1) * page + 63, (pages - 2) * page], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((3, H, D), generator=g).to(F16).cuda() for _ in range(3))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = K.kvc_ragged_append(torch.empty_like(q), kp, vp, q, k, v, slot.cuda(), slot.cuda(), status=st)
    assert st.item() == 0 and torch.equal(out, q)
    at = (slot // page).long().cuda(), (slot % page).long().cuda()
    assert torch.equal(kp[at[0], :, at[1]], k) and torch.equal(vp[at[0], :, at[1]], v)
    assert int((kp != 0).any(-1).sum()) == 3 * H
