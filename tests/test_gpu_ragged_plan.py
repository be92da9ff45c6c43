"""Pages given back (kvc_page_release) and taken with every token's place (kvc_ragged_plan): whole numbers, equal to
a walk over the requests in Python."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ceil(a, b):
    return -(-a // b)


def walk_release(K, released, table, page, stack, count, pool):
    """(stack, left, status)"""
    stack, n, st, full = list(stack), count, 0, False
    if not 0 <= n <= pool:
        n, st = 0, K.KVC_DEV_INDEX_OOB
    end = n
    for b, t in enumerate(released):
        k = ceil(t, page) if t > 0 else 0
        if t < 0 or k > len(table[b]):
            st |= K.KVC_DEV_SEQLEN_RANGE
            continue
        end += k
        if k and end > pool:
            st |= K.KVC_DEV_CAPACITY
            continue
        for j in range(k):
            stack[n] = table[b][j]
            st |= 0 if 0 <= table[b][j] < pool else K.KVC_DEV_INDEX_OOB
            n += 1
    return stack, n, st


def walk_plan(K, cached, new, table, page, stack, count, pool, tokens):
    """(offsets, positions, slots, lengths, table, left, status)"""
    table, n, st = [list(r) for r in table], count, 0
    if not 0 <= n <= pool:
        n, st = 0, K.KVC_DEV_INDEX_OOB
    offsets, pos, slot, lens, full, end = [0], [], [], [], False, 0
    most = len(table[0]) * page if table else 0
    for b, (P, S) in enumerate(zip(cached, new)):
        bad = 0
        if P < 0 or S < 0 or P + S > 2 ** 31 - 1:
            bad, S = K.KVC_DEV_SEQLEN_RANGE, 0
        end += S
        if not bad and (P + S > most or (S and end > tokens)):
            bad = K.KVC_DEV_CAPACITY
        elif not bad and S and P % page and not 0 <= table[b][P // page] < pool:
            bad = K.KVC_DEV_INDEX_OOB
        want = 0 if bad else ceil(P + S, page) - ceil(P, page)
        if want and (full or want > n):
            bad, full = K.KVC_DEV_CAPACITY, True
        st |= bad
        if not bad:
            for j in range(want):
                n -= 1
                ok = 0 <= stack[n] < pool
                st |= 0 if ok else K.KVC_DEV_INDEX_OOB
                table[b][ceil(P, page) + j] = stack[n] if ok else -1
        for p in range(P, P + S):
            if bad:
                pos.append(-1)
                slot.append(-1)
            else:
                pos.append(p)
                at = table[b][p // page]
                slot.append(at * page + p % page if at >= 0 else -1)
        offsets.append(min(end, tokens))
        lens.append([-1] * 5 if bad else [P, P + S, P, P + S, 0])
    pad = [-1] * max(0, tokens - len(pos))
    return offsets, (pos + pad)[:tokens], (slot + pad)[:tokens], lens, table, n, st


class Pool:
    def __init__(self, K, g, cached, page, max_pages, pool):
        self.K, self.page, self.pool = K, page, pool
        order = torch.randperm(pool, generator=g).tolist()
        self.table = [[-1] * max_pages for _ in cached]
        for b, t in enumerate(cached):
            for j in range(max(0, min(ceil(t, page), max_pages))):
                self.table[b][j] = order.pop()
        self.stack, self.count = order + [-1] * (pool - len(order)), len(order)

    def plan(self, cached, new, tokens, graph=False):
        K = self.K
        plan = K.RaggedPlan(len(cached), tokens, "cuda")
        table, stack, count, left = i32(self.table).reshape(len(cached), -1), i32(self.stack), i32([self.count]), i32([-7])
        st = i32([0])
        args = (i32(cached), i32(new), table, self.page, stack, count, left, plan)
        if graph:
            K.kvc_ragged_plan(*args, status=st)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                K.kvc_ragged_plan(*args, status=st)
            plan.positions.fill_(-9), plan.slots.fill_(-9)
            graph.replay()
        else:
            K.kvc_ragged_plan(*args, status=st)
        want = walk_plan(K, cached, new, self.table, self.page, self.stack, self.count, self.pool, tokens)
        assert plan.offsets.tolist() == want[0]
        assert plan.positions.tolist() == want[1]
        assert plan.slots.tolist() == want[2]
        assert plan.lengths.buf.T.tolist() == want[3]
        assert table.tolist() == want[4]
        assert left.item() == want[5]
        assert st.item() == want[6]
        assert stack.tolist() == self.stack and count.item() == self.count
        self.table, self.count = want[4], want[5]
        return plan, st.item()

    def release(self, released):
        K = self.K
        table, stack, count, left, st = i32(self.table), i32(self.stack), i32([self.count]), i32([-7]), i32([0])
        K.kvc_page_release(i32(released), table, self.page, stack, count, left, status=st)
        want = walk_release(K, released, self.table, self.page, self.stack, self.count, self.pool)
        assert stack.tolist() == want[0] and left.item() == want[1] and st.item() == want[2]
        assert table.tolist() == self.table and count.item() == self.count
        self.stack, self.count = want[0], want[1]
        return st.item()


@pytest.mark.parametrize("B,page,low,high,longest", [(1, 1, 0, 5, 3), (1, 64, 0, 0, 1), (3, 16, 0, 100, 40), (33, 48, 1, 300, 1),
                                                     (255, 16, 0, 200, 30), (256, 128, 0, 500, 300), (257, 7, 0, 99, 20),
                                                     (1000, 64, 0, 2000, 3)])
def test_plan(K, B, page, low, high, longest):
    g = torch.Generator().manual_seed(B * 1000 + page)
    cached = torch.randint(low, high + 1, (B,), generator=g).tolist()
    new = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    most = ceil(high + longest, page) + 1
    P = Pool(K, g, cached, page, most, B * most + 5)
    plan, st = P.plan(cached, new, sum(new) + 11)
    assert st == 0
    # no slot twice
    used = [s for s in plan.slots.tolist() if s >= 0]
    assert len(set(used)) == len(used) == sum(new)


@pytest.mark.parametrize("pool", [150, 60])
def test_steps_with_releases(K, pool):
    """A loop of steps: requests end, their pages are taken by others (24 requests of up to 7 pages: 60 are too few at times)."""
    g = torch.Generator().manual_seed(5)
    B, page, most = 24, 16, 12
    cached = [0] * B
    P = Pool(K, g, cached, page, most, pool)
    refused = 0
    for step in range(40):
        ended = [c if c > 100 or torch.rand((), generator=g) < 0.1 else 0 for c in cached]
        assert P.release(ended) == 0
        cached = [0 if e else c for c, e in zip(cached, ended)]
        new = torch.randint(0, 12, (B,), generator=g).tolist()
        plan, st = P.plan(cached, new, 256)
        total = plan.lengths.total_abs.tolist()
        refused += sum(t < 0 for t in total)
        cached = [t if t >= 0 else c for t, c in zip(total, cached)]
        held = [r[j] for r, c in zip(P.table, cached) for j in range(ceil(c, page))]
        assert len(set(held)) == len(held)
        assert sorted(held + P.stack[:P.count]) == list(range(pool))
    assert (refused > 0) == (pool == 60)


def test_rejected_requests(K):
    g = torch.Generator().manual_seed(9)
    page, most = 16, 4
    cached = [5, -1, 20, 60, 2 ** 31 - 1, 33, 17, 0, 48]
    new = [3, 4, -2, 10, 5, 40, 6, 0, 16]
    for tokens in (200, 64, 30, 8, 3, 1, 0):
        P = Pool(K, g, cached, page, most, 40)
        P.plan(cached, new, tokens)
    P = Pool(K, g, cached, page, most, 40)
    P.table[0][0] = 40       # goes on in a page that is not there
    P.table[6][1] = -1
    _, st = P.plan(cached, new, 200)
    assert st & K.KVC_DEV_INDEX_OOB and st & K.KVC_DEV_CAPACITY and st & K.KVC_DEV_SEQLEN_RANGE


@pytest.mark.parametrize("count", [0, 1, 2, 3, 5, -1, 100])
def test_few_free_pages(K, count):
    g = torch.Generator().manual_seed(count + 50)
    cached, new = [16, 10, 0, 32, 0], [1, 3, 20, 16, 1]
    P = Pool(K, g, cached, 16, 4, 30)
    P.count = count
    P.plan(cached, new, 64)


def test_bad_ids_on_the_stack(K):
    g = torch.Generator().manual_seed(3)
    cached, new = [0, 0], [40, 20]
    P = Pool(K, g, cached, 16, 4, 12)
    P.stack[P.count - 2], P.stack[P.count - 4] = 12, -5
    _, st = P.plan(cached, new, 64)
    assert st == K.KVC_DEV_INDEX_OOB


def test_release_refusals(K):
    g = torch.Generator().manual_seed(4)
    cached = [30, 64, 1, 17, 0]
    P = Pool(K, g, cached, 16, 4, 30)
    assert P.release([-1, 64, 0, 65, 0]) == K.KVC_DEV_SEQLEN_RANGE
    P = Pool(K, g, cached, 16, 4, 30)
    P.count = 25
    assert P.release([30, 64, 1, 17, 0]) == K.KVC_DEV_CAPACITY
    P = Pool(K, g, cached, 16, 4, 30)
    P.table[1][2], P.table[3][0] = 30, -1
    assert P.release([30, 64, 1, 17, 0]) == K.KVC_DEV_INDEX_OOB
    P.count = 31
    assert P.release([1, 0, 0, 0, 0]) & K.KVC_DEV_INDEX_OOB


def test_empty(K):
    st, left = i32([0]), i32([-1])
    plan = K.RaggedPlan(0, 5, "cuda")
    K.kvc_ragged_plan(i32([]), i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 16, i32([1, 2, 3]), i32([2]), left, plan, status=st)
    assert plan.offsets.tolist() == [0] and plan.positions.tolist() == [-1] * 5 and plan.slots.tolist() == [-1] * 5
    assert left.item() == 2 and st.item() == 0
    K.kvc_page_release(i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 16, i32([1, 2, 3]), i32([2]), left, status=st)
    assert left.item() == 2 and st.item() == 0


def test_most_requests(K):
    """16384 requests: two words of shared memory each."""
    g = torch.Generator().manual_seed(8)
    B = 16384
    cached = torch.randint(0, 40, (B,), generator=g).tolist()
    new = torch.randint(0, 3, (B,), generator=g).tolist()
    P = Pool(K, g, cached, 32, 2, 2 * B)
    _, st = P.plan(cached, new, sum(new) + 1)
    assert st == 0
    assert P.release(cached) == 0


def test_in_a_graph_and_on_another_stream(K):
    g = torch.Generator().manual_seed(2)
    cached, new = [5, 0, 31, 16], [20, 3, 1, 0]
    P = Pool(K, g, cached, 16, 4, 20)
    P.plan(cached, new, 40, graph=True)
    P = Pool(K, g, cached, 16, 4, 20)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        P.plan(cached, new, 40)
