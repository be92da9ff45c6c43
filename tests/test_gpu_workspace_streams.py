"""What a call allocates for a stream other than the current one (workspace="auto", a tree's masks) comes from
that stream's memory: a block that was freed on the current stream while a kernel queued there still reads it is
not written, and the call's own results are what they are without any of this."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def while_the_current_stream_reads(call, nbytes):
    """call(side) at once, with a block of nbytes just freed on the current stream, where a kernel behind a wait
    still reads it.  Returns whether that kernel read what the block held."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = torch.full((nbytes,), 77, dtype=torch.uint8, device="cuda")
    read = torch.empty_like(held)
    at = held.data_ptr()
    del held
    # the block that an allocation of this size on this stream gets next, and what it holds when the wait ends
    held = torch.full((nbytes,), 77, dtype=torch.uint8, device="cuda")
    assert held.data_ptr() == at
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    read.copy_(held)
    del held
    call(side)
    side.synchronize()
    torch.cuda.synchronize()
    return bool((read == 77).all())


def quant(K):
    B, H, G, D, C = 2, 4, 4, 128, 3000
    g = gen(1)
    kq, vq = (torch.randint(-127, 128, (B, H, C, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand((B, H, C), generator=g, device="cuda") for _ in range(2))
    q = torch.randn((B, H * G, 1, D), generator=g, device="cuda").to(BF16)
    L = K.kvc_seq_lengths(torch.tensor([C - 1, 1233], dtype=torch.int32, device="cuda"), 1, C, K.KVC_CONTIGUOUS)
    return (lambda out, **kw: K.kvc_gqa_decode_quant(out, q, kq, vq, ks, vs, L, K.KVC_CONTIGUOUS, **kw), q,
            K.quant_decode_workspace(q, kq).nbytes)


def tree(K):
    B, H, G, D, C, N = 2, 4, 4, 128, 3000, 9
    g = gen(2)
    k, v = (torch.randn((B, H, C, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((B, H * G, N, D), generator=g, device="cuda").to(BF16)
    L = K.kvc_seq_lengths(torch.tensor([C - 1, 1233], dtype=torch.int32, device="cuda"), N, C, K.KVC_CONTIGUOUS)
    mask, depth = K.kvc_tree_mask(torch.tensor([[i // 2 - 1 if i else -1 for i in range(N)]] * B, dtype=torch.int32, device="cuda"))
    return lambda out, **kw: K.kvc_gqa_tree(out, q, k, v, mask, depth, L, **kw), q, K.tree_workspace(q, k).nbytes


def sparse(K):
    B, H, G, D, page, m = 2, 4, 4, 128, 64, 40
    g = gen(3)
    k, v = (torch.randn((B * m, H, page, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    table = torch.randperm(B * m, generator=g, device="cuda").int().reshape(B, m)
    bounds = torch.randint(-127, 128, (B * m, H, 2, D), generator=g, device="cuda", dtype=torch.int8)
    scale = torch.rand((B * m, H), generator=g, device="cuda")
    q = torch.randn((B, H * G, 1, D), generator=g, device="cuda").to(BF16)
    selected = torch.zeros((B, H, 12), dtype=torch.int32, device="cuda")
    L = K.kvc_seq_lengths(torch.tensor([m * page - 1, 1233], dtype=torch.int32, device="cuda"), 1, m * page, K.KVC_CONTIGUOUS)
    return (lambda out, **kw: K.kvc_gqa_decode_sparse(out, q, k, v, bounds, scale, table, L, selected, **kw), q,
            K.sparse_workspace(q, k, selected).nbytes)


@pytest.mark.parametrize("make", [quant, tree, sparse])
@pytest.mark.parametrize("handle", [False, True])
def test_a_workspace_is_not_memory_that_the_current_stream_reads(K, make, handle):
    call, q, nbytes = make(K)
    want, got = call(torch.zeros_like(q)), torch.zeros_like(q)
    assert while_the_current_stream_reads(lambda s: call(got, stream=s.cuda_stream if handle else s), nbytes)
    assert torch.equal(want, got)


def test_masks_are_not_memory_that_the_current_stream_reads(K):
    B, N = 64, 256
    parents = torch.tensor([[i // 2 - 1 if i else -1 for i in range(N)]] * B, dtype=torch.int32, device="cuda")
    want = K.kvc_tree_mask(parents)
    got = []
    assert while_the_current_stream_reads(lambda s: got.extend(K.kvc_tree_mask(parents, stream=s)), want[0].nbytes)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_masks_freed_while_the_current_stream_reads_them(K):
    """the masks of one call on a side stream, read behind a wait on the current one and freed, and the next call's"""
    B, N = 64, 256
    one, two = (torch.tensor([[i // n - 1 if i else -1 for i in range(N)]] * B, dtype=torch.int32, device="cuda") for n in (2, 3))
    want = K.kvc_tree_mask(one)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mask, depth = K.kvc_tree_mask(one, stream=side)
    side.synchronize()
    read = torch.empty_like(mask)
    torch.cuda._sleep(100_000_000)
    read.copy_(mask)
    del mask, depth
    K.kvc_tree_mask(two, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(read, want)
