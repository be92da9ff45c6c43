"""A call that is the first thing a host thread asks of CUDA: the results of the same call on the thread that has been at
work all along."""
import threading

import pytest
import torch

from test_gpu_workspace_streams import K, gen, quant, sparse, tree  # noqa: F401

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(g, *s):
    return torch.randn(s, generator=g, device="cuda").to(BF16)


def decode(K):  # noqa: F811
    g = gen(5)
    q, k, v = rand(g, 2, 8, 1, 128), rand(g, 2, 2, 300, 128), rand(g, 2, 2, 300, 128)
    L, ws = K.kvc_seq_lengths(i32(299, 17), 1, 300, K.KVC_CONTIGUOUS), K.decode_workspace(q, k)
    return lambda out, **kw: K.kvc_gqa_decode(out, q, k, v, L, workspace=ws, **kw), q


def prefill(K):  # noqa: F811
    g = gen(6)
    q, k, v = rand(g, 2, 8, 40, 128), rand(g, 2, 2, 300, 128), rand(g, 2, 2, 300, 128)
    L = K.kvc_seq_lengths(i32(299, 77), 40, 300, K.KVC_CONTIGUOUS)
    return lambda out, **kw: K.kvc_gqa_prefill_chunk(out, q, k, v, L, workspace=None, **kw), q


def window(K):  # noqa: F811
    g = gen(7)
    q, k, v, nk, nv = rand(g, 2, 8, 1, 64), *(rand(g, 2, 2, n, 64) for n in (128, 128, 1, 1))
    last = i32(299, 77)
    return lambda out, **kw: K.kvc_window_decode_step(out, q, k, v, nk, nv, last, 128, windowed=K.KVC_RING, **kw), q


def ragged(K):  # noqa: F811
    g = gen(8)
    q, k, v = rand(g, 43, 8, 128), rand(g, 20, 2, 64, 128), rand(g, 20, 2, 64, 128)
    table, L = torch.randperm(20, generator=g, device="cuda").to(torch.int32).reshape(2, 10), K.Lengths(2, "cuda")
    L.buf.copy_(torch.tensor([[500, 3], [540, 6], [500, 3], [540, 6], [0, 0]]))
    ws, offsets = K.ragged_workspace(q, k, 2), i32(0, 40, 43)
    return lambda out, **kw: K.kvc_gqa_ragged(out, q, k, v, table, offsets, L, workspace=ws, **kw), q


def places(K):  # noqa: F811
    plan, count, left = K.RaggedPlan(2, 64, "cuda"), i32(16), i32(0)
    table, free = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), torch.arange(16, dtype=torch.int32, device="cuda")
    cached, new = i32(0, 0), i32(40, 3)

    def call(out, **kw):
        K.kvc_ragged_plan(cached, new, table, 16, free, count, left, plan, **kw)
        out.copy_(plan.slots)
    return call, plan.slots


def tables(K):  # noqa: F811
    cos, sin = torch.empty((2, 40, 32), device="cuda")
    return lambda out, **kw: out.copy_(K.kvc_rope_tables(cos, sin, **kw)[1]), sin


@pytest.mark.parametrize("make", [decode, prefill, window, ragged, places, tables, quant, tree, sparse])
def test_first_call_of_a_thread(K, make):  # noqa: F811
    call, like = make(K)[:2]
    want, got = torch.zeros_like(like), torch.zeros_like(like)
    call(want)
    torch.cuda.synchronize()
    failed = []

    def run():
        try:
            call(got)
        except Exception as e:  # (told by the test's own thread)
            failed.append(e)
    for _ in range(3):
        got.zero_()
        torch.cuda.synchronize()
        t = threading.Thread(target=run)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        assert torch.equal(got, want)
