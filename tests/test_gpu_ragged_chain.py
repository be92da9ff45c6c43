"""The calls of a ragged step one right behind the other on a stream: what a kernel writes is what the next one reads."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import kvc
    return kvc


@pytest.mark.parametrize("graph", [False, True])
def test_attention_right_behind_a_plan(K, graph):
    """Pages that a plan has just put into the table, read by an attention with nothing between the two: the bits of the
    same attention on a stream that has been waited for."""
    B, H, G, D, page, most = 40, 2, 4, 128, 16, 40
    g = torch.Generator(device="cuda").manual_seed(11)
    pool = B * most
    k, v = torch.randn((2, pool, H, page, D), generator=g, device="cuda").to(torch.bfloat16)
    new = torch.randint(1, 200, (B,), generator=g, device="cuda", dtype=torch.int32)
    cached = torch.randint(0, 20, (B,), generator=g, device="cuda", dtype=torch.int32) * page
    T = int(new.sum())
    q = torch.randn((T, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
    out, st = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    table, free = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, most), (pool,)))
    count, left = torch.tensor([[pool - B * 20], [0]], dtype=torch.int32, device="cuda")
    plan, ws = K.RaggedPlan(B, T, "cuda"), K.ragged_workspace(q, k, B)

    def step():
        K.kvc_ragged_plan(cached, new, table, page, free, count, left, plan, status=st)
        K.kvc_gqa_ragged(out, q, k, v, table, plan.offsets, plan.lengths, workspace=ws, status=st)

    def fill():
        # other pages every time: 20 a request are held, the others free
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table[:, :20], table[:, 20:] = order[:B * 20].reshape(B, 20), -1
        free.copy_(order)
        free[:pool - B * 20] = order[B * 20:]
        out.zero_()

    fill()
    run = step
    if graph:
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        run = captured.replay
    for _ in range(30):
        fill()
        run()
        torch.cuda.synchronize()
        got = out.clone()
        assert (table[:, 0] >= 0).all() and st.item() == 0
        torch.cuda.synchronize()
        K.kvc_gqa_ragged(out.zero_(), q, k, v, table, plan.offsets, plan.lengths, workspace=ws, status=st)
        torch.cuda.synchronize()
        assert torch.equal(out, got)
