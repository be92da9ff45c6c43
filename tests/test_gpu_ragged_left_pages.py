"""Pages that a local window has left behind may be given back: their entries in the table, whatever they are by then,
are not looked at by the attention (kvc_gqa_ragged) or by the next step's plan (kvc_ragged_plan)."""
import pytest
import torch

from test_gpu_ragged_attn import BF16, F16, Case, K, ceil  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,window", [(16, 33), (64, 200), (48, 1), (128, 128), (256, 300)])
@pytest.mark.parametrize("entry", [-1, 10 ** 9, -2 ** 31])
def test_attention(K, D, page, window, entry, dtype):  # noqa: F811
    past, new = [0, 31, 500, 513, 900, 255], [3, 1, 130, 1, 40, 257]
    c = Case(K, page + D, past, new, 2, 4, D, page, dtype)
    for b, p in enumerate(past):
        c.table[b, :max(0, p - window + 1) // page] = entry  # (up to the page of the first row that its first token sees)
    out, st = c.run(local_window_size=window)
    assert st == 0
    c.check(out, window)


def test_plan(K):  # noqa: F811
    page, most, pool = 16, 12, 40
    cached, new = [100, 37, 0, 64], [5, 1, 20, 1]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((4, most), -1, dtype=torch.int32)
    for b, p in enumerate(cached):
        if p % page:
            table[b, p // page] = 30 + b  # the page that it goes on in; the others were given back
    table, before = table.cuda(), table
    plan, left, st = K.RaggedPlan(4, 27, "cuda"), i32([0]), i32([0])
    K.kvc_ragged_plan(i32(cached), i32(new), table, page, torch.arange(pool, dtype=torch.int32, device="cuda"), i32([30]), left, plan, status=st)
    assert st.item() == 0 and left.item() == 30 - 3
    want = before.clone()
    want[2, :2], want[3, 4] = torch.tensor([29, 28]), 27
    assert torch.equal(table.cpu(), want) and plan.lengths.buf[1].tolist() == [105, 38, 20, 65]
    slots = plan.slots.tolist()
    assert slots[:5] == [30 * 16 + 4 + i for i in range(5)] and slots[5] == 31 * 16 + 5 and slots[26] == 27 * 16
