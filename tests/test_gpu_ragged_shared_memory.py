"""Batches whose sums in shared memory, with what the kernels hold there anyway, just pass what a kernel has without
asking for more (48 KB): each in a process of its own, which has made no larger call before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import torch
from persistent_kv_cache_gb300 import kvc as K

def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
"""

PLAN = """
def call(B):
    plan, zero, left = K.RaggedPlan(B, B, "cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"), i32([-1])
    table, free, st = i32([[-1]] * B), torch.randperm(B, device="cuda").to(torch.int32), i32([0])
    K.kvc_ragged_plan(zero, zero + 1, table, 16, free, i32([B]), left, plan, status=st)
    order = free.flip(0)
    assert st.item() == 0 and left.item() == 0 and torch.equal(table[:, 0], order)
    assert torch.equal(plan.offsets, torch.arange(B + 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(plan.slots, order * 16) and not plan.positions.any()
"""

RELEASE = """
def call(B):
    free, left, st = torch.full((B,), -1, dtype=torch.int32, device="cuda"), i32([-1]), i32([0])
    table = torch.randperm(B, device="cuda").to(torch.int32)[:, None]
    K.kvc_page_release(torch.full_like(free, 16), table, 16, free, i32([0]), left, status=st)
    assert st.item() == 0 and left.item() == B and torch.equal(free, table[:, 0])
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", HEAD + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# (two words a request and one, and 80 bytes: past 49152 from 6134 requests on)
@pytest.mark.parametrize("batches", [(6133, 6134, 6143, 6144, 6145), (6143,)])
def test_plan(batches):
    run(PLAN + f"\nfor B in {batches}: call(B)")


# (a word a request, and 64 bytes: past 49152 from 12273 requests on)
@pytest.mark.parametrize("batches", [(12272, 12273, 12288, 12289), (12288,)])
def test_release(batches):
    run(RELEASE + f"\nfor B in {batches}: call(B)")


@pytest.mark.parametrize("code", [PLAN, RELEASE], ids=["plan", "release"])
def test_two_threads(code):
    """Calls of the most requests beside smaller ones of another thread, each on a stream of its own."""
    run(code + """
import threading
failed = []
def calls(B, n):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(n):
                call(B)
    except Exception as e:
        failed.append((B, e))
threads = [threading.Thread(target=calls, args=a) for a in ((16384, 100), (13000, 300), (50, 300))]
for t in threads: t.start()
for t in threads: t.join()
assert not failed, failed
""")
