"""The page plan and the release at the batch sizes around 48 KB of shared memory, in a process of their own (a launch
with more leaves the kernel a higher limit)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# 12 B + 4 bytes of lengths for a plan of B requests, 8 B for a release, and some 500 bytes beside them
SIZES = """
import torch
from paged_gqa_attention_head_gb300 import sinkattn as sa

def i32(n, v):
    return torch.full((n,), v, dtype=torch.int32, device="cuda")

for update in (False, True):
    for B in (4051, 4052, 4095, 4096):
        free = torch.arange(B, dtype=torch.int32, device="cuda")
        p = sa.plan_step(i32(B, 1), i32(B, 0), i32(2 * B, -1).view(B, 2), free, i32(1, B), B, update=update)
        assert torch.equal(p.slots, 16 * free.flip(0).long()) and int(p.num_free) == 0, B
    for B in (6078, 6079, 6144, 6145):
        table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
        free = i32(B, -1)
        lens, left = sa.release_pages(torch.ones(B, dtype=torch.bool, device="cuda"), i32(B, 3), table, free, i32(1, 0),
                                      update=update)
        assert torch.equal(free, table.view(-1).flip(0)) and int(left) == B and not bool(lens.any()), B
assert sa.default_status() == 0
"""


def test_sizes_around_48_kb(sa, cuda_dev):
    run = subprocess.run([sys.executable, "-c", SIZES], cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT},
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
