"""The page plan and the release at the batch sizes around 48 KB of shared memory, in a process of their own (a launch
with more leaves the kernel a higher limit), and from threads with batches of unlike size."""
import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import plain

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


def test_threads_with_batches_of_unlike_size(sa, cuda_dev):
    """Every thread's plans launch, whatever the others' sizes: the library's calls alone, as fast as they go."""
    lib, wrong = sa.load(), []
    batches = (4500, 8192, 5500, 8000)
    start = threading.Barrier(len(batches))

    def work(B):
        r = np.random.default_rng(B)
        new, held = r.integers(0, 4, B), r.integers(0, 16, B)
        table = np.full((B, 2), -1)
        table[:, 0] = np.arange(B)
        free = np.concatenate([np.arange(B, 2 * B), np.zeros(B, dtype=np.int64)])
        T = int(new.sum())
        want = plain.plan_step(new, held, table, free, B, T)
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=cuda_dev)
        ins = [i32(new), i32(held), i32(table), i32(free), i32([B])]
        outs = [torch.empty(n, dtype=torch.int32, device=cuda_dev) for n in (B + 1, B, B, 1, T)]
        slots = torch.empty(T, dtype=torch.int64, device=cuda_dev)
        stream = torch.cuda.Stream(cuda_dev)
        desc = sa.PagedDesc(num_seqs=B, num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=16, num_pages=2 * B,
                            max_pages_per_seq=2)
        torch.cuda.synchronize()
        at = [x.data_ptr() for x in ins + outs]
        start.wait(60)
        codes = set()
        for i in range(3000):
            codes.add(lib.sinkattn_plan_step(*at[:5], T, *at[5:], slots.data_ptr(), ctypes.byref(desc), None, 0,
                                             stream.cuda_stream))
            if i % 100 == 99:
                stream.synchronize()
        if codes != {sa.OK} or not np.array_equal(slots.cpu().numpy(), want["slots"]):
            wrong.append((B, codes))

    threads = [threading.Thread(target=work, args=(B,)) for B in batches]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
