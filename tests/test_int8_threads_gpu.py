"""Host threads that call the INT8 attention on one stream: the bits of the calls alone."""
import threading

import pytest
import torch

from paged_gqa_attention_head_gb300 import inputs

pytestmark = pytest.mark.gpu


def _decode(dev, lens, seed):
    w = inputs.make_decode(lens, len(lens), 16, 2, 64, seed=seed, kv_dtype="int8")
    c = w.cache
    return [x.to(dev) for x in (w.q, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens, w.sinks)]


def _prefill(dev, new, pre, seed):
    p = inputs.make_prefill(new, 8, 1, 64, seed=seed, prefix_lens=pre, prefix_kv_dtype="int8")
    c = p.prefix
    return [x.to(dev) for x in (p.q, p.k, p.v, p.cu_seqlens, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens, p.sinks)]


def test_two_threads_on_one_stream(sa, cuda_dev):
    """Decodes that split their sequences and prefills that split their blocks, of different shapes, from
    two threads at once on the default stream."""
    jobs = [(sa.decode_int8, _decode(cuda_dev, [30000, 9000, 500], 1)), (sa.prefill_int8, _prefill(cuda_dev, [17], [4000], 2)),
            (sa.decode_int8, _decode(cuda_dev, [7000, 21000, 12000, 1], 3)),
            (sa.prefill_int8, _prefill(cuda_dev, [100, 3], [2500, 900], 4))]
    alone = [f(*a) for f, a in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    start = threading.Barrier(2)

    def work(i):
        start.wait()
        for r in range(100):
            for j in (2 * i, 2 * i + 1) if r % 2 else (2 * i + 1, 2 * i):
                got[i].append((j, jobs[j][0](*jobs[j][1])))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(g) for g in got] == [200, 200]
    for j, (out, lse) in got[0] + got[1]:
        assert torch.equal(out, alone[j][0]) and torch.equal(lse, alone[j][1])
