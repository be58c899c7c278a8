"""Host threads that call the 4-bit attention and the page plan on one stream: the bits of the calls alone; and
status bits of calls that are given no workspace."""
import threading

import pytest
import torch

from paged_gqa_attention_head_gb300 import inputs

pytestmark = pytest.mark.gpu


def _decode(dev, lens, heads, kv_heads, dim, seed):
    w = inputs.make_decode(lens, len(lens), heads, kv_heads, dim, seed=seed)
    c = w.cache
    return [x.to(dev) for x in (w.q, inputs.pack_int4(c.k_pages, c.v_pages), c.block_table, c.lens, w.sinks)]


def _prefill(dev, new, pre, seed):
    p = inputs.make_prefill(new, 8, 1, 64, seed=seed, prefix_lens=pre)
    c = p.prefix
    return [x.to(dev) for x in (p.q, p.k, p.v, p.cu_seqlens, inputs.pack_int4(c.k_pages, c.v_pages), c.block_table, c.lens,
                                p.sinks)]


def _plan(dev, seqs, seed):
    g = torch.Generator().manual_seed(seed)
    new, held = torch.randint(0, 40, (seqs,), generator=g), torch.randint(0, 90, (seqs,), generator=g)
    table = torch.arange(seqs * 9).view(seqs, 9)
    free = torch.arange(seqs * 9, seqs * 21) % (seqs * 12)  # as long as the pool; the first 3 seqs entries count
    return [x.to(torch.int32).to(dev) for x in (new, held, table, free, torch.tensor([seqs * 3]))] + [int(new.sum()) + 3]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_threads_on_one_stream(sa, cuda_dev):
    """Decodes that split their sequences, prefills that split their blocks and plans, of different shapes,
    from two threads at once on the default stream."""
    jobs = [(sa.decode_int4, _decode(cuda_dev, [30000, 9000, 500], 16, 2, 64, 1)), (sa.prefill_int4, _prefill(cuda_dev, [17], [4000], 2)),
            (sa.plan_step, _plan(cuda_dev, 70, 3)),
            (sa.decode_int4, _decode(cuda_dev, [7000, 21000, 1], 16, 1, 128, 4)),
            (sa.prefill_int4, _prefill(cuda_dev, [100, 3], [2500, 900], 5)), (sa.plan_step, _plan(cuda_dev, 900, 6))]
    alone = [f(*a) for f, a in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    start = threading.Barrier(2)

    def work(i):
        start.wait()
        for r in range(100):
            for j in range(3 * i, 3 * i + 3):
                got[i].append((j, jobs[j][0](*jobs[j][1])))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(g) for g in got] == [300, 300]
    for j, r in got[0] + got[1]:
        assert _same(r, alone[j])
    assert sa.default_status() == 0


@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_bad_pages_of_default_calls(sa, cuda_dev, what):
    """The table's entry goes bad and good again between eager calls and replays."""
    f, args, at = ((sa.decode_int4, _decode(cuda_dev, [3000, 100], 16, 2, 64, 7), 2) if what == "decode" else
                   (sa.prefill_int4, _prefill(cuda_dev, [17], [4000], 8), 5))
    table = args[at]
    good = table.clone()
    sa.default_status(cuda_dev)
    alone = f(*args)
    assert sa.default_status() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = f(*args)
    for run in (lambda: f(*args), g.replay):
        table[0, 1] = -5
        run()
        assert sa.default_status(cuda_dev) == sa.STATUS_BAD_PAGE
        table.copy_(good)
        run()
        assert sa.default_status(cuda_dev) == 0
    assert _same((out, lse), alone)


def test_too_few_pages_of_a_captured_plan(sa, cuda_dev):
    """A captured step that takes a page at each replay until the list is empty."""
    d = cuda_dev
    new, lens = torch.ones(1, dtype=torch.int32, device=d), torch.tensor([0], dtype=torch.int32, device=d)
    table = torch.full((1, 8), -1, dtype=torch.int32, device=d)
    free, left = torch.tensor([6, 4, 0, 0, 0, 0, 0], dtype=torch.int32, device=d), torch.tensor([2], dtype=torch.int32, device=d)
    new[0] = 16
    sa.default_status(d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = sa.plan_step(new, lens, table, free, left, 20, update=True)
    for at, (page, size) in enumerate(((4, 1), (6, 0), (None, 0))):
        g.replay()
        assert sa.default_status() == (sa.STATUS_NO_PAGES if page is None else 0)
        assert int(left) == size and int(lens) == min(at + 1, 2) * 16
        want = [-1] * 20 if page is None else [page * 16 + i for i in range(16)] + [-1] * 4
        assert p.slots.tolist() == want
