"""The page plan and the release on the GPU, whole numbers equal to their plain forms, and a serving
run of the plan with the 4-bit cache's operators."""
import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs

pytestmark = pytest.mark.gpu


def _i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


def _bits(sa, want):
    return ((sa.STATUS_NO_PAGES if want["short"] else 0) | (sa.STATUS_BAD_LENGTH if want["long"] else 0)
            | (sa.STATUS_BAD_PAGE if want["bad"] else 0))


def _compare(sa, dev, new, lens, table, free, nfree, tokens):
    want = plain.plan_step(new, lens, table, free, nfree, tokens)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    for update in (False, True):
        t, f, held, left = _i32(table, dev), _i32(free, dev), _i32(lens, dev), _i32([nfree], dev)
        p = sa.plan_step(_i32(new, dev), held, t, f, left, tokens, update=update, workspace_buf=ws)
        assert sa.get_status(ws) == _bits(sa, want)
        for name in ("cu_seqlens", "start_pos", "seq_lens", "positions", "slots"):
            assert np.array_equal(getattr(p, name).cpu().numpy(), want[name]), name
        assert int(p.num_free) == want["num_free"] and np.array_equal(t.cpu().numpy(), want["block_table"])
        assert (p.seq_lens is held) == update and (p.num_free is left) == update
        if not update:
            assert np.array_equal(held.cpu().numpy(), np.asarray(lens)) and int(left) == nfree
    return want


def _pool(lens, cols, spare, seed):
    r = np.random.default_rng(seed)
    used = [-(-n // 16) for n in lens]
    perm = r.permutation(sum(used) + spare)
    table, at = np.full((len(lens), cols), -1), 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    free = np.zeros(len(perm), dtype=np.int64)
    free[:spare] = perm[at:]
    return table, free, spare


@pytest.mark.parametrize("B,new,held,extra", [(1, 1, 0, 0), (1, 1, 16, 3), (3, 40, 100, 0), (64, 1, 300, 5),
                                               (300, 20, 50, 1), (1500, 3, 40, 2), (5, 9000, 3, 7), (2, 30000, 17, 1)])
def test_plan(sa, cuda_dev, B, new, held, extra):
    r = np.random.default_rng(B + new)
    n, lens = r.integers(0 if B > 1 else new, new + 1, B), r.integers(0, held + 1, B)
    table, free, spare = _pool(lens, -(-(new + held) // 16) + 1, sum(n) // 16 + B, B)
    want = _compare(sa, cuda_dev, n, lens, table, free, spare, int(n.sum()) + extra)
    assert not (want["short"] or want["long"] or want["bad"])


def test_the_largest_batch(sa, cuda_dev):
    """8192 requests; in place, the most shared memory that the blocks of a cluster take."""
    r = np.random.default_rng(4)
    new, lens = r.integers(0, 12, 8192), r.integers(0, 40, 8192)
    table, free, spare = _pool(lens, 4, 8192, 5)
    want = _compare(sa, cuda_dev, new, lens, table, free, spare, int(new.sum()) + 9)
    assert not (want["short"] or want["long"] or want["bad"])
    done = r.random(8192) < 0.5
    want = plain.release_pages(done, want["seq_lens"], want["block_table"], free, want["num_free"])
    for update in (False, True):
        f, held, left, t = _i32(free, cuda_dev), _i32(lens, cuda_dev), _i32([spare], cuda_dev), _i32(table, cuda_dev)
        sa.plan_step(_i32(new, cuda_dev), held, t, f, left, int(new.sum()), update=True)
        held, left = sa.release_pages(torch.from_numpy(done).to(cuda_dev), held, t, f, left, update=update)
        assert np.array_equal(held.cpu().numpy(), want[0]) and np.array_equal(f.cpu().numpy(), want[1])
        assert int(left) == want[2] and sa.default_status() == 0


def test_no_requests_and_no_tokens(sa, cuda_dev):
    _compare(sa, cuda_dev, [0, 0], [5, 0], [[3], [-1]], [0, 1, 2, 3], 2, 0)
    _compare(sa, cuda_dev, [], [], np.zeros((0, 4)), [0, 1, 2], 2, 5)


def test_too_few_pages(sa, cuda_dev):
    """The first requests that need pages get them as far as they reach; one that needs none is served."""
    lens, new = [15, 16, 3, 30, 8], [20, 16, 4, 40, 2]
    table, free, _ = _pool(lens, 8, 3, 1)
    for nfree in range(4):
        want = _compare(sa, cuda_dev, new, lens, table, free, nfree, 90)
        assert want["short"] and want["seq_lens"][2] == 7 and want["seq_lens"][4] == 10


def test_lengths_that_do_not_fit(sa, cuda_dev):
    lens, new = [10, -3, 60, 20, 70000, 5], [3, 4, 8, -2, 1, 4]
    table, free, spare = _pool([10, 0, 60, 20, 0, 5], 4, 9, 2)
    _compare(sa, cuda_dev, new, lens, table, free, spare, 30)
    for tokens in (0, 2, 3, 14, 15, 16):  # rows for some of the requests alone
        _compare(sa, cuda_dev, [3, 0, 12, 5], [10, 4, 0, 20], table[[0, 1, 2, 3]], free, spare, tokens)


def test_pages_outside_the_pool(sa, cuda_dev):
    table, free, spare = _pool([10, 20], 6, 8, 3)
    free[spare - 1], table[1, 1] = 999, -7
    want = _compare(sa, cuda_dev, [20, 3], [10, 20], table, free, spare, 23)
    assert want["bad"]
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    for size, left in ((-3, 0), (99, len(free) - 1)):
        p = sa.plan_step(_i32([20, 3], cuda_dev), _i32([10, 20], cuda_dev), _i32(np.abs(table), cuda_dev), _i32(free, cuda_dev),
                         _i32([size], cuda_dev), 23, workspace_buf=ws)
        assert sa.get_status(ws) & sa.STATUS_BAD_LENGTH and int(p.num_free) == left


@pytest.mark.parametrize("B,held,share", [(1, 1, 1.0), (3, 100, 0.5), (64, 3000, 0.3), (1200, 60, 0.6), (4, 131072, 1.0)])
def test_release(sa, cuda_dev, B, held, share):
    r = np.random.default_rng(B)
    lens = r.integers(0, held + 1, B)
    lens[0] = held
    done = r.random(B) < share
    table, free, spare = _pool(lens, -(-held // 16) + 2, 5, B)
    want = plain.release_pages(done, lens, table, free, spare)
    for update in (False, True):
        f, l, n = _i32(free, cuda_dev), _i32(lens, cuda_dev), _i32([spare], cuda_dev)
        out, left = sa.release_pages(torch.from_numpy(done).to(cuda_dev), l, _i32(table, cuda_dev), f, n, update=update)
        assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(f.cpu().numpy(), want[1])
        assert int(left) == want[2] and (out is l) == update and (left is n) == update
    assert sa.default_status() == 0


def test_release_of_what_is_not_there(sa, cuda_dev):
    """A bad length releases nothing, a bad entry is reported, a list that would run over is cut."""
    d = cuda_dev
    ws = torch.zeros(256, dtype=torch.uint8, device=d)
    done, table = torch.ones(3, dtype=torch.bool, device=d), _i32([[4, 5], [6, 7], [2, 99]], d)
    free, n = _i32(np.arange(10), d), _i32([3], d)
    lens, left = sa.release_pages(done, _i32([20, -1, 40], d), table, free, n, workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_LENGTH
    assert lens.tolist() == [0, 0, 0] and int(left) == 5 and free.tolist()[:5] == [0, 1, 2, 5, 4]
    sa.release_pages(done, _i32([0, 0, 32], d), table, free, n, workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE
    lens, left = sa.release_pages(done, _i32([32, 32, 0], d), table, free, _i32([8], d), workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_LENGTH and int(left) == 10 and free.tolist()[8:] == [7, 6]


def test_release_undoes_a_plan(sa, cuda_dev):
    r = np.random.default_rng(9)
    new = r.integers(0, 900, 50)
    free = r.permutation(4000)
    f, n, lens = _i32(free, cuda_dev), _i32([4000], cuda_dev), _i32(np.zeros(50), cuda_dev)
    table = torch.full((50, 60), -1, dtype=torch.int32, device=cuda_dev)
    sa.plan_step(_i32(new, cuda_dev), lens, table, f, n, int(new.sum()), update=True)
    sa.release_pages(torch.ones(50, dtype=torch.bool, device=cuda_dev), lens, table, f, n, update=True)
    assert int(n) == 4000 and np.array_equal(f.cpu().numpy(), free) and not lens.any()


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 8), (128, 1, 4)])
def test_a_serving_run(sa, cuda_dev, D, Hkv, G):
    """Prompts, then decode steps captured once and replayed, then requests that end and others in
    their place: pages come from the plan, rows go by its slots, attention reads both; at the end the
    attention equals the fp64 form over the rows as the cache holds them."""
    dev, B, pages = cuda_dev, 5, 120
    g = torch.Generator().manual_seed(D)
    rows = lambda t, h: torch.randn(t, h, D, generator=g).to(torch.bfloat16)  # noqa: E731
    kv = torch.zeros(pages, Hkv, 2, 9, D, dtype=torch.uint8, device=dev)
    table = torch.full((B, 40), -1, dtype=torch.int32, device=dev)
    free, nfree = _i32(np.random.default_rng(1).permutation(pages), dev), _i32([pages], dev)
    lens = _i32(np.zeros(B), dev)
    history = [[torch.zeros(0, Hkv, D, dtype=torch.bfloat16)] * 2 for _ in range(B)]

    def held(b, i):
        x = history[b][i]
        codes, z, s = plain.coded_int4(x.double().numpy())
        return ((codes.reshape(*z.shape, 32) - z[..., None]) * s[..., None]).reshape(x.shape)

    def attend(q, b, n, fresh):
        """Output of the last n rows of request b over its history; fresh: these rows as they came, as a
        prefill attends its own."""
        k, v = held(b, 0), held(b, 1)
        if fresh:
            k, v = (np.concatenate([c[:-n], h[-n:].double().numpy()]) for c, h in zip((k, v), history[b]))
        L = len(k)
        out = np.zeros((n, Hkv * G, D))
        for h in range(Hkv * G):
            s = q[:, h].double().numpy() @ k[:, h // G].T * D ** -0.5
            s[np.arange(L)[None, :] > np.arange(L - n, L)[:, None]] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            out[:, h] = p @ v[:, h // G] / p.sum(1, keepdims=True)
        return out

    def prompt(new):
        T = sum(new)
        k, v, q = rows(T, Hkv), rows(T, Hkv), rows(T, Hkv * G)
        p = sa.plan_step(_i32(new, dev), lens, table, free, nfree, T, update=True)
        out, _ = sa.prefill_int4(q.to(dev), k.to(dev), v.to(dev), p.cu_seqlens, kv, table, p.start_pos)
        sa.append_kv_int4(k.to(dev), v.to(dev), p.slots, kv)
        t = 0
        for b, n in enumerate(new):
            if n:
                history[b] = [torch.cat([h, x[t:t + n]]) for h, x in zip(history[b], (k, v))]
                want = attend(q[t:t + n], b, n, True)
                assert np.abs(out[t:t + n].double().cpu().numpy() - want).max() <= 2.0 ** -8 * 5 + 2.0 ** -10 * 5, b
            t += n

    prompt([37, 1, 100, 0, 16])
    prompt([3, 20, 0, 50, 16])
    # a decode step: one token for each request, its rows in buffers that every replay reads anew
    ones = _i32(np.ones(B), dev)
    kb, vb, qb = (torch.zeros(B, h, D, dtype=torch.bfloat16, device=dev) for h in (Hkv, Hkv, Hkv * G))
    sa.default_status()

    def step():
        p = sa.plan_step(ones, lens, table, free, nfree, B + 2, update=True)
        sa.append_kv_int4(kb, vb, p.slots[:B], kv)
        return sa.decode_int4(qb, kv, table, p.seq_lens)[0]

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()

    def replay():
        k, v, q = rows(B, Hkv), rows(B, Hkv), rows(B, Hkv * G)
        for buf, x in ((kb, k), (vb, v), (qb, q)):
            buf.copy_(x)
        graph.replay()
        for b in range(B):
            history[b] = [torch.cat([h, x[b:b + 1]]) for h, x in zip(history[b], (k, v))]
        assert lens.tolist() == [len(h[0]) for h in history]
        for b in range(B):
            assert np.abs(out[b:b + 1].double().cpu().numpy() - attend(q[b:b + 1], b, 1, False)).max() <= 2.0 ** -8 * 5 + 2.0 ** -10 * 5

    for _ in range(20):
        replay()
    done = torch.tensor([False, True, False, True, True], device=dev)
    sa.release_pages(done, lens, table, free, nfree, update=True)
    for b in (1, 3, 4):
        history[b] = [torch.zeros(0, Hkv, D, dtype=torch.bfloat16)] * 2
    prompt([0, 90, 5, 33, 1])
    for _ in range(5):
        replay()
    used = sum(-(-len(h[0]) // 16) for h in history)
    assert int(nfree) == pages - used and sa.default_status() == 0


def test_refusals(sa, cuda_dev):
    d = cuda_dev
    new, lens, table, free, n = _i32([1, 2], d), _i32([0, 0], d), _i32([[0], [0]], d), _i32([0, 1], d), _i32([2], d)
    for bad in (dict(new=new[:1]), dict(lens=lens[:1]), dict(n=_i32([1, 1], d)), dict(free=free.long()), dict(table=table[0]),
                dict(table=table.cpu())):
        a = dict(dict(new=new, lens=lens, table=table, free=free, n=n), **bad)
        with pytest.raises((TypeError, ValueError)):
            sa.plan_step(a["new"], a["lens"], a["table"], a["free"], a["n"], 3)
    with pytest.raises(TypeError):
        sa.release_pages(new, lens, table, free, n)
    with pytest.raises(RuntimeError):
        sa.plan_step(new, lens, table, free, n, -1)
