"""The 4-bit cache on the GPU: append and unpack bit for bit their fp64 forms, decode and chunked
prefill against theirs.

Tolerance of an attention output: one rounding to bf16 (half a step, 2^-8 of the value); the
probabilities' rounding to fp16 (2^-11 each at most, so 2^-11 of the largest |v| seen); and fp32
scores of up to ~100 accumulated over head_dim products (relative 2^-24 each: at most 1e-4 in the
exponent), 2^-12 of the largest |v|.  lse: the scores' 1e-4, held to the 1e-3 of the other decodes."""
import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs
from tolerances import check_lse

pytestmark = pytest.mark.gpu


def check(out, lse, ref):
    ro, rl, vmax = ref
    g = out.detach().double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -12) * vmax[..., None]
    err = np.abs(g - ro)
    assert np.all(np.isfinite(g)) and np.all(err <= bound), f"worst {np.max(err - bound):.3e} over its bound"
    if lse is not None:
        check_lse(lse, rl)


# ------------------------------------------------------------------ append, unpack
def _rows(shape, seed, spread=2.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape) * np.exp(r.uniform(-spread, spread, shape[:-1] + (1,))) + r.standard_normal(shape[-1])
    return torch.from_numpy(x).to(torch.bfloat16)


def _random_cache(n, H, D, seed):
    return inputs.pack_int4(_rows((n, H, 16, D), seed), _rows((n, H, 16, D), seed + 1))


@pytest.mark.parametrize("D,H,T", [(64, 1, 1), (64, 8, 7), (64, 2, 100), (128, 1, 9), (128, 4, 33)])
def test_append_bits(sa, cuda_dev, D, H, T):
    n = T // 8 + 3
    r = np.random.default_rng(T)
    slots = torch.from_numpy(r.permutation(n * 16)[:T].astype(np.int64))
    slots[r.random(T) < 0.1] = -1
    wide = _rows((T, 2 * H + 3, D), T, 10.0)  # K and V inside a wider row
    k, v = wide[:, :H], wide[:, H + 1:2 * H + 1]
    kv = _random_cache(n, H, D, T)
    want = plain.append_kv_int4(k, v, slots, kv)
    w = wide.to(cuda_dev)
    got = kv.to(cuda_dev)
    assert sa.append_kv_int4(w[:, :H], w[:, H + 1:2 * H + 1], slots.to(cuda_dev), got) is got
    assert np.array_equal(got.cpu().numpy(), want)
    assert sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_append_of_hard_rows(sa, cuda_dev, D):
    """Ties, zeros, one-signed groups, the ends of bf16's range, scales at the floor, infinities, NaN."""
    rows = [np.zeros(D), np.full(D, -3.0), np.full(D, 5.0), np.arange(D) * 0.5 - 8.0, np.arange(D) % 16 + 0.5,
            np.where(np.arange(D) % 2, 3.38e38, -3.38e38), np.where(np.arange(D) % 3, 1e-30, -2e-30), np.full(D, 1e-38),
            np.where(np.arange(D) == 5, 1e30, 1.0), np.linspace(-7.5, 7.5, D), np.arange(D) * 0.25 - 4]
    x = torch.from_numpy(np.array(rows)).to(torch.bfloat16)[:, None]
    bad = x[:4].clone()
    bad[0, 0, 3], bad[1, 0, 40], bad[2, 0, 0], bad[3, 0, 9] = float("nan"), float("inf"), float("-inf"), float("nan")
    kv = _random_cache(2, 1, D, 5)
    for rows, status in ((x, 0), (bad, sa.STATUS_VALUE_RANGE)):
        T = rows.shape[0]
        slots = torch.arange(3, 3 + T)
        got = sa.append_kv_int4(rows.to(cuda_dev), -rows.to(cuda_dev), slots.to(cuda_dev), kv.to(cuda_dev))
        assert np.array_equal(got.cpu().numpy(), plain.append_kv_int4(rows, -rows, slots, kv))
        assert sa.default_status() == status


def test_slots_outside_the_pool(sa, cuda_dev):
    kv = _random_cache(3, 2, 64, 6)
    k = _rows((4, 2, 64), 7)
    slots = torch.tensor([-5, 48, 2 ** 40, 47])
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    got = sa.append_kv_int4(k.to(cuda_dev), k.to(cuda_dev), slots.to(cuda_dev), kv.to(cuda_dev), workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE
    assert np.array_equal(got.cpu().numpy(), plain.append_kv_int4(k, k, slots, kv))


@pytest.mark.parametrize("D,H,n", [(64, 1, 1), (64, 8, 5), (128, 2, 7)])
def test_unpack_bits(sa, cuda_dev, D, H, n):
    kv = _random_cache(n, H, D, n)
    want = plain.values_int4(kv)
    for g, w in zip(sa.unpack_kv_int4(kv.to(cuda_dev)), want):
        assert np.array_equal(g.double().cpu().numpy(), w)
    pages = torch.tensor([n - 1, 0, n, -1, 0], dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    got = sa.unpack_kv_int4(kv.to(cuda_dev), pages.to(cuda_dev), workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE
    for g, w in zip(got, want):
        g = g.double().cpu().numpy()
        assert np.array_equal(g[[0, 1, 4]], w[[n - 1, 0, 0]]) and not g[2:4].any()


# ------------------------------------------------------------------ decode
def _dev(w, dev):
    c = w.cache
    return (w.q.to(dev), inputs.pack_int4(c.k_pages, c.v_pages).to(dev), c.block_table.to(dev), c.lens.to(dev),
            None if w.sinks is None else w.sinks.to(dev), w.scale)


def _ref(w, window=0):
    c = w.cache
    return plain.attend_int4(w.q, inputs.pack_int4(c.k_pages, c.v_pages), c.block_table, c.lens, w.sinks, w.scale, window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("sinks", [True, False])
def test_decode_shapes(sa, cuda_dev, D, G, sinks):
    lens = [0, 1, 15, 16, 17, 33, 300, 1000, 2049]
    w = inputs.make_decode(lens, len(lens), 2 * G, 2, D, seed=G * 7 + D, sinks=sinks)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=cuda_dev)
    out, lse = sa.decode_int4(*_dev(w, cuda_dev), workspace_buf=ws)
    check(out, lse, _ref(w))
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("D,G", [(64, 8), (64, 16), (128, 2), (128, 16)])
@pytest.mark.parametrize("window", [1, 16, 100, 1000, 5000])
def test_decode_window(sa, cuda_dev, D, G, window):
    lens = [0, 1, 15, 16, 17, 100, 128, 129, 300, 2049, 9000]
    w = inputs.make_decode(lens, len(lens), 2 * G, 2, D, seed=window)
    out, lse = sa.decode_int4(*_dev(w, cuda_dev), window=window)
    check(out, lse, _ref(w, window))


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 8), (128, 1, 16), (64, 1, 1)])
def test_long_sequences_split_across_warps(sa, cuda_dev, D, Hkv, G):
    w = inputs.make_decode([40000, 70001, 5, 131072], 4, Hkv * G, Hkv, D, seed=D)
    a, ref = _dev(w, cuda_dev), _ref(w)
    for sms in (0, 7):
        out, lse = sa.decode_int4(*a, max_sms=sms)
        check(out, lse, ref)
    out, lse = sa.decode_int4(*a, return_lse=False)
    assert lse is None


def _scaled(kv, D, f):
    """The cache with each group's scale times f(shape), powers of two (0 allowed)."""
    n, H = kv.shape[:2]
    words = kv[:, :, :, 8].contiguous().view(torch.int16).to(torch.int32) & 0xFFFF
    s = ((words & 0xFFF0) << 16).view(torch.float32) * torch.from_numpy(f((n, H, 2, D // 2)).astype(np.float32))
    words = (s.view(torch.int32) >> 16) & 0xFFF0 | words & 15
    out = kv.clone()
    out[:, :, :, 8] = words.to(torch.int16).view(torch.uint8)
    return out


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_every_size(sa, cuda_dev, D):
    """Groups of zero scale, V scales from 2^-60 to 2^60 in one sequence, small K scales."""
    w = inputs.make_decode([500, 64, 17], 3, 16, 2, D, seed=4, poison=False)
    r = np.random.default_rng(0)

    def f(shape):
        e = np.exp2(np.round(r.uniform(-60, 60, shape)))
        e[:, :, 0] = np.where(r.random(shape)[:, :, 0] < 0.2, 2.0 ** -40, 1.0)
        e[r.random(shape) < 0.1] = 0.0
        return e
    c = w.cache
    kv = _scaled(inputs.pack_int4(c.k_pages, c.v_pages), D, f)
    ref = plain.attend_int4(w.q, kv, c.block_table, c.lens, w.sinks, w.scale)
    a = list(_dev(w, cuda_dev))
    a[1] = kv.to(cuda_dev)
    out, lse = sa.decode_int4(*a)
    check(out, lse, ref)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e5, 1e20])
def test_queries_of_every_size(sa, cuda_dev, size):
    w = inputs.make_decode([100, 33], 2, 16, 2, 64, seed=5)
    w.q = (w.q.double() * 2.0 ** round(np.log2(size))).to(torch.bfloat16)
    w.scale = w.scale / 2.0 ** round(np.log2(size))
    out, lse = sa.decode_int4(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))


@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_score_scales(sa, cuda_dev, scale):
    w = inputs.make_decode([100, 33, 2], 3, 16, 2, 64, seed=15)
    w.scale = scale
    out, lse = sa.decode_int4(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))


def test_rising_scores(sa, cuda_dev):
    """Scores that grow along the sequence move the running maximum again and again."""
    w = inputs.make_decode([3000], 1, 8, 1, 64, seed=16, poison=False)
    c = w.cache
    order = c.block_table[0].long()
    c.k_pages[order] = c.k_pages[order] * torch.linspace(0.1, 6.0, len(order))[:, None, None, None].to(torch.bfloat16)
    out, lse = sa.decode_int4(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))


def test_a_non_finite_query_head_stays_alone(sa, cuda_dev):
    w = inputs.make_decode([100, 33], 2, 16, 2, 64, seed=6)
    ref = _ref(w)
    w.q[0, 3, 7], w.q[1, 9, 0] = float("nan"), float("inf")
    out, lse = sa.decode_int4(*_dev(w, cuda_dev))
    ok = np.ones((2, 16), dtype=bool)
    ok[0, 3] = ok[1, 9] = False
    check(out[torch.from_numpy(ok)], lse[torch.from_numpy(ok)], tuple(x[ok] for x in ref))


def test_a_cache_past_two_gigabytes(sa, cuda_dev):
    """Pages whose records lie past 2^31, and slots into them."""
    npages, Hkv, D = 300000, 8, 64
    w = inputs.make_decode([37, 16, 200], 3, 64, Hkv, D, seed=7)
    c, dev = w.cache, cuda_dev
    kv = inputs.pack_int4(c.k_pages, c.v_pages)
    ref = _ref(w)
    big = torch.full((npages, Hkv, 2, 9, D), 255, dtype=torch.uint8, device=dev)
    at = npages - c.num_pages
    big[at:] = kv.to(dev)
    bt = torch.where(c.block_table >= 0, c.block_table + at, c.block_table).to(dev)
    out, lse = sa.decode_int4(w.q.to(dev), big, bt, c.lens.to(dev), w.sinks.to(dev), w.scale)
    check(out, lse, ref)
    k, v = inputs.new_rows(3, Hkv, D, seed=1)
    slots = torch.tensor([c.num_pages * 16 - 1, 5, 20]) + 16 * at
    sa.append_kv_int4(k.to(dev), v.to(dev), slots.to(dev), big)
    assert np.array_equal(big[at:].cpu().numpy(), plain.append_kv_int4(k, v, slots - 16 * at, kv))
    assert bool((big[:at] == 255).all())
    pages = torch.arange(at, npages, dtype=torch.int32, device=dev)
    keep = torch.isfinite(sa.unpack_kv_int4(big, pages)[0].float())
    assert torch.equal(torch.isfinite(sa.unpack_kv_int4(big[at:].contiguous())[0].float()), keep)


@pytest.mark.parametrize("G", [2, 16])
def test_nothing_to_see(sa, cuda_dev, G):
    """No token in any sequence: the sink alone, or nothing; an empty batch."""
    w = inputs.make_decode([0, 0, 0], 3, G, 1, 64, seed=17)
    a = list(_dev(w, cuda_dev))
    out, lse = sa.decode_int4(*a)
    assert not out.any() and torch.equal(lse, a[4].expand(3, G))
    a[4] = None
    out, lse = sa.decode_int4(*a)
    assert not out.any() and bool((lse == -float("inf")).all())
    out, lse = sa.decode_int4(a[0][:0], a[1], a[2][:0], a[3][:0])
    assert out.shape == (0, G, 64) and lse.shape == (0, G)


def test_many_sequences(sa, cuda_dev):
    """More sequences than a block has threads, most of a page or less."""
    lens = np.random.default_rng(2).integers(0, 40, 900).tolist()
    w = inputs.make_decode(lens, len(lens), 8, 2, 64, seed=18)
    out, lse = sa.decode_int4(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))


def test_the_same_page_for_several_sequences(sa, cuda_dev):
    """A shared prefix: rows of the block table that name the same pages."""
    w = inputs.make_decode([600, 640, 64], 3, 8, 1, 128, seed=19, poison=False)
    w.cache.block_table[1, :30] = w.cache.block_table[0, :30]
    w.cache.block_table[2, :4] = w.cache.block_table[0, :4]
    out, lse = sa.decode_int4(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))


def test_bad_pages_and_lengths_set_the_status(sa, cuda_dev):
    w = inputs.make_decode([100, 40, 60], 3, 16, 2, 64, seed=8)
    ref = _ref(w)
    a = list(_dev(w, cuda_dev))
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=cuda_dev)
    a[2] = a[2].clone()
    a[2][1, 1] = w.cache.num_pages
    a[3] = a[3].clone()
    a[3][2] = -4
    out, lse = sa.decode_int4(*a, workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE | sa.STATUS_BAD_LENGTH
    check(out[:1], lse[:1], tuple(x[:1] for x in ref))
    out, lse = sa.decode_int4(*_dev(w, cuda_dev), workspace_buf=ws)
    check(out, lse, ref)
    assert sa.get_status(ws) == 0


def test_waits_that_run_out_report(sa, cuda_dev):
    w = inputs.make_decode([3000, 500], 2, 16, 2, 64, seed=9)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=cuda_dev)
    a = _dev(w, cuda_dev)
    flush = torch.empty(512 << 20, dtype=torch.uint8, device=cuda_dev)
    st = 0
    for _ in range(20):  # the testing limit ends a wait whose copy from HBM is in flight: none of it in L2
        flush.zero_()
        sa.decode_int4(*a, workspace_buf=ws, wait_limit_us=1)
        st |= sa.get_status(ws)
        if st:
            break
    assert st == sa.STATUS_WAIT_TIMEOUT
    out, lse = sa.decode_int4(*a, workspace_buf=ws)
    check(out, lse, _ref(w))
    assert sa.get_status(ws) == 0


def test_streams_and_graphs_do_not_share_scratch(sa, cuda_dev):
    """Two batches at once on two streams, and two graphs with different batches replayed at once,
    each many times: the same bits as alone."""
    ws = [inputs.make_decode([30000, 9000, 500], 3, 16, 2, 64, seed=20),
          inputs.make_decode([7000, 21000, 12000, 1], 4, 16, 2, 64, seed=21)]
    args = [_dev(w, cuda_dev) for w in ws]
    alone = [sa.decode_int4(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(20):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(sa.decode_int4(*a))
        torch.cuda.synchronize()
        for (o, l), (p, m) in zip(got, alone):
            assert torch.equal(o, p) and torch.equal(l, m)
    sa.default_status()
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sa.decode_int4(*a))
        graphs.append(g)
    for _ in range(20):
        for o, l in outs:
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, l), (p, m) in zip(outs, alone):
            assert torch.equal(o, p) and torch.equal(l, m)


# ------------------------------------------------------------------ prefill
def _pre(p, dev, kv=None):
    c = p.prefix
    kv = inputs.pack_int4(c.k_pages, c.v_pages) if kv is None else kv
    return (p.q.to(dev), p.k.to(dev), p.v.to(dev), p.cu_seqlens.to(dev), kv.to(dev), c.block_table.to(dev), c.lens.to(dev),
            None if p.sinks is None else p.sinks.to(dev), p.scale)


def _pre_ref(p, window=0, kv=None):
    c = p.prefix
    kv = inputs.pack_int4(c.k_pages, c.v_pages) if kv is None else kv
    return plain.attend_int4(p.q, kv, c.block_table, c.lens, p.sinks, p.scale, window, (p.k, p.v, p.cu_seqlens))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 8, 16])
@pytest.mark.parametrize("window", [0, 70])
def test_prefill_shapes(sa, cuda_dev, D, G, window):
    p = inputs.make_prefill([130, 1, 0, 17, 60], G, 1, D, seed=D + G, sinks=G > 1, prefix_lens=[20, 300, 5, 0, 1001])
    out, lse = sa.prefill_int4(*_pre(p, cuda_dev), window=window)
    check(out, lse, _pre_ref(p, window))
    assert sa.default_status() == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 64, 8), (128, 16, 8)])
@pytest.mark.parametrize("pre", [1003, 4000])
def test_prefill_split(sa, cuda_dev, D, Hq, Hkv, pre):
    """One short chunk over a long prefix, its key tiles split over the SMs, and whole in 256 bytes."""
    p = inputs.make_prefill([17], Hq, Hkv, D, seed=pre, prefix_lens=[pre])
    ref, a = _pre_ref(p), _pre(p, cuda_dev)
    check(*sa.prefill_int4(*a), ref)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    check(*sa.prefill_int4(*a, workspace_buf=ws), ref)
    check(*sa.prefill_int4(*a, max_sms=3), ref)
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("pre", [[300, 20], [2000, 0]])
def test_prefill_leaves_the_rows_behind(sa, cuda_dev, pre):
    """Rows behind the last request stay as they were, whole and in parts; what the pages and the padding
    hold there does not matter."""
    p = inputs.make_prefill([9, 5, 6], 8, 1, 64, seed=21, prefix_lens=pre + [40])
    a = list(_pre(p, cuda_dev))
    ref = _pre_ref(p)
    a[3] = a[3][:3].contiguous()  # two requests; the third's rows are padding
    for i in (0, 1, 2):
        a[i][14:] = float("nan")
    a[5], a[6] = a[5][:2].contiguous(), a[6][:2].contiguous()
    out = torch.full_like(a[0], 7.0)
    lse = torch.full((20, 8), 5.0, device=cuda_dev)
    sa.prefill_int4(*a, out=out, lse=lse)
    check(out[:14], lse[:14], tuple(x[:14] for x in ref))
    assert bool((out[14:] == 7.0).all()) and bool((lse[14:] == 5.0).all())


def test_prefill_of_many_requests(sa, cuda_dev):
    r = np.random.default_rng(3)
    new, pre = r.integers(0, 40, 90).tolist(), r.integers(0, 200, 90).tolist()
    p = inputs.make_prefill(new, 8, 2, 64, seed=11, prefix_lens=pre)
    check(*sa.prefill_int4(*_pre(p, cuda_dev)), _pre_ref(p))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("top", [-9, 0, 12, 17])
def test_prefill_scales(sa, cuda_dev, D, top):
    """V scales up to 2^top, groups of zero scale; K scales small enough for the scores."""
    p = inputs.make_prefill([40, 9], 8, 1, D, seed=12, prefix_lens=[700, 130], poison=False)
    c = p.prefix
    r = np.random.default_rng(top + 20)
    p.v = (p.v.double() * 2.0 ** top).to(torch.bfloat16)
    c.v_pages = torch.from_numpy(c.v_pages.double().numpy() * 2.0 ** top / 2).to(torch.bfloat16)

    def f(shape):
        e = np.exp2(np.round(r.uniform(-6, 0, shape)))
        e[:, :, 0] = 1.0
        e[r.random(shape) < 0.1] = 0.0
        return e
    kv = _scaled(inputs.pack_int4(c.k_pages, c.v_pages), D, f)
    out, lse = sa.prefill_int4(*_pre(p, cuda_dev, kv))
    check(out, lse, _pre_ref(p, kv=kv))
    assert sa.default_status() == 0


def test_prefill_reports_scales_out_of_range(sa, cuda_dev):
    p = inputs.make_prefill([20], 8, 1, 64, seed=13, prefix_lens=[100], poison=False)
    c = p.prefix
    kv = _scaled(inputs.pack_int4(c.k_pages, c.v_pages), 64, lambda s: np.full(s, 2.0 ** 24))
    sa.default_status()
    sa.prefill_int4(*_pre(p, cuda_dev, kv))
    assert sa.default_status() == sa.STATUS_VALUE_RANGE


def test_prefill_bad_pages_and_waits(sa, cuda_dev):
    p = inputs.make_prefill([30, 40], 8, 2, 64, seed=14, prefix_lens=[200, 90])
    ref, a = _pre_ref(p), list(_pre(p, cuda_dev))
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    a[5] = a[5].clone()
    a[5][1, 2] = p.prefix.num_pages + 7
    out, lse = sa.prefill_int4(*a, workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE
    check(out[:30], lse[:30], tuple(x[:30] for x in ref))
    assert bool(torch.isfinite(out.float()).all())
    sa.prefill_int4(*_pre(p, cuda_dev), workspace_buf=ws, wait_limit_us=1)
    assert sa.get_status(ws) == sa.STATUS_WAIT_TIMEOUT
    ws.zero_()  # a call that gave up leaves the counters behind
    check(*sa.prefill_int4(*_pre(p, cuda_dev), workspace_buf=ws), ref)


def test_refusals(sa, cuda_dev):
    w = inputs.make_decode([30], 1, 8, 2, 64, seed=2)
    q, kv, bt, ln, sk, scale = _dev(w, cuda_dev)
    for bad in (kv.view(torch.int8), kv[:, :, :1], kv[:, :, :, :8].contiguous(), kv[0], kv.cpu(),
                torch.zeros(2, 2, 2, 9, 128, dtype=torch.uint8, device=cuda_dev)):
        with pytest.raises((TypeError, ValueError)):
            sa.decode_int4(q, bad, bt, ln, sk, scale)
        with pytest.raises((TypeError, ValueError)):
            sa.append_kv_int4(q[:, :2], q[:, :2], torch.zeros(1, dtype=torch.int64, device=cuda_dev), bad)
    with pytest.raises(TypeError):
        sa.append_kv_int4(q[:, :2], q[:, :2], ln, kv)
    with pytest.raises(ValueError):
        sa.decode_int4(q, kv, bt, ln, sk, scale, out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device=cuda_dev))
    with pytest.raises(sa.SinkAttnError, match="workspace"):
        sa.decode_int4(q, kv, bt, ln, sk, scale, workspace_buf=torch.zeros(256, dtype=torch.uint8, device=cuda_dev))
    with pytest.raises(ValueError):
        sa.unpack_kv_int4(kv, k_out=torch.empty(1, 2, 16, 64, dtype=torch.bfloat16, device=cuda_dev))
