"""Decode over an INT8 cache with a scale per page and KV head (sinkattn_decode_int8) on the GPU
against its fp64 form.

Tolerance of an output: one rounding to bf16 (half a step, 2^-8 of the value); the probabilities'
rounding to fp16 (2^-11 each at most, so 2^-11 of the largest |v| seen); and fp32 scores of up to
~100 accumulated over head_dim products (relative 2^-24 each: at most 1e-4 in the exponent), 2^-12 of
the largest |v|.  lse: the scores' 1e-4, held to the 1e-3 of the other decodes."""
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


def _dev(w, dev):
    c = w.cache
    return (w.q.to(dev), c.k_pages.to(dev), c.v_pages.to(dev), c.kv_scales.to(dev), c.block_table.to(dev), c.lens.to(dev),
            None if w.sinks is None else w.sinks.to(dev), w.scale)


def _ref(w, window=0):
    c = w.cache
    return plain.attend_int8(w.q, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens, w.sinks, w.scale, window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("sinks", [True, False])
def test_shapes(sa, cuda_dev, D, G, sinks):
    lens = [0, 1, 15, 16, 17, 33, 300, 1000, 2049]
    w = inputs.make_decode(lens, len(lens), 2 * G, 2, D, seed=G * 7 + D, sinks=sinks, kv_dtype="int8")
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=cuda_dev)
    out, lse = sa.decode_int8(*_dev(w, cuda_dev), workspace_buf=ws)
    check(out, lse, _ref(w))
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("D,G", [(64, 8), (64, 16), (128, 2), (128, 16)])
@pytest.mark.parametrize("window", [1, 16, 100, 1000, 5000])
def test_window(sa, cuda_dev, D, G, window):
    lens = [0, 1, 15, 16, 17, 100, 128, 129, 300, 2049, 9000]
    w = inputs.make_decode(lens, len(lens), 2 * G, 2, D, seed=window, kv_dtype="int8")
    out, lse = sa.decode_int8(*_dev(w, cuda_dev), window=window)
    check(out, lse, _ref(w, window))


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 8), (128, 1, 16), (64, 1, 1)])
def test_long_sequences_split_across_warps(sa, cuda_dev, D, Hkv, G):
    w = inputs.make_decode([40000, 70001, 5, 131072], 4, Hkv * G, Hkv, D, seed=D, kv_dtype="int8")
    a = _dev(w, cuda_dev)
    ref = _ref(w)
    for sms in (0, 7):
        out, lse = sa.decode_int8(*a, max_sms=sms)
        check(out, lse, ref)


def test_one_sequence_of_one_head_pair(sa, cuda_dev):
    w = inputs.make_decode([4097], 1, 1, 1, 64, seed=3, kv_dtype="int8")
    out, lse = sa.decode_int8(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))
    out, lse = sa.decode_int8(*_dev(w, cuda_dev), return_lse=False)
    assert lse is None
    check(out, None, _ref(w))


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_every_size(sa, cuda_dev, D):
    """Pages of zero scale, V scales from 2^-60 to 2^60 in one sequence, K scales that leave the
    scores in range; a page's V meets the others' in fp32 only."""
    w = inputs.make_decode([500, 64, 17], 3, 16, 2, D, seed=4, kv_dtype="int8")
    r = np.random.default_rng(0)
    sc = w.cache.kv_scales
    n = sc.shape[0]
    sc[:, :, 1] = torch.from_numpy(np.exp2(r.uniform(-60, 60, (n, 2))).astype(np.float32))
    sc[::5, :, 1] = 0.0
    sc[::3, :, 0] = 0.0
    sc[1::7, :, 0] *= 2.0 ** -40
    out, lse = sa.decode_int8(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e5, 1e20])
def test_queries_of_every_size(sa, cuda_dev, size):
    """q times `size` with the score scale divided by it: the same attention, far outside fp16."""
    w = inputs.make_decode([100, 33], 2, 16, 2, 64, seed=5, kv_dtype="int8")
    w.q = (w.q.double() * 2.0 ** round(np.log2(size))).to(torch.bfloat16)
    w.scale = w.scale / 2.0 ** round(np.log2(size))
    out, lse = sa.decode_int8(*_dev(w, cuda_dev))
    check(out, lse, _ref(w))


def test_a_non_finite_query_head_stays_alone(sa, cuda_dev):
    w = inputs.make_decode([100, 33], 2, 16, 2, 64, seed=6, kv_dtype="int8")
    ref = _ref(w)
    w.q[0, 3, 7], w.q[1, 9, 0] = float("nan"), float("inf")
    out, lse = sa.decode_int8(*_dev(w, cuda_dev))
    ok = np.ones((2, 16), dtype=bool)
    ok[0, 3] = ok[1, 9] = False
    check(out[torch.from_numpy(ok)], lse[torch.from_numpy(ok)], tuple(x[ok] for x in ref))


def test_a_cache_past_two_gigabytes(sa, cuda_dev):
    """Pages whose codes and offsets lie past 2^31."""
    npages, Hkv, D = 300000, 8, 64
    w = inputs.make_decode([37, 16, 200], 3, 64, Hkv, D, seed=7, kv_dtype="int8")
    c, dev = w.cache, cuda_dev
    ref = _ref(w)
    kp = torch.zeros(npages, Hkv, 16, D, dtype=torch.int8, device=dev)
    vp = torch.zeros_like(kp)
    sc = torch.full((npages, Hkv, 2), float("nan"), device=dev)
    at = npages - c.num_pages
    kp[at:], vp[at:], sc[at:] = c.k_pages.to(dev), c.v_pages.to(dev), c.kv_scales.to(dev)
    bt = torch.where(c.block_table >= 0, c.block_table + at, c.block_table).to(dev)
    out, lse = sa.decode_int8(w.q.to(dev), kp, vp, sc, bt, c.lens.to(dev), w.sinks.to(dev), w.scale)
    check(out, lse, ref)
    # and the append into those pages
    k, v = inputs.new_rows(3, Hkv, D, seed=1)
    got = [x[at:].cpu() for x in sa.append_kv_int8(k.to(dev), v.to(dev), torch.arange(4, dtype=torch.int32, device=dev), bt,
                                                   (c.lens - 1).to(dev), kp, vp, sc)]
    want = plain.append_kv_int8(k, v, [0, 1, 2, 3], c.block_table, c.lens - 1, c.k_pages, c.v_pages, c.kv_scales)
    assert np.array_equal(got[0].numpy(), want[0]) and np.array_equal(got[1].numpy(), want[1])
    assert np.array_equal(got[2].double().numpy(), want[2], equal_nan=True)


def test_bad_pages_and_lengths_set_the_status(sa, cuda_dev):
    w = inputs.make_decode([100, 40, 60], 3, 16, 2, 64, seed=8, kv_dtype="int8")
    ref = _ref(w)
    a = list(_dev(w, cuda_dev))
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=cuda_dev)
    a[4] = a[4].clone()
    a[4][1, 1] = w.cache.num_pages
    a[5] = a[5].clone()
    a[5][2] = -4
    out, lse = sa.decode_int8(*a, workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE | sa.STATUS_BAD_LENGTH
    check(out[:1], lse[:1], tuple(x[:1] for x in ref))
    out, lse = sa.decode_int8(*_dev(w, cuda_dev), workspace_buf=ws)
    check(out, lse, ref)
    assert sa.get_status(ws) == 0


def test_waits_that_run_out_report(sa, cuda_dev):
    w = inputs.make_decode([3000, 500], 2, 16, 2, 64, seed=9, kv_dtype="int8")
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=cuda_dev)
    a = _dev(w, cuda_dev)
    flush = torch.empty(512 << 20, dtype=torch.uint8, device=cuda_dev)
    st = 0
    for _ in range(20):  # the testing limit ends a wait whose copy from HBM is in flight: none of it in L2
        flush.zero_()
        sa.decode_int8(*a, workspace_buf=ws, wait_limit_us=1)
        st |= sa.get_status(ws)
        if st:
            break
    assert st == sa.STATUS_WAIT_TIMEOUT
    out, lse = sa.decode_int8(*_dev(w, cuda_dev), workspace_buf=ws)
    check(out, lse, _ref(w))
    assert sa.get_status(ws) == 0


def test_streams_and_graphs_do_not_share_scratch(sa, cuda_dev):
    """Two batches at once on two streams, and two graphs with different batches replayed at once,
    each many times: the same bits as alone."""
    ws = [inputs.make_decode([30000, 9000, 500], 3, 16, 2, 64, seed=20, kv_dtype="int8"),
          inputs.make_decode([7000, 21000, 12000, 1], 4, 16, 2, 64, seed=21, kv_dtype="int8")]
    args = [_dev(w, cuda_dev) for w in ws]
    alone = [sa.decode_int8(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(20):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(sa.decode_int8(*a))
        torch.cuda.synchronize()
        for (o, l), (p, m) in zip(got, alone):
            assert torch.equal(o, p) and torch.equal(l, m)
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sa.decode_int8(*a))
        graphs.append(g)
    big = inputs.make_decode([2000] * 40, 40, 16, 2, 64, seed=22, kv_dtype="int8")  # a larger eager workspace
    sa.decode_int8(*_dev(big, cuda_dev))
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


def test_refusals(sa, cuda_dev):
    w = inputs.make_decode([30], 1, 8, 2, 64, seed=2, kv_dtype="int8")
    q, kp, vp, sc, bt, ln, sk, scale = _dev(w, cuda_dev)
    for bad in (dict(k=kp.view(torch.uint8)), dict(sc=sc[:, :, :1].contiguous()), dict(sc=sc.double()), dict(v=vp[:-1])):
        with pytest.raises((TypeError, ValueError)):
            sa.decode_int8(q, bad.get("k", kp), bad.get("v", vp), bad.get("sc", sc), bt, ln, sk, scale)
    with pytest.raises(ValueError):
        sa.decode_int8(q, kp, vp, sc, bt, ln, sk, scale, out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device=cuda_dev))
    with pytest.raises(sa.SinkAttnError, match="workspace"):
        sa.decode_int8(q, kp, vp, sc, bt, ln, sk, scale, workspace_buf=torch.zeros(256, dtype=torch.uint8, device=cuda_dev))
