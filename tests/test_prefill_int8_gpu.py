"""Chunked prefill over an INT8 prefix (sinkattn_prefill_int8) on the GPU against its fp64 form, and a
serving run of the INT8 operators together.

Tolerance of an output: one rounding to bf16 (2^-8 of the value); P rounded to fp16 (2^-11 each, and
2^-25 for each of n keys where P is below fp16's normals) and fp32 scores (1e-4 in the exponent, 2^-12),
both of the largest |v| seen.  lse as for the decodes."""
import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs
from tolerances import check_lse

pytestmark = pytest.mark.gpu


def check(out, lse, ref, keys):
    ro, rl, vmax = ref
    g = out.detach().double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -12 + keys * 2.0 ** -25) * vmax[..., None]
    err = np.abs(g - ro)
    assert np.all(np.isfinite(g)) and np.all(err <= bound), f"worst {np.max(err - bound):.3e} over its bound"
    if lse is not None:
        check_lse(lse, rl)


def _args(p, dev):
    c = p.prefix
    return (p.q.to(dev), p.k.to(dev), p.v.to(dev), p.cu_seqlens.to(dev), c.k_pages.to(dev), c.v_pages.to(dev),
            c.kv_scales.to(dev), c.block_table.to(dev), c.lens.to(dev), None if p.sinks is None else p.sinks.to(dev),
            p.scale)


def _ref(p, window=0):
    c = p.prefix
    return plain.attend_int8(p.q, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens, p.sinks, p.scale, window,
                             new=(p.k, p.v, p.cu_seqlens))


def _make(new, pre, Hq, Hkv, D, seed, sinks=True):
    return inputs.make_prefill(new, Hq, Hkv, D, seed=seed, sinks=sinks, prefix_lens=pre, prefix_kv_dtype="int8")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("sinks", [True, False])
def test_shapes(sa, cuda_dev, D, G, sinks):
    new, pre = [1, 0, 17, 128, 129, 200, 5], [0, 30, 15, 128, 129, 500, 1]
    p = _make(new, pre, 2 * G, 2, D, seed=G + D, sinks=sinks)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    out, lse = sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws)
    check(out, lse, _ref(p), 700)
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 8), (128, 2, 2), (64, 1, 1)])
@pytest.mark.parametrize("window", [1, 16, 100, 128, 1000])
def test_window(sa, cuda_dev, D, Hkv, G, window):
    p = _make([1, 130, 300, 64], [0, 50, 1111, 2000], Hkv * G, Hkv, D, seed=window)
    out, lse = sa.prefill_int8(*_args(p, cuda_dev), window=window)
    check(out, lse, _ref(p, window), 2200)


def test_long_prefix_on_few_sms(sa, cuda_dev):
    p = _make([300, 33], [9000, 16384], 8, 1, 64, seed=3)
    ref = _ref(p)
    got = [sa.prefill_int8(*_args(p, cuda_dev), max_sms=m) for m in (0, 3)]
    for out, lse in got:
        check(out, lse, ref, 17000)
    assert torch.equal(got[0][0], got[1][0])
    out, none = sa.prefill_int8(*_args(p, cuda_dev), return_lse=False)
    assert none is None and torch.equal(out, got[0][0])


@pytest.mark.parametrize("n", [1, 200, 256, 257, 1030])
def test_many_requests(sa, cuda_dev, n):
    """Requests in the order of their length (up to 256 of them) and as they come; equal ones, ones
    without a prefix, empty ones."""
    r = np.random.default_rng(n)
    new, pre = r.integers(0, 4, n).tolist(), (r.integers(0, 40, n) * r.integers(0, 2, n)).tolist()
    new[0], new[n // 2] = 200, 140
    p = _make(new, pre, 2, 1, 64, seed=n)
    out, lse = sa.prefill_int8(*_args(p, cuda_dev))
    check(out, lse, _ref(p), 300)


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_every_size(sa, cuda_dev, D):
    """V scales from 2^-30 to 2^14 page by page, zero scales of K and V, K scales far below the rest."""
    p = _make([200, 16], [777, 40], 16, 2, D, seed=4)
    r = np.random.default_rng(0)
    sc = p.prefix.kv_scales
    n = sc.shape[0]
    sc[:, :, 1] = torch.from_numpy(np.exp2(r.uniform(-30, 14, (n, 2))).astype(np.float32))
    sc[::5, :, 1] = 0.0
    sc[::3, :, 0] = 0.0
    sc[1::7, :, 0] *= 2.0 ** -40
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    out, lse = sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws)
    check(out, lse, _ref(p), 1000)
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("e", [-24, -14, -1, 8, 14])
def test_all_v_scales_alike(sa, cuda_dev, e):
    """Nothing larger beside them: V scales at the ends of their exact range, new V rows of their size."""
    p = _make([100], [300], 16, 2, 64, seed=5)
    m = torch.from_numpy(1 + np.random.default_rng(1).random(p.prefix.kv_scales.shape[:2]).astype(np.float32))
    p.prefix.kv_scales[:, :, 1] = m * 2.0 ** e
    p.v = torch.zeros_like(p.v) if e < -14 else (p.v.double() * 2.0 ** (e + 5)).to(torch.bfloat16)
    out, lse = sa.prefill_int8(*_args(p, cuda_dev))
    check(out, lse, _ref(p), 400)


def test_a_v_scale_out_of_range_is_reported(sa, cuda_dev):
    p = _make([20], [60], 8, 2, 64, seed=6)
    p.prefix.kv_scales[p.prefix.block_table[0, 1], 1, 1] = 2.0 ** 15
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_VALUE_RANGE


def test_growing_scores(sa, cuda_dev):
    """Each later prefix tile's scores far above the tiles before: the running maximum moves every tile."""
    p = _make([130], [1500], 8, 1, 64, seed=7)
    c = p.prefix
    at = c.block_table[0, :94].long()
    c.kv_scales[at, :, 0] *= torch.linspace(0.05, 3.0, 94)[:, None]
    out, lse = sa.prefill_int8(*_args(p, cuda_dev))
    check(out, lse, _ref(p), 1700)


def test_bad_pages_set_the_status_and_rows_behind_the_last_request_stay(sa, cuda_dev):
    p = _make([40, 30], [100, 200], 8, 2, 64, seed=8)
    ref = _ref(p)
    a = list(_args(p, cuda_dev))
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    bad = a[7].clone()
    bad[1, 3] = -7
    bad[1, 4] = p.prefix.num_pages
    out, lse = sa.prefill_int8(*a[:7], bad, *a[8:], workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE
    check(out[:40], lse[:40], tuple(x[:40] for x in ref), 300)
    # a padded step: 9 more rows than the requests hold
    pad = lambda x: torch.cat([x, x[:9]])  # noqa: E731
    out = torch.full((79, 8, 64), 42.0, dtype=torch.bfloat16, device=cuda_dev)
    lse = torch.full((79, 8), 42.0, device=cuda_dev)
    sa.prefill_int8(pad(a[0]), pad(a[1]), pad(a[2]), *a[3:], out=out, lse=lse, workspace_buf=ws)
    check(out[:70], lse[:70], ref, 300)
    assert torch.all(out[70:] == 42.0) and torch.all(lse[70:] == 42.0)


def test_waits_that_run_out_report(sa, cuda_dev):
    p = _make([512, 300], [1000, 37], 16, 2, 64, seed=9)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    st = 0
    for _ in range(20):
        sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws, wait_limit_us=1)
        st |= sa.get_status(ws)
        if st:
            break
    assert st == sa.STATUS_WAIT_TIMEOUT
    out, lse = sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws)
    check(out, lse, _ref(p), 1600)
    assert sa.get_status(ws) == 0


def test_streams_and_graphs_do_not_share_scratch(sa, cuda_dev):
    ps = [_make([300, 20], [900, 3000], 16, 2, 64, seed=20), _make([64, 500], [2500, 0], 8, 2, 128, seed=21)]
    args = [_args(p, cuda_dev) for p in ps]
    alone = [sa.prefill_int8(*a) for a in args]
    torch.cuda.synchronize()
    for a, p, got in zip(args, ps, alone):
        check(*got, _ref(p), 3100)
    streams = [torch.cuda.Stream() for _ in args]
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sa.prefill_int8(*a))
        graphs.append(g)
    for use_graph in (False, True):
        for _ in range(10):
            got = []
            torch.cuda.synchronize()
            for s, g, a, o in zip(streams, graphs, args, outs):
                with torch.cuda.stream(s):
                    if use_graph:
                        g.replay()
                        got.append(o)
                    else:
                        got.append(sa.prefill_int8(*a))
            torch.cuda.synchronize()
            for (o, l), (q, m) in zip(got, alone):
                assert torch.equal(o, q) and torch.equal(l, m)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 2), (128, 16, 4)])
def test_a_serving_run(sa, cuda_dev, D, Hq, Hkv):
    """Two chunks of a prompt and then tokens, as a layer serves them: projection rows -> norm and
    rotation -> chunked prefill over the INT8 pages and append into them -> decode.  Each attention
    against fp64 over the cache as it then stands, the cache bit for bit at every step."""
    dev, r = cuda_dev, dict(base=10000.0, rotary_dim=D // 2, factor=4.0, scaling="linear", interleaved=True)
    n, pages = 3, 40
    rng = np.random.default_rng(D)
    bt = torch.from_numpy(rng.permutation(pages)[:n * 12].reshape(n, 12).astype(np.int32))
    wq, wk = (torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
    sinks = torch.from_numpy(rng.standard_normal(Hq).astype(np.float32))
    kp, vp = (torch.randint(-127, 128, (pages, Hkv, 16, D), dtype=torch.int8) for _ in range(2))  # left by others
    sc = torch.rand(pages, Hkv, 2)
    state = [x.to(dev) for x in (kp, vp, sc)]
    ref = (kp.numpy(), vp.numpy(), sc.double().numpy())
    lens, rot = [0] * n, sa.rotary_desc(**r)
    scale = D ** -0.5
    for step, new in enumerate([[50, 3, 17], [20, 33, 16]] + [[1, 1, 1]] * 9):
        T = sum(new)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        pos = torch.tensor([l + t for l, c in zip(lens, new) for t in range(c)], dtype=torch.int32)
        wide = inputs.normal_bf16((T, (Hq + 2 * Hkv) * D), 100 + step, 0)
        w = wide.to(dev)
        cut = lambda x: (x[:, :Hq * D].unflatten(1, (Hq, D)), x[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)),  # noqa: E731
                         x[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D)))
        q, k, v = cut(w)
        q, k = sa.qk_norm_rope(q, k, pos.to(dev), rot, wq.to(dev), wk.to(dev))
        want = plain.norm_rope(cut(wide)[1], pos, wk, rotary=r)
        assert np.all(np.abs(k.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 8e-6 * np.abs(want).max(-1, keepdims=True))
        start = torch.tensor(lens, dtype=torch.int32)
        kc, vc = k.cpu(), cut(wide)[2]
        app = (cu.to(dev), bt.to(dev), start.to(dev), *state)
        if step < 2:
            out, lse = sa.prefill_int8(q, k, v.contiguous(), cu.to(dev), *state, bt.to(dev), start.to(dev), sinks.to(dev), scale)
            check(out, lse, plain.attend_int8(q.cpu(), *ref, bt, start, sinks, scale, new=(kc, vc, cu)), 100)
        sa.append_kv_int8(k, v, *app)
        ref = plain.append_kv_int8(kc, vc, cu, bt, start, *ref)
        assert np.array_equal(state[0].cpu().numpy(), ref[0]) and np.array_equal(state[1].cpu().numpy(), ref[1])
        assert np.array_equal(state[2].double().cpu().numpy(), ref[2])
        lens = [l + c for l, c in zip(lens, new)]
        if step >= 2:
            held = torch.tensor(lens, dtype=torch.int32)
            out, lse = sa.decode_int8(q, *state, bt.to(dev), held.to(dev), sinks.to(dev), scale)
            check(out, lse, plain.attend_int8(q.cpu(), *ref, bt, held, sinks, scale), 100)


def test_empty_calls(sa, cuda_dev):
    """No tokens, no sequences: nothing is written, nothing is refused."""
    kp = torch.ones(3, 2, 16, 64, dtype=torch.int8, device=cuda_dev)
    vp, sc = kp.clone(), torch.ones(3, 2, 2, device=cuda_dev)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    rows = lambda t, h: torch.zeros(t, h, 64, dtype=torch.bfloat16, device=cuda_dev)  # noqa: E731
    out, lse = sa.decode_int8(rows(0, 8), kp, vp, sc, i32(0, 4), i32(0))
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    for n in (0, 2):
        out, lse = sa.prefill_int8(rows(0, 8), rows(0, 2), rows(0, 2), i32(n + 1), kp, vp, sc, i32(n, 4), i32(n))
        assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
        sa.append_kv_int8(rows(0, 2), rows(0, 2), i32(n + 1), i32(n, 4), i32(n), kp, vp, sc)
    torch.cuda.synchronize()
    assert torch.all(kp == 1) and torch.all(vp == 1) and torch.all(sc == 1)


# ------------------------------------------------------------ split query blocks

def _parts_ws(sa, p, dev, window=0):
    """A workspace that lets the call split its query blocks, and into how many parts it does."""
    T, Hq, D = p.q.shape
    c = p.prefix
    desc = sa.paged_desc(len(p.cu_seqlens) - 1, Hq, p.k.shape[1], D, c.k_pages.shape[0], c.block_table.shape[1], window=window)
    n = sa.prefill_int8_workspace_size(desc, T)
    return torch.zeros(n, dtype=torch.uint8, device=dev), (n - 256) // (T * Hq * (D + 2) * 4) if T else 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 1), (128, 4, 2), (64, 3, 3), (128, 1, 1)])
@pytest.mark.parametrize("new,pre", [([17], [1003]), ([1], [4096]), ([130], [2000]), ([128], [128 * 31]),
                                     ([0, 3, 200, 0, 1], [70, 2500, 0, 9, 640])])
@pytest.mark.parametrize("window", [0, 700])
def test_split_blocks(sa, cuda_dev, D, Hq, Hkv, new, pre, window):
    """Few rows over long prefixes, whole and in parts; requests with fewer tiles than parts."""
    p = _make(new, pre, Hq, Hkv, D, seed=D + Hq, sinks=D == 64)
    ref = _ref(p, window)
    ws, parts = _parts_ws(sa, p, cuda_dev, window)
    assert 2 <= parts <= 32
    out, lse = sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws, window=window)
    check(out, lse, ref, 4300)
    small = torch.zeros(ws.numel() - 256, dtype=torch.uint8, device=cuda_dev)  # too small for the parts: whole
    whole, whole_lse = sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=small, window=window)
    check(whole, whole_lse, ref, 4300)
    assert torch.all(small[256:] == 0)
    # the default workspace splits too, whatever SMs the call may use
    for kw in ({}, {"max_sms": 2}, {"return_lse": False}):
        o, m = sa.prefill_int8(*_args(p, cuda_dev), window=window, **kw)
        assert torch.equal(o, out) and (m is None or torch.equal(m, lse))
    assert sa.get_status(ws) == 0 and sa.get_status(small) == 0


def test_split_blocks_of_padded_steps_and_bad_pages(sa, cuda_dev):
    """Rows behind the last request stay; a bad page in one part is reported and hurts its request alone;
    a step in which a page's V scale is out of range is reported."""
    p = _make([5, 9], [3000, 2000], 8, 1, 64, seed=31)
    ref = _ref(p)
    a = list(_args(p, cuda_dev))
    ws, parts = _parts_ws(sa, p, cuda_dev)
    assert parts > 2
    pad = lambda x: torch.cat([x, x[:9]])  # noqa: E731
    out = torch.full((23, 8, 64), 42.0, dtype=torch.bfloat16, device=cuda_dev)
    lse = torch.full((23, 8), 42.0, device=cuda_dev)
    big = torch.zeros(2 * ws.numel(), dtype=torch.uint8, device=cuda_dev)
    sa.prefill_int8(pad(a[0]), pad(a[1]), pad(a[2]), *a[3:], out=out, lse=lse, workspace_buf=big)
    check(out[:14], lse[:14], ref, 3100)
    assert torch.all(out[14:] == 42.0) and torch.all(lse[14:] == 42.0)
    a[7] = a[7].clone()
    a[7][1, 100] = -7
    out, lse = sa.prefill_int8(*a, workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE
    check(out[:5], lse[:5], tuple(x[:5] for x in ref), 3100)


def test_split_blocks_whose_waits_run_out(sa, cuda_dev):
    p = _make([17], [5000], 8, 1, 64, seed=32)
    ws, parts = _parts_ws(sa, p, cuda_dev)
    assert parts > 2
    st = 0
    for _ in range(20):
        sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws, wait_limit_us=1)
        st |= sa.get_status(ws)
        if st:
            break
    assert st == sa.STATUS_WAIT_TIMEOUT
    out, lse = sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws)
    check(out, lse, _ref(p), 5100)
    assert sa.get_status(ws) == 0


def test_split_blocks_on_streams_and_in_graphs(sa, cuda_dev):
    ps = [_make([17], [4000], 8, 1, 64, seed=33), _make([100, 3], [2500, 900], 4, 2, 128, seed=34)]
    args = [_args(p, cuda_dev) for p in ps]
    alone = [sa.prefill_int8(*a) for a in args]
    torch.cuda.synchronize()
    for p, got in zip(ps, alone):
        check(*got, _ref(p), 4100)
    streams, graphs, outs = [torch.cuda.Stream() for _ in args], [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):  # twice on the same stream: the second call's parts wait for the first's merge
                o = sa.prefill_int8(*a)
        graphs.append(g)
        outs.append(o)
    for use_graph in (False, True):
        for _ in range(10):
            got = []
            torch.cuda.synchronize()
            for s, g, a, o in zip(streams, graphs, args, outs):
                with torch.cuda.stream(s):
                    if use_graph:
                        g.replay()
                        got.append(o)
                    else:
                        got.append(sa.prefill_int8(*a))
            torch.cuda.synchronize()
            for (o, l), (q, m) in zip(got, alone):
                assert torch.equal(o, q) and torch.equal(l, m)


def test_which_calls_split(sa, cuda_dev):
    """Those that leave half the SMs or more idle over a table of 4 tiles or more."""
    size = lambda n, Hq, Hkv, D, cols, T, window=0: sa.prefill_int8_workspace_size(  # noqa: E731
        sa.paged_desc(n, Hq, Hkv, D, 8, cols, window=window), T)
    assert size(1, 64, 8, 64, 63, 17) > 256
    assert size(1, 64, 8, 64, 24, 17) == 256  # a short prefix
    assert size(1, 64, 8, 64, 63, 17, 128) == 256  # a short window
    assert size(8, 64, 8, 64, 1024, 4096) == 256  # work for all SMs
    assert size(0, 64, 8, 64, 1024, 0) == 256
    assert size(1, 1, 1, 128, 100000, 1) < 1 << 20
