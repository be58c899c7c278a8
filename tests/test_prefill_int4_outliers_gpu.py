"""Chunked prefill over a 4-bit prefix with a few V far larger than the others: a row keeps the precision that
its own visible values allow, whatever other keys of its tiles hold.

Tolerance: that of test_int4_gpu.py (a rounding to bf16; P in fp16 and fp32 scores, 2^-11 and 2^-12 of the
largest |v| that the row sees).  Where a large V is seen with a weight below 2^-60, it is left out of that largest
|v|: 2^21 of it and 32 such keys add less than 2^-30 of an ordinary one."""
import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs
from test_int4_gpu import _pre, _pre_ref, _scaled, check

pytestmark = pytest.mark.gpu


def _large(shape, e, seed):
    """Values of either sign from 2^e to 2^(e + 1)."""
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.uniform(1.0, 1.9, shape) * r.choice([-1.0, 1.0], shape) * 2.0 ** e).to(torch.bfloat16)


def _hide(p, kv_rows=(), new_rows=()):
    """A negligible weight for some keys, whatever the query: channel 0 is 8 in every query, 0 in every
    key but these, -64 there (scores of -512 / sqrt(D), below -45)."""
    p.q[:, :, 0] = 8.0
    p.k[:, :, 0] = 0.0
    c = p.prefix
    c.k_pages[..., 0] = 0.0
    for b, j in kv_rows:
        c.k_pages[int(c.block_table[b, j // 16]), :, j % 16, 0] = -64.0
    for t in new_rows:
        p.k[t, :, 0] = -64.0


def _times(p, exponents):
    """The prefix's cache with the V scales of pages of the first request times powers of two."""
    c = p.prefix
    up = np.zeros(c.num_pages)
    for n, e in exponents.items():
        up[int(c.block_table[0, n])] = e

    def f(shape):
        x = np.ones(shape)
        x[:, :, 1] = np.exp2(up)[:, None, None]
        return x
    return _scaled(inputs.pack_int4(c.k_pages, c.v_pages), p.q.shape[2], f)


def _words_times(p, up):
    """The prefix's cache with V scales times 2^up, up [pages, heads, groups of 32 channels, tokens]."""
    def f(shape):
        x = np.ones(shape)
        x[:, :, 1] = np.exp2(up).reshape(shape[0], shape[1], shape[3])
        return x
    return _scaled(inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages), p.q.shape[2], f)


def _quiet_ref(p, kv, window=0, new_rows=(), kv_small=None):
    """The reference, with the largest |v| that a row sees from a cache and new rows without the large ones."""
    out, lse, _ = _pre_ref(p, window, kv)
    v = p.v
    p.v = v.clone()
    for t in new_rows:
        p.v[t] = 0.0
    vmax = _pre_ref(p, window, kv if kv_small is None else kv_small)[2]
    p.v = v
    return out, lse, vmax


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pre", [0, 300])
@pytest.mark.parametrize("e", [8, 14, 17, 20])
def test_a_later_token_of_another_quarter(sa, cuda_dev, D, pre, e):
    """Causal mask: the last of 128 new tokens is large; the rows of the first 96 share its tile alone."""
    p = inputs.make_prefill([128, 128], 8, 2, D, seed=31, prefix_lens=[pre, 40], poison=False)
    p.v[127] = _large(p.v[127].shape, e, 1)
    kv = inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages)
    ref = _pre_ref(p, kv=kv)
    out, lse = sa.prefill_int4(*_pre(p, cuda_dev, kv))
    for rows in (slice(0, 96), slice(127, 256)):
        check(out[rows], lse[rows], tuple(x[rows] for x in ref))
    assert sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pre", [0, 300])
@pytest.mark.parametrize("e", [8, 14, 17, 20])
def test_later_and_earlier_tokens_of_the_same_quarter(sa, cuda_dev, D, pre, e):
    """Of 32 new tokens that share a power of two the last is large, or, with a window, the first."""
    p = inputs.make_prefill([128, 60], 8, 2, D, seed=36, prefix_lens=[pre, 40], poison=False)
    kv = inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages)
    v = p.v.clone()
    p.v[[31, 95, 127]] = _large(p.v[:3].shape, e, 4)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), _pre_ref(p, kv=kv))
    p.v = v
    p.v[[0, 64]] = _large(p.v[:2].shape, e, 5)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), window=20), _pre_ref(p, 20, kv))
    assert sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [-60, -20, -9, 5])
@pytest.mark.parametrize("window", [0, 2, 40])
def test_large_tokens_among_values_of_any_size(sa, cuda_dev, D, size, window):
    """Tokens 2^14 times the others, whatever the others' size; two of 32 among the new ones, one of 64 in the prefix."""
    p = inputs.make_prefill([150, 70], 4, 2, D, seed=42, sinks=window == 2, prefix_lens=[0, 300], poison=False)
    v = p.v.double() * 2.0 ** size
    v[5::16] *= 2.0 ** 14
    p.v = v.to(torch.bfloat16)
    up = np.full((p.prefix.num_pages, 2, D // 32, 16), float(size))
    up[::4, :, :, 9] += 12.0
    kv = _words_times(p, up)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), window=window), _pre_ref(p, window, kv))
    assert sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [True, False])
@pytest.mark.parametrize("e", [8, 13, 18])
def test_a_prefix_token_before_the_window(sa, cuda_dev, D, sinks, e):
    """Window 70: one token of the 32 that share a power of two is large, and hidden from the rows that see the rest."""
    p = inputs.make_prefill([60], 8, 2, D, seed=38, sinks=sinks, prefix_lens=[400], poison=False)
    up = np.zeros((p.prefix.num_pages, 2, D // 32, 16))
    for j in (352, 384):
        up[int(p.prefix.block_table[0, j // 16]), :, :, j % 16] = e
    kv = _words_times(p, up)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), window=70), _pre_ref(p, 70, kv))
    assert sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [3, 60, 1000])
@pytest.mark.parametrize("e", [6, 9, 13, 18])
def test_a_prefix_token_of_no_weight(sa, cuda_dev, D, at, e):
    """One large token of the prefix that every row sees with a weight below 2^-60; whole and in parts."""
    p = inputs.make_prefill([60, 3], 8, 2, D, seed=39, prefix_lens=[1100, 64], poison=False)
    _hide(p, [(0, at)])
    up = np.zeros((p.prefix.num_pages, 2, D // 32, 16))
    page = int(p.prefix.block_table[0, at // 16])
    up[page, :, :, at % 16] = e
    kv = _words_times(p, up)
    up[page, :, :, at % 16] = -np.inf
    ref = _quiet_ref(p, kv, kv_small=_words_times(p, up))
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), ref)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), workspace_buf=ws), ref)
    assert sa.get_status(ws) == 0 and sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [6, 9, 13, 18])
@pytest.mark.parametrize("base", [0, -40])
def test_large_channels_of_the_prefix(sa, cuda_dev, D, e, base):
    """The first 32 channels of every token are large: the others keep the precision of their own size, to the
    last bit where a row sees one token."""
    p = inputs.make_prefill([40, 1], 8, 2, D, seed=40, sinks=False, prefix_lens=[700, 0], poison=False)
    p.v[:] = 0.0
    up = np.full((p.prefix.num_pages, 2, D // 32, 16), float(base))
    small = up.copy()
    up[:, :, 0] += e
    small[:, :, 0] = -np.inf
    kv = _words_times(p, up)
    ref = _pre_ref(p, kv=kv)
    out, lse = sa.prefill_int4(*_pre(p, cuda_dev, kv))
    check(out, lse, ref)
    check(out[..., 32:], lse, (ref[0][..., 32:], ref[1], _pre_ref(p, kv=_words_times(p, small))[2]))
    # a window of two: the first new row sees the prefix's last token and itself, whose weight is nothing
    p.q[:, :, 0] = 8.0
    p.k[:, :, 0] = -64.0
    p.prefix.k_pages[..., 0] = 0.0
    kv = _words_times(p, up)
    want = plain.values_int4(kv)[1][int(p.prefix.block_table[0, 43]), :, 699 % 16]
    out = sa.prefill_int4(*_pre(p, cuda_dev, kv), window=2)[0][0].double().cpu().numpy()
    assert np.array_equal(out, np.repeat(want, 4, axis=0))
    assert sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pre", [0, 300])
@pytest.mark.parametrize("e", [0, 10, 13, 17])
def test_a_large_channel(sa, cuda_dev, D, pre, e):
    """One channel of the new V is large: the others keep the precision of their own size."""
    p = inputs.make_prefill([150, 20], 8, 2, D, seed=37, sinks=pre > 0, prefix_lens=[pre, 0], poison=False)
    p.v[:, :, 5] = _large(p.v[:, :, 5].shape, e, 6)
    kv = inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages)
    ref = _pre_ref(p, kv=kv)
    out, lse = sa.prefill_int4(*_pre(p, cuda_dev, kv))
    check(out, lse, ref)
    rest = [i for i in range(D) if i != 5]
    v = p.v.clone()
    p.v[:, :, 5] = 0.0
    check(out[..., rest], lse, (ref[0][..., rest], ref[1], _pre_ref(p, kv=kv)[2]))
    if not pre:
        # a row that sees one key, no sink: that key's V.  V lies in fp16 over 2^k (k at most 0 for a largest below 2^4,
        # (e - 2) / 2 for one from 2^e on), whose steps are 2^-24: eight bits are exact from 2^(k - 17) on, below that
        # half a step of 2^(k - 24) is lost at most, and then a rounding to bf16
        k = max(0, (e - 2) // 2)
        for got, want in ((out[0, :4], v[0, :1]), (out[150, 4:], v[150, 1:])):
            err = (got.cpu().double() - want.double()).abs()
            assert bool((err <= torch.where(want.double().abs() >= 2.0 ** (k - 17), 0.0, 2.0 ** (k - 25) * (1 + 2.0 ** -8)
                                            + 2.0 ** (k - 25))).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [True, False])
@pytest.mark.parametrize("e", [8, 14, 17])
def test_tokens_before_the_window(sa, cuda_dev, D, sinks, e):
    """Window 70: large V of 32 keys of the prefix and of the first 32 new tokens, seen by the first rows alone."""
    p = inputs.make_prefill([200], 8, 2, D, seed=32, sinks=sinks, prefix_lens=[400], poison=False)
    p.v[:32] = _large(p.v[:32].shape, e, 2)
    kv = _times(p, {20: e, 21: e})  # keys 320 .. 351 of 400: rows past 21 see none of them
    ref = _pre_ref(p, 70, kv)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), window=70), ref)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), window=70, workspace_buf=ws), ref)
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 1), (64, 16, 2), (128, 4, 2)])
@pytest.mark.parametrize("at", [0, 100, 1000])
@pytest.mark.parametrize("e", [10, 14, 17])
def test_a_page_of_no_weight(sa, cuda_dev, D, Hq, Hkv, at, e):
    """A quarter (32 keys) of large V that every row sees with a weight below 2^-60, in the first tile or a later one;
    whole and in parts."""
    p = inputs.make_prefill([60, 3], Hq, Hkv, D, seed=33, prefix_lens=[1100, 64], poison=False)
    rows = [(0, at // 32 * 32 + j) for j in range(32)]
    _hide(p, rows)
    first = at // 32 * 2
    kv = _times(p, {first: e, first + 1: e})
    ref = _quiet_ref(p, kv, kv_small=_times(p, {first: -np.inf, first + 1: -np.inf}))
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), ref)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), workspace_buf=ws), ref)
    assert sa.get_status(ws) == 0 and sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pre", [0, 200])
@pytest.mark.parametrize("e", [10, 16, 20])
def test_new_tokens_of_no_weight(sa, cuda_dev, D, pre, e):
    """The first 32 new tokens are large and weigh nothing for the rows behind them."""
    p = inputs.make_prefill([300], 8, 2, D, seed=34, prefix_lens=[pre], poison=False)
    p.v[:32] = _large(p.v[:32].shape, e, 3)
    _hide(p, new_rows=range(32))
    kv = inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages)
    first = 0 if pre else 32  # without a prefix they are all that the first rows see
    ref = _quiet_ref(p, kv, new_rows=range(32))
    out, lse = sa.prefill_int4(*_pre(p, cuda_dev, kv))
    check(out[first:], lse[first:], tuple(x[first:] for x in ref))
    if first:
        check(out[:first], lse[:first], tuple(x[:first] for x in _pre_ref(p, kv=kv)))
    assert sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 40, 200])
@pytest.mark.parametrize("sink", [-30.0, 0.0, 30.0, 60.0])
def test_sinks_beside_values_of_any_size(sa, cuda_dev, D, window, sink):
    """V of the first tiles zero, then tiny, ordinary and large; with a window some rows see nothing of their
    item's first tile."""
    p = inputs.make_prefill([150], 4, 2, D, seed=35, prefix_lens=[700], poison=False)
    p.sinks = torch.full((4,), sink)
    kv = _times(p, dict(enumerate(np.repeat([-np.inf, -50.0, -50.0, 0.0, 12.0, 0.0], 8)[:44])))
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), window=window), _pre_ref(p, window, kv))
    assert sa.default_status() == 0
