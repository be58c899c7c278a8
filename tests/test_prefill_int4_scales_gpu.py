"""Chunked prefill over a 4-bit prefix whose V scales are far below fp16's exponents: the result keeps its
precision whatever their size, as the decode's over the same cache does.

Tolerance: that of test_int4_gpu.py, relative to the largest |v| a row sees, so it shrinks with the
scales.  (What the powers of two add: fp16's steps of V, 2^-15 of the largest scale in 32 keys, and of P where
a tile's scales are smaller than those met, 2^-25 of the largest |v| for each key: 2^-14 for the 1400 here,
together within the fp32 scores' 2^-12, which these small scores do not use up.)  Where the prefix alone is
small the new rows' V are zeros, and their keys count."""
import numpy as np
import pytest
import torch

from paged_gqa_attention_head_gb300 import inputs
from test_int4_gpu import _pre, _pre_ref, _scaled, check

pytestmark = pytest.mark.gpu


def _v_times(p, exponents):
    """The prefix's cache with the V scales of page n times 2^exponents[n]; V of the new rows 0."""
    c = p.prefix
    p.v = torch.zeros_like(p.v)

    def f(shape):
        e = np.ones(shape)
        e[:, :, 1] = np.exp2(exponents)[:, None, None]
        return e
    return _scaled(inputs.pack_int4(c.k_pages, c.v_pages), p.q.shape[2], f)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [-8, -16, -22, -30, -60, -95])
@pytest.mark.parametrize("window", [0, 200])
def test_all_v_scales_alike(sa, cuda_dev, D, e, window):
    p = inputs.make_prefill([100, 300], 16, 2, D, seed=5, prefix_lens=[300, 700], poison=False)
    kv = _v_times(p, np.full(p.prefix.num_pages, float(e)))
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    out, lse = sa.prefill_int4(*_pre(p, cuda_dev, kv), window=window, workspace_buf=ws)
    check(out, lse, _pre_ref(p, window, kv))
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 2), (128, 4, 2), (64, 3, 3)])
@pytest.mark.parametrize("step", [-3.0, 3.0, 0.0])
@pytest.mark.parametrize("top", [0, -20, -60])
def test_scales_that_move_along_the_sequence(sa, cuda_dev, D, Hq, Hkv, step, top):
    """From one key tile to the next by 2^step: every tile raises the largest scale, or none does, or
    neighbouring pages differ; whole and in parts, with tiles of zero scales among them."""
    p = inputs.make_prefill([40, 7], Hq, Hkv, D, seed=11, sinks=D == 64, prefix_lens=[1400, 900], poison=False)
    c = p.prefix
    e = np.zeros(c.num_pages)
    for b, held in enumerate((1400, 900)):
        at = c.block_table[b, :(held + 15) // 16].long().numpy()
        tile = np.arange(len(at)) // 8
        by = step * tile if step else -2.0 * (np.arange(len(at)) % 8)
        e[at] = top - by.max() + by
    e[c.block_table[1, 16:24].long().numpy()] = -np.inf  # a whole tile
    e[int(c.block_table[0, 0])] = -np.inf
    kv = _v_times(p, e)
    ref, a = _pre_ref(p, kv=kv), _pre(p, cuda_dev, kv)
    check(*sa.prefill_int4(*a), ref)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)  # too little for parts
    check(*sa.prefill_int4(*a, workspace_buf=ws), ref)
    assert sa.get_status(ws) == 0 and sa.default_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_ordinary_rows_after_small_ones(sa, cuda_dev, D):
    """A prefix that begins with tiles of zero and of tiny scales, then ordinary pages and ordinary new rows."""
    p = inputs.make_prefill([64], 8, 1, D, seed=12, prefix_lens=[520], poison=False)
    v = p.v
    e = np.zeros(p.prefix.num_pages)
    e[p.prefix.block_table[0, :8].long().numpy()] = -np.inf
    e[p.prefix.block_table[0, 8:16].long().numpy()] = -40.0
    kv = _v_times(p, e)
    p.v = v
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), _pre_ref(p, kv=kv))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("top", [0.0, -50.0])
def test_scores_that_rise_and_sinks_above_them(sa, cuda_dev, D, top):
    """K scales that grow by 2 from tile to tile, V's smaller by as much; sinks below, among and above the scores."""
    p = inputs.make_prefill([33], 8, 1, D, seed=14, prefix_lens=[900], poison=False)
    p.sinks = torch.tensor([-40.0, -3.0, 0.0, 1.0, 4.0, 8.0, 12.0, 16.0])
    kv = inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages)
    p.v = torch.zeros_like(p.v)
    up = np.zeros(p.prefix.num_pages)
    up[p.prefix.block_table[0, :57].long().numpy()] = np.arange(57) // 8
    e = np.stack([up - 4, top - up], axis=1)[:, None, :, None]
    kv = _scaled(kv, D, lambda shape: np.exp2(e) * np.ones(shape))
    ref = _pre_ref(p, kv=kv)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), ref)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv), workspace_buf=ws), ref)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [-60, -20, 0, 12, 20])
def test_k_scales_of_every_size(sa, cuda_dev, D, e):
    """K scales times 2^e against queries and new keys times powers of two that keep the scores' size."""
    p = inputs.make_prefill([40, 9], 8, 2, D, seed=15, prefix_lens=[700, 130], poison=False)
    kv = _scaled(inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages), D,
                 lambda shape: np.exp2(np.array([e, 0.0]))[None, None, :, None] * np.ones(shape))
    p.q = (p.q.double() * 2.0 ** -e).to(torch.bfloat16)
    p.k = (p.k.double() * 2.0 ** e).to(torch.bfloat16)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), _pre_ref(p, kv=kv))
    assert sa.default_status() == 0


@pytest.mark.parametrize("e", [-100, -50, -20, -3, 10])
def test_new_values_of_every_size(sa, cuda_dev, e):
    """The new tokens' V times 2^e, alone and beside a prefix of the same size."""
    p = inputs.make_prefill([200, 30], 8, 2, 64, seed=16, prefix_lens=[0, 700], poison=False)
    kv = _v_times(p, np.full(p.prefix.num_pages, float(e)))
    p.v = (inputs.make_prefill([200, 30], 8, 2, 64, seed=16, prefix_lens=[0, 700], poison=False).v.double() * 2.0 ** e).to(
        torch.bfloat16)
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), _pre_ref(p, kv=kv))
    assert sa.default_status() == 0


def test_k_scales_out_of_range(sa, cuda_dev):
    """2^34 is reported, where a token's word is; in a slot that holds none it is nothing."""
    p = inputs.make_prefill([20], 8, 1, 64, seed=17, prefix_lens=[100], poison=False)
    kv = inputs.pack_int4(p.prefix.k_pages, p.prefix.v_pages)
    ref = _pre_ref(p, kv=kv)
    last = int(p.prefix.block_table[0, 6])
    words = kv.view(torch.int16)[:, :, 0, 8].view(-1, 1, 2, 16)  # [page, head, group, token]
    words[last, 0, 1, 4:] = 0x5080
    sa.default_status()
    check(*sa.prefill_int4(*_pre(p, cuda_dev, kv)), ref)
    assert sa.default_status() == 0
    words[last, 0, 1, 3] = 0x5080
    sa.prefill_int4(*_pre(p, cuda_dev, kv))
    assert sa.default_status() == sa.STATUS_VALUE_RANGE
