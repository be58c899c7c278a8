"""Quantising append into an INT8 cache (sinkattn_append_kv_int8) on the GPU, bit for bit against its
fp64 form: codes, scales, and every byte that the append does not own."""
import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs

pytestmark = pytest.mark.gpu


def _run(sa, dev, k, v, cu, bt, start, c, ws=None):
    kp, vp, sc = c.k_pages.to(dev), c.v_pages.to(dev), c.kv_scales.to(dev)
    sa.append_kv_int8(k, v, cu.to(dev), bt.to(dev), start.to(dev), kp, vp, sc, workspace_buf=ws)
    torch.cuda.synchronize()
    return kp.cpu().numpy(), vp.cpu().numpy(), sc.cpu().double().numpy()


def _same(got, ref):
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
    assert np.array_equal(got[2], ref[2], equal_nan=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 4, 8])
@pytest.mark.parametrize("new,start", [
    ([1], [0]), ([1, 1, 1, 1], [0, 15, 16, 100]), ([5, 16, 33, 0, 1, 70], [0, 7, 16, 3, 31, 100]),
    ([0, 0, 2], [5, 0, 14]), ([16, 17, 15], [0, 0, 1])])
def test_codes_and_scales_bit_exact(sa, cuda_dev, D, Hkv, new, start):
    a = inputs.make_append(new, start, Hkv, D, seed=sum(start) + D + Hkv, kv_dtype="int8")
    # rows of very different sizes: some pages grow their scale, some keep it
    mag = np.exp(np.random.default_rng(D).uniform(-3, 3, (a.k.shape[0], 1, 1))).astype(np.float32)
    k, v = (a.k.float() * torch.from_numpy(mag)).to(torch.bfloat16), (a.v.float() * torch.from_numpy(mag)).to(torch.bfloat16)
    c = a.cache
    got = _run(sa, cuda_dev, k.to(cuda_dev), v.to(cuda_dev), a.cu_seqlens, c.block_table, a.start_pos, c)
    _same(got, plain.append_kv_int8(k, v, a.cu_seqlens, c.block_table, a.start_pos, c.k_pages, c.v_pages, c.kv_scales))
    assert sa.get_status(sa.workspace(256, cuda_dev, "append")) == 0


@pytest.mark.parametrize("new,start,Hkv", [([700, 1, 1301, 16, 333], [3, 50, 0, 16, 9], 8), ([1] * 1500, None, 2),
                                           ([13] * 1100, None, 1)])
def test_many_tokens_and_many_sequences(sa, cuda_dev, new, start, Hkv):
    """Enough tokens for the group-of-16 plan; more sequences than a block stages."""
    start = start or [(7 * i) % 40 for i in range(len(new))]
    a = inputs.make_append(new, start, Hkv, 64, seed=5, kv_dtype="int8")
    c = a.cache
    got = _run(sa, cuda_dev, a.k.to(cuda_dev), a.v.to(cuda_dev), a.cu_seqlens, c.block_table, a.start_pos, c)
    _same(got, plain.append_kv_int8(a.k, a.v, a.cu_seqlens, c.block_table, a.start_pos, c.k_pages, c.v_pages, c.kv_scales))


def test_token_by_token_and_strided_rows(sa, cuda_dev):
    """A page filled one token at a time from a fused projection's rows."""
    Hkv, D, T = 2, 64, 35
    wide = inputs.normal_bf16((T, (4 + 2 * Hkv) * D), 3, 0)
    wide = (wide.float() * torch.exp(torch.linspace(-2, 2, T))[:, None]).to(torch.bfloat16)
    k, v = wide[:, 4 * D:(4 + Hkv) * D].unflatten(1, (Hkv, D)), wide[:, (4 + Hkv) * D:].unflatten(1, (Hkv, D))
    c = inputs.make_append([T], [0], Hkv, D, seed=8, kv_dtype="int8").cache
    dev = cuda_dev
    w = wide.to(dev)
    kd, vd = w[:, 4 * D:(4 + Hkv) * D].unflatten(1, (Hkv, D)), w[:, (4 + Hkv) * D:].unflatten(1, (Hkv, D))
    kp, vp, sc = c.k_pages.to(dev), c.v_pages.to(dev), c.kv_scales.to(dev)
    ref = (c.k_pages, c.v_pages, c.kv_scales)
    cu, bt = torch.tensor([0, 1], dtype=torch.int32), c.block_table
    for t in range(T):
        sa.append_kv_int8(kd[t:t + 1], vd[t:t + 1], cu.to(dev), bt.to(dev), torch.tensor([t], dtype=torch.int32, device=dev),
                          kp, vp, sc)
        ref = plain.append_kv_int8(k[t:t + 1], v[t:t + 1], cu, bt, [t], *ref)
    _same((kp.cpu().numpy(), vp.cpu().numpy(), sc.cpu().double().numpy()), ref)
    # the same rows in one call: the whole pages hold the same, the strided rows are read as they lie
    kp2, vp2, sc2 = c.k_pages.to(dev), c.v_pages.to(dev), c.kv_scales.to(dev)
    sa.append_kv_int8(kd, vd, torch.tensor([0, T], dtype=torch.int32, device=dev), bt.to(dev),
                      torch.zeros(1, dtype=torch.int32, device=dev), kp2, vp2, sc2)
    _same((kp2.cpu().numpy(), vp2.cpu().numpy(), sc2.cpu().double().numpy()),
          plain.append_kv_int8(k, v, [0, T], bt, [0], c.k_pages, c.v_pages, c.kv_scales))


@pytest.mark.parametrize("start", [0, 5])
def test_special_values(sa, cuda_dev, start):
    """Zeros, subnormals, ties, infinities and NaN."""
    Hkv, D, T = 8, 64, 20
    a = inputs.make_append([T], [start], Hkv, D, seed=6, kv_dtype="int8")
    k = a.k.clone()
    k[:, 0] = 0
    k[:, 1] = 1e-40
    k[:, 2] = (torch.arange(T * D).view(T, D) % 255 - 127).to(torch.bfloat16) * 0.5  # ties at a scale of 0.5
    k[:, 2, 0] = 63.5
    k[:, 3] = 1e-33
    k[3, 4, 5], k[4, 4, 6], k[5, 4, 7] = float("inf"), float("-inf"), float("nan")
    k[:, 5] = float("nan")
    k[:, 6] = 3e38
    k[2, 6] = 1.0
    c = a.cache
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    got = _run(sa, cuda_dev, k.to(cuda_dev), a.v.to(cuda_dev), a.cu_seqlens, c.block_table, a.start_pos, c, ws)
    assert sa.get_status(ws) == sa.STATUS_VALUE_RANGE
    _same(got, plain.append_kv_int8(k, a.v, a.cu_seqlens, c.block_table, a.start_pos, c.k_pages, c.v_pages, c.kv_scales))


def test_bad_pages_lengths_and_padding_are_skipped(sa, cuda_dev):
    Hkv, D = 2, 64
    new, start = [4, 20, 3, 6], [2, 10, 0, 5]
    a = inputs.make_append(new, start, Hkv, D, seed=7, kv_dtype="int8")
    c = a.cache
    bt = c.block_table.clone()
    bt[1, 1] = c.num_pages  # the second page of sequence 1
    bt[2, 0] = -1
    st = a.start_pos.clone()
    st[3] = -1  # its tokens' positions: -1, 0, ..
    pad = inputs.normal_bf16((5, Hkv, D), 1, 0)
    k, v = torch.cat([a.k, pad]), torch.cat([a.v, pad])
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    got = _run(sa, cuda_dev, k.to(cuda_dev), v.to(cuda_dev), a.cu_seqlens, bt, st, c, ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_PAGE | sa.STATUS_BAD_LENGTH | sa.STATUS_BAD_CU_SEQLENS
    # what is left: sequence 0, sequence 1's first page (6 tokens) and its third, sequence 3 from position 0
    rows = lambda x: torch.cat([x[0:4], x[4:10], x[28:33]])  # noqa: E731
    t2 = torch.tensor([[int(bt[0, i]) for i in range(1)] + [0], [int(bt[1, 0]), 0], [int(bt[3, 0]), 0]])
    ref = plain.append_kv_int8(rows(k), rows(v), [0, 4, 10, 15], t2, [2, 10, 0], c.k_pages, c.v_pages, c.kv_scales)
    _same(got, ref)


def test_captured(sa, cuda_dev):
    Hkv, D, B = 8, 64, 16
    a = inputs.make_append([1] * B, [5 * i for i in range(B)], Hkv, D, seed=9, kv_dtype="int8")
    c, dev = a.cache, cuda_dev
    k, v, cu, bt, st = (x.to(dev) for x in (a.k, a.v, a.cu_seqlens, c.block_table, a.start_pos))
    kp, vp, sc = c.k_pages.to(dev), c.v_pages.to(dev), c.kv_scales.to(dev)
    sa.append_kv_int8(k, v, cu, bt, st, kp.clone(), vp.clone(), sc.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.append_kv_int8(k, v, cu, bt, st, kp, vp, sc)
    ref = (c.k_pages, c.v_pages, c.kv_scales)
    for i in range(3):
        x, y = inputs.new_rows(B, Hkv, D, seed=i)
        x = x * (i + 1)
        k.copy_(x)
        v.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        ref = plain.append_kv_int8(x, y, a.cu_seqlens, c.block_table, a.start_pos, *ref)
    _same((kp.cpu().numpy(), vp.cpu().numpy(), sc.cpu().double().numpy()), ref)
