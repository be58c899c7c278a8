"""Chunked prefill over an INT8 prefix whose V scales are far below the fp16 exponents that the V tiles
have: the result keeps its precision whatever the size, as the decode's over the same cache does.

Tolerance: that of test_prefill_int8_gpu.py, relative to the largest |v| a row sees, so it shrinks with
the scales.  The new rows' V are zeros (in fp16 they have no such range), and their keys count."""
import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs
from test_prefill_int8_gpu import _args, _make, _parts_ws, _ref, check

pytestmark = pytest.mark.gpu


def _tiny(p, exponents, seed):
    """V scales m * 2^e with e of each page of the pool, by page and head; V of the new rows 0."""
    n, heads = p.prefix.kv_scales.shape[:2]
    m = 1 + np.random.default_rng(seed).random((n, heads))
    p.prefix.kv_scales[:, :, 1] = torch.from_numpy((m * np.exp2(exponents)).astype(np.float32))
    p.v = torch.zeros_like(p.v)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [-25, -30, -48, -90, -100])
@pytest.mark.parametrize("window", [0, 200])
def test_all_v_scales_alike(sa, cuda_dev, D, e, window):
    p = _make([100, 300], [300, 700], 16, 2, D, seed=5)
    _tiny(p, np.full(p.prefix.kv_scales.shape[:2], float(e)), 1)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    out, lse = sa.prefill_int8(*_args(p, cuda_dev), window=window, workspace_buf=ws)
    check(out, lse, _ref(p, window), 1000)
    assert sa.get_status(ws) == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 2), (128, 4, 2), (64, 3, 3)])
@pytest.mark.parametrize("step", [-3.0, 3.0, 0.0])
@pytest.mark.parametrize("top", [-26, -40, -85])
def test_scales_that_move_along_the_sequence(sa, cuda_dev, D, Hq, Hkv, step, top):
    """From one key tile to the next by 2^step: every tile raises the largest scale, or none does, or
    neighbouring pages differ; whole and in parts, with tiles of zero scales among them."""
    p = _make([40, 7], [1400, 900], Hq, Hkv, D, seed=11, sinks=D == 64)
    c = p.prefix
    e = np.zeros(c.kv_scales.shape[:2])
    for b, held in enumerate((1400, 900)):
        at = c.block_table[b, :(held + 15) // 16].long().numpy()
        tile = np.arange(len(at)) // 8
        by = step * tile if step else -2.0 * (np.arange(len(at)) % 8)
        e[at] = (top - by.max() + by)[:, None]
    _tiny(p, np.maximum(e, -100), 2)
    at = c.block_table[1, 16:24].long()
    c.kv_scales[at, :, 1] = 0.0  # a whole tile
    c.kv_scales[c.block_table[0, 0], :, 1] = 0.0
    ref = _ref(p)
    whole = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    parts_ws, parts = _parts_ws(sa, p, cuda_dev)
    assert parts >= 2
    for ws in (whole, parts_ws):
        out, lse = sa.prefill_int8(*_args(p, cuda_dev), workspace_buf=ws)
        check(out, lse, ref, 1500)
        assert sa.get_status(ws) == 0


def test_a_first_tile_of_zero_scales(sa, cuda_dev):
    """Zeros say nothing of the sizes to come: ordinary pages, and new rows, after them."""
    p = _make([64], [520], 8, 1, 64, seed=12)
    p.prefix.kv_scales[p.prefix.block_table[0, :8].long(), :, 1] = 0.0
    out, lse = sa.prefill_int8(*_args(p, cuda_dev))
    check(out, lse, _ref(p), 600)


def test_scales_below_the_least_one_are_zeros(sa, cuda_dev):
    """Below 2^-100, which no append writes: as pages of zeros, beside tiny and ordinary ones."""
    p = _make([64], [520], 8, 1, 64, seed=13)
    sc = p.prefix.kv_scales
    sc[::2, :, 1] = 1e-38
    sc[::4, :, 1] = 2.0 ** -120
    out, lse = sa.prefill_int8(*_args(p, cuda_dev))
    check(out, lse, _ref(p), 600)


def test_a_cache_of_tiny_values_as_it_is_served(sa, cuda_dev):
    """Appended by the library, then read by the prefill and by the decode."""
    dev, n, D = cuda_dev, 700, 64
    k = inputs.normal_bf16((n, 2, D), 1, 0)
    v = (inputs.normal_bf16((n, 2, D), 2, 0).double() * 2.0 ** -45).to(torch.bfloat16)
    cols = (n + 15) // 16
    kp, vp = (torch.zeros(cols, 2, 16, D, dtype=torch.int8, device=dev) for _ in range(2))
    sc = torch.zeros(cols, 2, 2, device=dev)
    bt = torch.arange(cols, dtype=torch.int32, device=dev).view(1, -1)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    sa.append_kv_int8(k.to(dev), v.to(dev), i32(0, n), bt, i32(0), kp, vp, sc)
    q = inputs.normal_bf16((1, 16, D), 3, 0)
    own_k, own_v = inputs.normal_bf16((1, 2, D), 4, 0), torch.zeros(1, 2, D, dtype=torch.bfloat16)
    pages = (kp, vp, sc)
    out, lse = sa.prefill_int8(q.to(dev), own_k.to(dev), own_v.to(dev), i32(0, 1), *pages, bt, i32(n))
    host = [x.cpu() for x in (*pages, bt)]
    check(out, lse, plain.attend_int8(q, *host, [n], None, D ** -0.5, new=(own_k, own_v, [0, 1])), 701)
    out, lse = sa.decode_int8(q.to(dev), *pages, bt, i32(n))
    check(out, lse, plain.attend_int8(q, *host, [n], None, D ** -0.5), 701)
