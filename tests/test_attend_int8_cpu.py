"""The fp64 form of the attention over INT8 pages pinned to the C oracle, and the refusals of the
entry points that attend (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs


def _as_bf16(c):
    """Scales that are powers of two and codes of at most 8 bits are bf16 values."""
    c.kv_scales = torch.exp2(torch.floor(torch.log2(c.kv_scales)))
    return [torch.from_numpy(plain.values(p, c.kv_scales, i)).to(torch.bfloat16)
            for i, p in enumerate((c.k_pages, c.v_pages))]


@pytest.mark.parametrize("window", [0, 5])
@pytest.mark.parametrize("sinks", [True, False])
def test_attend_matches_the_c_oracle(oracle_mod, window, sinks):
    D, Hkv, G = 64, 2, 4
    lens = [0, 1, 16, 37, 90]
    w = inputs.make_decode(lens, len(lens), Hkv * G, Hkv, D, seed=5, sinks=sinks, kv_dtype="int8", poison=False)
    kb, vb = _as_bf16(w.cache)
    c = w.cache
    ro, rl = oracle_mod.decode(w.q, kb, vb, c.block_table, c.lens, w.sinks, w.scale, window=window)
    out, lse, _ = plain.attend_int8(w.q, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens, w.sinks, w.scale,
                                    window=window)
    np.testing.assert_allclose(out, ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)
    p = inputs.make_prefill([3, 0, 20], Hkv * G, Hkv, D, seed=6, sinks=sinks, prefix_lens=[17, 5, 0],
                            prefix_kv_dtype="int8", poison=False)
    kb, vb = _as_bf16(p.prefix)
    c = p.prefix
    ro, rl = oracle_mod.prefill(p.q, p.k, p.v, p.cu_seqlens, p.sinks, p.scale, kb, vb, c.block_table, c.lens,
                                window=window)
    out, lse, _ = plain.attend_int8(p.q, c.k_pages, c.v_pages, c.kv_scales, c.block_table, c.lens, p.sinks, p.scale,
                                    window=window, new=(p.k, p.v, p.cu_seqlens))
    np.testing.assert_allclose(out, ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)


def _host():
    buf = (ctypes.c_uint8 * 8192)()
    return buf, (ctypes.addressof(buf) + 255) // 256 * 256


def _desc(sa, **kw):
    d = dict(num_seqs=4, num_qo_heads=8, num_kv_heads=2, head_dim=64, num_pages=10, max_pages_per_seq=4)
    d.update(kw)
    return sa.paged_desc(**d)


def test_decode_int8_rejects(sa):
    lib, (buf, p) = sa.load(), _host()

    def dec(q=p, kp=p, vp=p, sc=p, bt=p, sl=p, out=p, ws=p, d=_desc(sa)):
        return lib.sinkattn_decode_int8(q, kp, vp, sc, bt, sl, None, 0.125, out, None, ctypes.byref(d), ws, 256, None)
    for kw in (dict(q=None), dict(kp=None), dict(vp=None), dict(sc=None), dict(bt=None), dict(sl=None), dict(out=None),
               dict(ws=None), dict(kp=p + 8), dict(vp=p + 4), dict(sc=p + 4), dict(q=p + 2)):
        assert dec(**kw) == 1, kw
    assert dec(d=_desc(sa, num_seqs=0), q=None, kp=None) == 0
    assert dec(d=_desc(sa, head_dim=32)) == 2
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sa.decode_int8(x, None, None, None, None, None)


def test_prefill_int8_rejects(sa):
    lib, (buf, p) = sa.load(), _host()

    def pre(q=p, k=p, v=p, cu=p, T=8, kp=p, vp=p, sc=p, bt=p, pl=p, out=p, ws=p, wb=256, scale=0.125, d=_desc(sa)):
        return lib.sinkattn_prefill_int8(q, k, v, cu, T, kp, vp, sc, bt, pl, None, scale, out, None, ctypes.byref(d),
                                         ws, wb, None)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(kp=None), dict(vp=None), dict(sc=None),
               dict(bt=None), dict(pl=None), dict(out=None), dict(ws=None), dict(sc=p + 4), dict(out=p + 16), dict(T=-1),
               dict(kp=p + 8), dict(scale=0.0), dict(scale=float("nan")), dict(d=_desc(sa, num_pages=0))):
        assert pre(**kw) == 1, kw
    assert pre(wb=128) == 3
    assert pre(d=_desc(sa, head_dim=32)) == 2
    assert pre(T=0, q=None, kp=None) == 0
    assert pre(d=_desc(sa, num_seqs=0), q=None) == 0
    n = ctypes.c_size_t()
    size = lambda T=8, d=_desc(sa), out=ctypes.byref(n): lib.sinkattn_prefill_int8_workspace_size(  # noqa: E731
        None if d is None else ctypes.byref(d), T, out)
    assert size(T=-1) == 1 and size(d=None) == 1 and size(out=None) == 1 and size(d=_desc(sa, head_dim=32)) == 2
    assert size(T=0) == 0 and n.value == 256 and size(d=_desc(sa, num_seqs=0)) == 0 and n.value == 256
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sa.prefill_int8(x, x, x, None, None, None, None, None, None)
