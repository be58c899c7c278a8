"""The fp64 form of the query/key preparation pinned to the C oracle, to closed forms and to itself;
the entry point's refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs


def test_yarn_matches_the_c_oracle(oracle_mod):
    x = inputs.normal_bf16((5, 3, 64), 9, 0)
    pos = np.array([0, 1, 77, 4096, 131071])
    r = dict(base=150000.0, rotary_dim=64, factor=32.0, scaling="yarn")
    np.testing.assert_allclose(plain.norm_rope(x, pos, rotary=r), oracle_mod.rope(x, pos, 150000.0, 32.0), atol=1e-9)


def test_layouts_agree_up_to_a_permutation():
    x = inputs.normal_bf16((5, 3, 64), 9, 0).double().numpy()
    pos = np.array([0, 1, 77, 4096, 131071])
    r = dict(base=10000.0, rotary_dim=32, factor=4.0, scaling="linear")
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2), np.arange(32, 64)])
    a = plain.norm_rope(x[..., perm], pos, rotary=r)
    b = plain.norm_rope(x, pos, rotary=dict(r, interleaved=True))
    np.testing.assert_allclose(a, b[..., perm], atol=1e-12)


def test_closed_forms():
    w = plain.rotary_rates(500000.0, 128)[0]
    np.testing.assert_allclose(plain.rotary_rates(500000.0, 128, 4.0, "linear")[0], w / 4, rtol=1e-15)
    th, ms = plain.rotary_rates(500000.0, 128, 8.0, "wavelength", 8192, 4.0, 1.0)
    assert ms == 1.0 and th[0] == w[0]
    np.testing.assert_allclose(th[-1], w[-1] / 8, rtol=1e-15)
    assert np.all(th <= w) and np.all(th >= w / 8 * (1 - 1e-15))
    x = np.random.default_rng(1).standard_normal((2, 3, 64))
    y = plain.norm_rope(x, [3, 4], weight=np.full(64, 2.0), eps=0.0, rotary=dict(base=10000.0, rotary_dim=64))
    np.testing.assert_allclose((y ** 2).mean(-1), 4.0, rtol=1e-12)  # a rotation keeps the norm
    # the scores of two rotated rows depend on the distance of their positions alone
    r = dict(base=10000.0, rotary_dim=64, interleaved=True)
    s = [np.vdot(plain.norm_rope(x[:1, :1], [p + 5], rotary=r), plain.norm_rope(x[1:, :1], [p], rotary=r))
         for p in (0, 17, 4000)]
    np.testing.assert_allclose(s, s[0], atol=1e-9)


def _desc(sa, **kw):
    d = dict(num_seqs=0, num_qo_heads=1, num_kv_heads=1, head_dim=64, num_pages=0, max_pages_per_seq=0)
    d.update(kw)
    return sa.paged_desc(**d)


def test_rejects(sa):
    lib = sa.load()
    buf = (ctypes.c_uint8 * 16384)()
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    far = p + 8192
    rot = sa.rotary_desc(10000.0, 64)

    def call(q=p, qs=64, k=p + 1024, ks=64, wq=None, wk=None, eps=1e-6, pos=p, T=2, r=rot, qo=far, ko=far + 1024, d=None,
             ws=None, wb=0):
        d = d or _desc(sa)
        return lib.sinkattn_qk_norm_rope(q, qs, k, ks, wq, wk, eps, pos, T, ctypes.byref(r) if r else None, qo, ko,
                                         ctypes.byref(d), ws, wb, None)
    for kw in (dict(q=None), dict(qo=None), dict(ko=None), dict(k=None), dict(q=None, qo=None, k=None, ko=None),
               dict(pos=None), dict(q=p + 2), dict(qo=far + 8), dict(wq=p + 4), dict(wk=p + 8), dict(qs=63), dict(ks=68),
               dict(eps=-1.0), dict(eps=float("nan")), dict(T=-1), dict(ws=p, wb=128), dict(ws=p + 16, wb=256),
               dict(qo=p + 128), dict(ko=p), dict(qo=p + 1024), dict(ko=far), dict(qo=p, qs=128),
               dict(r=sa.rotary_desc(1.0, 64)), dict(r=sa.rotary_desc(10000.0, 0)), dict(r=sa.rotary_desc(10000.0, 80)),
               dict(r=sa.rotary_desc(float("nan"), 64)), dict(r=sa.rotary_desc(10000.0, 64, 0.5, "linear")),
               dict(r=sa.rotary_desc(10000.0, 64, 4.0, "yarn", beta_fast=1.0, beta_slow=1.0)),
               dict(r=sa.rotary_desc(10000.0, 64, 4.0, "wavelength", original_context=0)),
               dict(r=sa.rotary_desc(10000.0, 64, float("inf"), "yarn"))):
        assert call(**kw) == 1, kw
    assert call(r=sa.rotary_desc(10000.0, 24)) == 2
    assert call(d=_desc(sa, head_dim=96)) == 2
    assert call(T=0) == 0
    with pytest.raises(ValueError):
        sa.rotary_desc(10000.0, 64, 4.0, "cubic")


def test_binding_refuses_host_tensors(sa):
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sa.qk_norm_rope(x, x, torch.zeros(1, dtype=torch.int32), sa.rotary_desc(10000.0, 64))
