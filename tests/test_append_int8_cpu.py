"""The fp64 form of the INT8 append pinned to bounds it must meet, and the entry point's refusals
(no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs


def test_page_scale_bounds():
    rng = np.random.default_rng(1)
    a = np.abs(torch.from_numpy(rng.standard_normal(2000) * np.exp(rng.uniform(-20, 20, 2000))).to(torch.bfloat16)
               .double().numpy())
    s = plain.page_scale(a)
    assert np.all(s * 127 >= a) and np.all(s <= a / 127 * (1 + 2.0 ** -7))
    mant, _ = np.frexp(s)
    assert np.array_equal(mant * 256, np.round(mant * 256))
    assert plain.page_scale(np.array(127.0)) == 1.0 and plain.page_scale(np.array(0.0)) == 0.0
    assert plain.page_scale(np.array(1e-35)) == 0.0


def test_input_scales_are_the_append_scales():
    amax = torch.tensor([1.0, 127.0, 3.5, 254.0, 0.01], dtype=torch.bfloat16).float()
    assert np.array_equal(inputs.int8_scale(amax).double().numpy(), plain.page_scale(amax.double().numpy()))


def test_quotients_are_exact_ties_or_far_from_one():
    """Why x * (1 / s) snapped to 2^-11 rounds as x / s does: 8-bit significands on both sides."""
    x = np.arange(128, 256, dtype=np.float64)
    for s in range(128, 256):
        for k in range(-1, 8):
            q = x * 2.0 ** k / s
            frac = np.abs(q - np.floor(q) - 0.5)
            frac = frac[(q >= 0.25) & (q <= 127)]
            assert np.all((frac == 0) | (frac >= 2.0 ** -10))


@pytest.mark.parametrize("step", [1, 3, 16, 50])
def test_append_steps_stay_near_the_rows(step):
    """Rows appended `step` at a time: each element within half a scale for every rounding."""
    rng = np.random.default_rng(step)
    T, H, D = 50, 2, 64
    x = torch.from_numpy(rng.standard_normal((T, H, D)) * np.exp(rng.uniform(-2, 2, (T, 1, 1)))).to(torch.bfloat16)
    kp = vp = np.zeros((5, H, 16, D), np.int8)
    sc = np.full((5, H, 2), 7.0)  # stale: a page begun anew must not see it
    bt = np.array([[3, 0, 4, 1]])
    for t in range(0, T, step):
        n = min(step, T - t)
        kp, vp, sc = plain.append_kv_int8(x[t:t + n], -x[t:t + n], [0, n], bt, [t], kp, vp, sc)
    got = plain.values(kp, sc, 0)[bt[0]].transpose(0, 2, 1, 3).reshape(-1, H, D)[:T]
    assert np.array_equal(got, -plain.values(vp, sc, 1)[bt[0]].transpose(0, 2, 1, 3).reshape(-1, H, D)[:T])
    scale = sc[bt[0], :, 0].repeat(16, axis=0)[:T]
    err = np.abs(got - x.double().numpy()).max(axis=2) / scale
    rounds = 1 if step >= 16 else 16 // step + 1
    assert np.all(err <= 0.5 * rounds + 1e-9)
    assert np.all(sc[2] == 7.0)


def test_append_int8_rejects(sa):
    lib = sa.load()
    buf = (ctypes.c_uint8 * 8192)()
    p = (ctypes.addressof(buf) + 255) // 256 * 256

    def desc(**kw):
        d = dict(num_seqs=4, num_qo_heads=2, num_kv_heads=2, head_dim=64, num_pages=10, max_pages_per_seq=4)
        d.update(kw)
        return sa.paged_desc(**d)
    ok = dict(k=p, ks=128, v=p, vs=128, cu=p, T=8, bt=p, st=p, kp=p, vp=p, sc=p, d=desc(), ws=None, wb=0)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.sinkattn_append_kv_int8(a["k"], a["ks"], a["v"], a["vs"], a["cu"], a["T"], a["bt"], a["st"], a["kp"],
                                           a["vp"], a["sc"], ctypes.byref(a["d"]) if a["d"] else None, a["ws"], a["wb"],
                                           None)
    for name in ("k", "v", "cu", "bt", "st", "kp", "vp", "sc", "d"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(k=p + 8), dict(v=p + 2), dict(kp=p + 8), dict(vp=p + 8), dict(sc=p + 4), dict(cu=p + 2),
               dict(ks=127), dict(ks=120), dict(vs=130), dict(vs=0), dict(ks=-128), dict(T=-1), dict(ws=p, wb=128),
               dict(ws=p + 16, wb=256), dict(d=desc(num_pages=0)), dict(d=desc(max_pages_per_seq=0))):
        assert call(**kw) == 1, kw
    assert call(d=desc(head_dim=96)) == 2
    assert call(T=0, k=None, v=None) == 0
    assert call(d=desc(num_seqs=0), k=None) == 0


def test_binding_refuses_host_tensors(sa):
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sa.append_kv_int8(x, x, None, None, None, None, None, None)
