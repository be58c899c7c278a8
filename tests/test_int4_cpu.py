"""The fp64 forms of the 4-bit cache and of the page plan pinned to bounds and invariants, and the
entry points' refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs


def _rows(shape, seed, spread=2.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape) * np.exp(r.uniform(-spread, spread, shape[:-1] + (1,))) + r.standard_normal(shape[-1])
    return torch.from_numpy(x).to(torch.bfloat16)


def test_scales_and_codes_bounds():
    x = _rows((500, 128), 1, 20.0)
    codes, z, s = plain.coded_int4(x)
    v = x.double().numpy().reshape(500, 4, 32)
    span = np.maximum(v.max(-1), 0) - np.minimum(v.min(-1), 0)
    assert np.all(15 * s >= span) and np.all(15 * s <= span * (1 + 2.0 ** -3))
    part, _ = np.frexp(s)
    assert np.array_equal(part * 16, np.round(part * 16))
    assert codes.min() >= 0 and codes.max() <= 15 and z.min() >= 0 and z.max() <= 15
    got = (codes.reshape(500, 4, 32) - z[..., None]) * s[..., None]
    assert np.all(np.abs(got - v) <= s[..., None] / 2)
    # every value is a bf16 number
    assert np.array_equal(torch.from_numpy(got).to(torch.bfloat16).double().numpy(), got)


def test_zero_and_non_finite_elements():
    x = torch.zeros(64, dtype=torch.bfloat16)
    x[3], x[5], x[7], x[9], x[40] = 3.0, float("inf"), float("-inf"), float("nan"), float("inf")
    codes, z, s = plain.coded_int4(x)
    val = (codes.reshape(2, 32) - z[:, None]) * s[:, None]
    assert val[0, 0] == 0 and abs(val[0, 3] - 3) <= s[0] / 2 and codes[5] == 15 and codes[7] == 0 and val[0, 9] == 0
    assert s[1] == 0 and not val[1].any()
    assert plain.coded_int4(torch.full((32,), 1e-32, dtype=torch.bfloat16))[2][0] == 0


def test_quotients_are_exact_ties_or_far_from_one():
    """Why x * (1 / s) + z snapped to 2^-11 rounds as the quotient does: significands of 8 and 4 bits."""
    x = np.arange(128, 256, dtype=np.float64)
    for s in range(8, 16):
        for k in range(-12, 2):
            q = x * 2.0 ** k / s
            frac = np.abs(q - np.floor(q) - 0.5)[(q >= 0.25) & (q <= 16)]
            assert np.all((frac == 0) | (frac >= 2.0 ** -11))


def test_the_layout_in_words():
    """Eight channels of a token are one little-endian word, a pair of neighbours 16 bits apart."""
    kv = np.zeros((1, 1, 2, 9, 64), dtype=np.int64)
    x = np.zeros(64)
    x[32:64] = np.arange(32) % 16  # codes of their own values: s = 1, z = 0
    plain.put_int4(kv[0, 0, 1], 5, x)
    words = kv.astype(np.uint8)[0, 0, 1, :8].reshape(-1).view("<u4").reshape(2, 16, 4)
    for run in range(4):
        w = int(words[1, 5, run])
        for pair in range(4):
            assert (w >> 4 * pair) & 0x000F000F == ((8 * run + 2 * pair) % 16) | ((8 * run + 2 * pair + 1) % 16) << 16
    scales = kv.astype(np.uint8)[0, 0, 1, 8].view("<u2").reshape(2, 16)
    assert scales[1, 5] == 0x3F80 and scales.sum() == 0x3F80
    assert np.array_equal(plain.values_int4(kv)[1][0, 0, 5], x)


def test_packed_inputs_are_what_the_append_writes():
    k, v = _rows((3, 2, 16, 64), 3), _rows((3, 2, 16, 64), 4)
    kv = inputs.pack_int4(k, v)
    rows = [t.transpose(1, 2).reshape(48, 2, 64) for t in (k, v)]
    got = plain.append_kv_int4(rows[0], rows[1], np.arange(48), np.zeros((3, 2, 2, 9, 64)))
    assert np.array_equal(kv.numpy(), got)
    k[1, 0, 4] = float("nan")
    assert np.isnan(plain.values_int4(inputs.pack_int4(k, v))[0][1, 0, 4]).any()


def test_attend_matches_the_c_oracle(oracle_mod):
    w = inputs.make_decode([0, 1, 16, 37, 90], 5, 8, 2, 64, seed=5, poison=False)
    c = w.cache
    kv = inputs.pack_int4(c.k_pages, c.v_pages)
    kb, vb = (torch.from_numpy(x).to(torch.bfloat16) for x in plain.values_int4(kv))
    for window in (0, 5):
        ro, rl = oracle_mod.decode(w.q, kb, vb, c.block_table, c.lens, w.sinks, w.scale, window=window)
        out, lse, _ = plain.attend_int4(w.q, kv, c.block_table, c.lens, w.sinks, w.scale, window=window)
        np.testing.assert_allclose(out, ro, atol=1e-12)
        np.testing.assert_allclose(lse, rl, atol=1e-12)


def test_plan_and_release_keep_every_page_once():
    r = np.random.default_rng(0)
    pages, B, cols = 60, 7, 12
    free, nfree = r.permutation(pages), pages
    lens, table = np.zeros(B, dtype=np.int64), np.full((B, cols), -1)
    for step in range(200):
        p = plain.plan_step(r.integers(0, 30, B), lens, table, free, nfree, 300)
        lens, table, nfree = p["seq_lens"], p["block_table"], p["num_free"]
        held = [table[b, c] for b in range(B) for c in range(-(-lens[b] // 16))]
        assert sorted(held + list(free[:nfree])) == list(range(pages))
        live = p["slots"][p["slots"] >= 0]
        assert len(set(live)) == len(live)
        lens, free, nfree = plain.release_pages(r.random(B) < 0.3, lens, table, free, nfree)
    p = plain.plan_step([40, 7], [0, 0], np.full((2, 4), -1), np.arange(9), 9, 64)
    again = plain.release_pages([True, True], p["seq_lens"], p["block_table"], np.arange(9), p["num_free"])
    assert list(again[1]) == list(range(9)) and again[2] == 9


# ------------------------------------------------------------------ refusals
def _host():
    buf = (ctypes.c_uint8 * 8192)()
    return buf, (ctypes.addressof(buf) + 255) // 256 * 256


def _desc(sa, **kw):
    d = dict(num_seqs=4, num_qo_heads=8, num_kv_heads=2, head_dim=64, num_pages=10, max_pages_per_seq=4)
    d.update(kw)
    return sa.paged_desc(**d)


def test_append_int4_rejects(sa):
    lib, (buf, p) = sa.load(), _host()

    def call(k=p, ks=128, v=p, vs=128, sl=p, T=8, kv=p, d=_desc(sa), ws=None, wb=0):
        return lib.sinkattn_append_kv_int4(k, ks, v, vs, sl, T, kv, None if d is None else ctypes.byref(d), ws, wb, None)
    for kw in (dict(k=None), dict(v=None), dict(sl=None), dict(kv=None), dict(d=None), dict(k=p + 8), dict(v=p + 2),
               dict(sl=p + 4), dict(kv=p + 8), dict(ks=127), dict(ks=120), dict(vs=130), dict(vs=0), dict(ks=-128),
               dict(T=-1), dict(ws=p, wb=128), dict(ws=p + 16, wb=256), dict(d=_desc(sa, num_pages=0))):
        assert call(**kw) == 1, kw
    assert call(d=_desc(sa, head_dim=96)) == 2
    assert call(T=0, k=None, v=None, sl=None) == 0


def test_unpack_int4_rejects(sa):
    lib, (buf, p) = sa.load(), _host()

    def call(kv=p, pg=p, n=3, ko=p, vo=p, d=_desc(sa), ws=None, wb=0):
        return lib.sinkattn_unpack_kv_int4(kv, pg, n, ko, vo, ctypes.byref(d), ws, wb, None)
    for kw in (dict(kv=None), dict(ko=None), dict(vo=None), dict(kv=p + 8), dict(pg=p + 2), dict(ko=p + 8), dict(n=-1),
               dict(pg=None, n=11), dict(ws=p, wb=128), dict(d=_desc(sa, num_pages=0))):
        assert call(**kw) == 1, kw
    assert call(d=_desc(sa, head_dim=32)) == 2 and call(n=0, kv=None) == 0


def test_decode_int4_rejects(sa):
    lib, (buf, p) = sa.load(), _host()

    def dec(q=p, kv=p, bt=p, sl=p, out=p, ws=p, st=None, d=_desc(sa)):
        return lib.sinkattn_decode_int4(q, kv, bt, sl, None, 0.125, out, None, ctypes.byref(d), ws, 256, st, None)
    for kw in (dict(q=None), dict(kv=None), dict(bt=None), dict(sl=None), dict(out=None), dict(ws=None), dict(kv=p + 8),
               dict(q=p + 2), dict(st=p + 2)):
        assert dec(**kw) == 1, kw
    assert dec(d=_desc(sa, num_seqs=0), q=None, kv=None) == 0
    assert dec(d=_desc(sa, head_dim=32)) == 2


def test_prefill_int4_rejects(sa):
    lib, (buf, p) = sa.load(), _host()

    def pre(q=p, k=p, v=p, cu=p, T=8, kv=p, bt=p, pl=p, out=p, ws=p, wb=256, scale=0.125, st=None, d=_desc(sa)):
        return lib.sinkattn_prefill_int4(q, k, v, cu, T, kv, bt, pl, None, scale, out, None, ctypes.byref(d), ws, wb, st,
                                         None)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(kv=None), dict(bt=None), dict(pl=None),
               dict(out=None), dict(ws=None), dict(out=p + 16), dict(T=-1), dict(kv=p + 8), dict(scale=0.0), dict(st=p + 2),
               dict(scale=float("nan")), dict(d=_desc(sa, num_pages=0))):
        assert pre(**kw) == 1, kw
    assert pre(wb=128) == 3
    assert pre(scale=float("inf")) == 1 and pre(scale=2.0 ** 80) == 2
    assert pre(d=_desc(sa, head_dim=32)) == 2
    assert pre(T=0, q=None, kv=None) == 0 and pre(d=_desc(sa, num_seqs=0), q=None) == 0
    n = ctypes.c_size_t()
    assert lib.sinkattn_prefill_int4_workspace_size(ctypes.byref(_desc(sa)), -1, ctypes.byref(n)) == 1
    assert lib.sinkattn_prefill_int4_workspace_size(ctypes.byref(_desc(sa)), 0, ctypes.byref(n)) == 0 and n.value == 256


def test_plan_and_release_reject(sa):
    lib, (buf, p) = sa.load(), _host()

    # arrays of their own, 256 bytes apart (4 requests of 4 columns, 10 pages, 8 rows)
    new, sl, bt, fr, nf, cu, lo, no, pos, slots, st = (p + 256 * i for i in range(11))

    def plan(new=new, sl=sl, bt=bt, fr=fr, nf=nf, T=8, cu=cu, st=st, lo=lo, no=no, pos=pos, slots=slots, d=_desc(sa), ws=None, wb=0):
        return lib.sinkattn_plan_step(new, sl, bt, fr, nf, T, cu, st, lo, no, pos, slots, ctypes.byref(d), ws, wb, None)

    def release(done=new, sl=sl, bt=bt, fr=fr, nf=nf, lo=lo, no=no, d=_desc(sa), ws=None, wb=0):
        return lib.sinkattn_release_pages(done, sl, bt, fr, nf, lo, no, ctypes.byref(d), ws, wb, None)
    both = [dict(sl=None), dict(bt=None), dict(fr=None), dict(nf=None), dict(lo=None), dict(no=None), dict(sl=sl + 2),
            dict(bt=bt + 2), dict(fr=fr + 1), dict(nf=nf + 2), dict(lo=lo + 2), dict(no=no + 2), dict(ws=p, wb=128),
            dict(ws=p + 16, wb=256), dict(d=_desc(sa, num_pages=0)), dict(d=_desc(sa, max_pages_per_seq=0)),
            dict(d=_desc(sa, num_seqs=-1)),
            # memory shared in other ways than the two that are allowed
            dict(lo=sl + 4), dict(no=sl), dict(lo=nf), dict(no=lo + 8), dict(lo=fr + 36), dict(fr=bt + 60)]
    for kw in both:
        assert plan(**kw) == 1, kw
        assert release(**kw) == 1, kw
    for kw in (dict(new=None), dict(cu=None), dict(pos=None), dict(slots=None), dict(T=-1), dict(pos=pos + 4),
               dict(slots=slots + 8), dict(st=sl), dict(st=lo), dict(new=new + 2), dict(cu=cu + 2), dict(cu=new), dict(pos=slots),
               dict(lo=new), dict(slots=bt), dict(cu=lo - 16), dict(bt=new)):
        assert plan(**kw) == 1, kw
    for kw in (dict(done=None), dict(done=lo + 3), dict(done=fr)):
        assert release(**kw) == 1, kw
    for call in (plan, release):
        assert call(d=_desc(sa, num_seqs=8193)) == 2
        assert call(d=_desc(sa, num_seqs=8192, max_pages_per_seq=1 << 18)) == 2


def test_binding_refuses_host_tensors(sa):
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    kv = torch.zeros(1, 2, 2, 9, 64, dtype=torch.uint8)
    for call in (lambda: sa.append_kv_int4(x, x, None, kv), lambda: sa.unpack_kv_int4(kv),
                 lambda: sa.decode_int4(x, kv, i, i), lambda: sa.prefill_int4(x, x, x, i, kv, i, i),
                 lambda: sa.plan_step(i, i, i, i, i, 1), lambda: sa.release_pages(i, i, i, i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
