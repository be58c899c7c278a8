"""Query/key preparation (sinkattn_qk_norm_rope) on the GPU against its fp64 form.

Tolerance: the result is rounded once to bf16, half a step at most (2^-8 of the value).  Before
that everything is fp32: the angle is within 1e-6 rad (2e-6 with sincos), and the norm, the
weight, the rotation and mscale are a dozen roundings of 2^-24; both move an element by at most
their relative size times the magnitude of its pair, bounded here by 4e-6 of twice the row's
largest element of the exact result (a pair's magnitude is at most sqrt(2) of that)."""
import numpy as np
import pytest
import torch

from oracle import plain
from paged_gqa_attention_head_gb300 import inputs

pytestmark = pytest.mark.gpu


def _check(got, ref, what):
    g = got.detach().double().cpu().numpy()
    assert g.shape == ref.shape
    bound = 2.0 ** -8 * np.abs(ref) + 8e-6 * np.abs(ref).max(axis=-1, keepdims=True)
    err = np.abs(g - ref)
    assert np.all(np.isfinite(g)) and np.all(err <= bound), f"{what}: worst {np.max(err - bound):.3e} over its bound"


def _rows(T, Hq, Hkv, D, seed):
    return (inputs.normal_bf16((T, Hq, D), seed, 0) * 3).to(torch.bfloat16), inputs.normal_bf16((T, Hkv, D), seed, 1)


def _positions(T, seed, top=131072):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, top, T).astype(np.int32))


def _weights(D, seed):
    r = np.random.default_rng(seed)
    return [torch.from_numpy((1 + 0.3 * r.standard_normal(D)).astype(np.float32)) for _ in range(2)]


SCALINGS = [dict(), dict(scaling="linear", factor=8.0), dict(scaling="yarn", factor=32.0),
            dict(scaling="wavelength", factor=8.0, original_context=8192, beta_fast=4.0, beta_slow=1.0)]


@pytest.mark.parametrize("heads", [(1, 1), (2, 2), (8, 2), (16, 1), (64, 8), (64, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 7, 130])
def test_shapes(sa, cuda_dev, heads, D, T):
    Hq, Hkv = heads
    q, k = _rows(T, Hq, Hkv, D, seed=T + D + Hq)
    pos, (wq, wk) = _positions(T, T), _weights(D, 3)
    for interleaved in (False, True):
        r = dict(base=10000.0, rotary_dim=D, interleaved=interleaved)
        qo, ko = sa.qk_norm_rope(q.to(cuda_dev), k.to(cuda_dev), pos.to(cuda_dev), sa.rotary_desc(**r), wq.to(cuda_dev),
                                 wk.to(cuda_dev))
        _check(qo, plain.norm_rope(q, pos, wq, rotary=r), "q")
        _check(ko, plain.norm_rope(k, pos, wk, rotary=r), "k")


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("D,R", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 80), (128, 112), (128, 128)])
@pytest.mark.parametrize("norm", [False, True])
def test_parts_and_scalings(sa, cuda_dev, scaling, D, R, norm):
    T, Hq, Hkv = 37, 8, 2
    q, k = _rows(T, Hq, Hkv, D, seed=R)
    pos, (wq, wk) = _positions(T, R, 1 << 24), _weights(D, R)
    pos[0], pos[1] = 0, (1 << 24) - 1
    for interleaved in (False, True):
        r = dict(base=150000.0, rotary_dim=R, interleaved=interleaved, **scaling)
        qo, ko = sa.qk_norm_rope(q.to(cuda_dev), k.to(cuda_dev), pos.to(cuda_dev), sa.rotary_desc(**r),
                                 wq.to(cuda_dev) if norm else None, wk.to(cuda_dev) if norm else None, eps=1e-5)
        _check(qo, plain.norm_rope(q, pos, wq if norm else None, 1e-5, r), "q")
        _check(ko, plain.norm_rope(k, pos, wk if norm else None, 1e-5, r), "k")
        if not norm:  # what does not turn is the input, bit for bit
            assert torch.equal(qo[..., R:].cpu(), q[..., R:])


def test_matches_decode_rope(sa, oracle_mod, cuda_dev):
    """The decode entry point's rotation (YaRN, whole head) is this one's."""
    q, k = _rows(64, 8, 8, 64, seed=2)
    pos = _positions(64, 5)
    r = dict(base=150000.0, rotary_dim=64, factor=32.0, scaling="yarn")
    qo, _ = sa.qk_norm_rope(q.to(cuda_dev), None, pos.to(cuda_dev), sa.rotary_desc(**r))
    _check(qo, oracle_mod.rope(q, pos.numpy(), 150000.0, 32.0), "q")


@pytest.mark.parametrize("T", [1, 33, 5001])
def test_fused_projection_rows(sa, cuda_dev, T):
    """q and k as parts of wider rows; enough tokens for the one-warp-a-token split at the largest."""
    Hq, Hkv, D = 16, 4, 64
    row = (Hq + 2 * Hkv) * D + 8
    wide = inputs.normal_bf16((T, row), 11, 0)
    pos, (wq, wk) = _positions(T, 8), _weights(D, 4)
    d = wide.to(cuda_dev)
    q, k = d[:, :Hq * D].unflatten(1, (Hq, D)), d[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    r = dict(base=10000.0, rotary_dim=32, interleaved=True)
    qo, ko = sa.qk_norm_rope(q, k, pos.to(cuda_dev), sa.rotary_desc(**r), wq.to(cuda_dev), wk.to(cuda_dev))
    _check(qo, plain.norm_rope(wide[:, :Hq * D].unflatten(1, (Hq, D)), pos, wq, rotary=r), "q")
    _check(ko, plain.norm_rope(wide[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)), pos, wk, rotary=r), "k")
    assert torch.equal(d.cpu(), wide)


def test_in_place_and_one_sided(sa, cuda_dev):
    T, Hq, Hkv, D = 50, 8, 2, 128
    q, k = _rows(T, Hq, Hkv, D, seed=21)
    pos, (wq, wk) = _positions(T, 9), _weights(D, 9)
    rot = sa.rotary_desc(10000.0, D)
    args = (pos.to(cuda_dev), rot, wq.to(cuda_dev), wk.to(cuda_dev))
    qo, ko = sa.qk_norm_rope(q.to(cuda_dev), k.to(cuda_dev), *args)
    qi, ki = q.to(cuda_dev), k.to(cuda_dev)
    a, b = sa.qk_norm_rope(qi, ki, *args, q_out=qi, k_out=ki)
    assert a is qi and b is ki and torch.equal(qi, qo) and torch.equal(ki, ko)
    only, none = sa.qk_norm_rope(q.to(cuda_dev), None, *args)
    assert none is None and torch.equal(only, qo)
    # neither a norm nor a rotation: a copy; a norm alone
    c, _ = sa.qk_norm_rope(q.to(cuda_dev), k.to(cuda_dev))
    assert torch.equal(c.cpu(), q)
    n, _ = sa.qk_norm_rope(q.to(cuda_dev), k.to(cuda_dev), q_weight=wq.to(cuda_dev))
    _check(n, plain.norm_rope(q, pos, wq), "norm alone")
    with pytest.raises(sa.SinkAttnError):
        flat = torch.zeros(2 * T * Hq * D, dtype=torch.bfloat16, device=cuda_dev)
        x = flat[:T * Hq * D].view(T, Hq, D)
        sa.qk_norm_rope(x, None, *args, q_out=flat[64:64 + T * Hq * D].view(T, Hq, D))


def test_padding_and_positions_out_of_range(sa, cuda_dev):
    T, Hq, Hkv, D = 9, 8, 2, 64
    q, k = _rows(T, Hq, Hkv, D, seed=31)
    pos = torch.tensor([5, -1, 7, 1 << 24, 0, -(1 << 31), 2, (1 << 31) - 1, 3], dtype=torch.int32)
    left = [1, 3, 5, 7]
    r = dict(base=10000.0, rotary_dim=64)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_dev)
    qo = torch.full((T, Hq, D), 42.0, dtype=torch.bfloat16, device=cuda_dev)
    ko = torch.full((T, Hkv, D), 42.0, dtype=torch.bfloat16, device=cuda_dev)
    sa.qk_norm_rope(q.to(cuda_dev), k.to(cuda_dev), pos.to(cuda_dev), sa.rotary_desc(**r), q_out=qo, k_out=ko,
                    workspace_buf=ws)
    assert sa.get_status(ws) == sa.STATUS_BAD_LENGTH
    keep = [t for t in range(T) if t not in left]
    assert torch.all(qo[left] == 42.0) and torch.all(ko[left] == 42.0)
    _check(qo[keep], plain.norm_rope(q[keep], pos[keep], rotary=r), "q")
    _check(ko[keep], plain.norm_rope(k[keep], pos[keep], rotary=r), "k")
    e, f = sa.qk_norm_rope(q[:0].to(cuda_dev), k[:0].to(cuda_dev), pos[:0].to(cuda_dev), sa.rotary_desc(**r))
    assert e.shape == (0, Hq, D) and f.shape == (0, Hkv, D)


def test_non_finite_rows_stay_alone(sa, cuda_dev):
    T, Hq, Hkv, D = 6, 8, 2, 64
    q, k = _rows(T, Hq, Hkv, D, seed=41)
    pos, (wq, wk) = _positions(T, 1), _weights(D, 1)
    r = dict(base=10000.0, rotary_dim=64)
    bad = q.clone()
    bad[2, 3, 5], bad[4, 0, 0] = float("nan"), float("inf")
    qo, _ = sa.qk_norm_rope(bad.to(cuda_dev), k.to(cuda_dev), pos.to(cuda_dev), sa.rotary_desc(**r), wq.to(cuda_dev),
                            wk.to(cuda_dev))
    ref = plain.norm_rope(q, pos, wq, rotary=r)
    ok = np.ones((T, Hq), dtype=bool)
    ok[2, 3] = ok[4, 0] = False
    g = qo.double().cpu().numpy()
    assert np.all(np.isnan(g[2, 3])) and np.isnan(g[4, 0]).any()
    err = np.abs(g[ok] - ref[ok])
    assert np.all(err <= 2.0 ** -8 * np.abs(ref[ok]) + 8e-6 * np.abs(ref[ok]).max(axis=-1, keepdims=True))


def test_captured_and_on_two_streams(sa, cuda_dev):
    T, Hq, Hkv, D = 64, 64, 8, 64
    q, k = _rows(T, Hq, Hkv, D, seed=51)
    rot = sa.rotary_desc(150000.0, 64, 32.0, "yarn")
    r = dict(base=150000.0, rotary_dim=64, factor=32.0, scaling="yarn")
    qd, kd, pd = q.to(cuda_dev), k.to(cuda_dev), _positions(T, 2).to(cuda_dev)
    sa.qk_norm_rope(qd, kd, pd, rot)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qo, ko = sa.qk_norm_rope(qd, kd, pd, rot)
    for seed in (3, 4):
        p = _positions(T, seed)
        pd.copy_(p)
        g.replay()
        torch.cuda.synchronize()
        _check(qo, plain.norm_rope(q, p, rotary=r), "replay q")
        _check(ko, plain.norm_rope(k, p, rotary=r), "replay k")
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            got.append(sa.qk_norm_rope(qd, kd, pd, rot))
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], qo) and torch.equal(got[1][0], qo) and torch.equal(got[1][1], ko)
