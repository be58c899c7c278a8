"""Plain fp64 forms of the operators around the INT8 KV cache and of the query/key preparation,
straight from their definitions in include/sinkattn.h: sequence by sequence, page by page, head by
head, in numpy doubles.  Inputs are torch tensors or numpy arrays; outputs numpy.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np

PAGE = 16


def _np(t, dtype=np.float64) -> np.ndarray:
    if hasattr(t, "detach"):
        t = t.detach().cpu()
        t = t.double().numpy() if t.is_floating_point() else t.numpy()
    return np.asarray(t, dtype=dtype)


def page_scale(amax) -> np.ndarray:
    """amax / 127 rounded up to 8 significant bits; 0 where that is below 2^-100."""
    part, power = np.frexp(np.asarray(amax, dtype=np.float64) / 127.0)
    s = np.ldexp(np.ceil(part * 256.0) / 256.0, power)
    return np.where(s < 2.0 ** -100, 0.0, s)


def _quantise(x: np.ndarray, s: np.ndarray) -> np.ndarray:
    """Codes of x [H, t, D] at scales s [H]: nearest, ties to even; infinities +-127, NaN 0."""
    safe = np.where(s > 0, s, 1.0)[:, None, None]
    with np.errstate(invalid="ignore", over="ignore"):
        c = np.where(s[:, None, None] > 0, np.clip(np.rint(x / safe), -127, 127), 0.0)
    return np.where(np.isnan(x), 0.0, c)


def append_kv_int8(k, v, cu_seqlens, block_table, start_pos, k_pages, v_pages, kv_scales):
    """The cache after the append: (k_pages, v_pages int8, kv_scales float64)."""
    rows = [_np(k), _np(v)]
    cu, bt, start = _np(cu_seqlens, np.int64), _np(block_table, np.int64), _np(start_pos, np.int64)
    pages = [_np(k_pages, np.int64).copy(), _np(v_pages, np.int64).copy()]
    scales = _np(kv_scales).copy()
    for b in range(len(start)):
        t, pos = int(cu[b]), int(start[b])
        while t < int(cu[b + 1]):
            slot, pg = pos % PAGE, int(bt[b, pos // PAGE])
            take = min(PAGE - slot, int(cu[b + 1]) - t)
            for i in range(2):
                x = rows[i][t:t + take].transpose(1, 0, 2)  # [Hkv, take, D]
                finite = np.where(np.isfinite(x), np.abs(x), 0.0)
                was = scales[pg, :, i] if slot else np.zeros(x.shape[0])
                was = np.where(was >= 2.0 ** -100, was, 0.0)
                now = np.maximum(was, page_scale(finite.max(axis=(1, 2))))
                grown = now > was
                if slot and grown.any():
                    old = pages[i][pg, grown, :slot] * was[grown][:, None, None] / now[grown][:, None, None]
                    pages[i][pg, grown, :slot] = np.rint(old).astype(np.int64)
                pages[i][pg, :, slot:slot + take] = _quantise(x, now).astype(np.int64)
                scales[pg, :, i] = now
            t, pos = t + take, pos + take
    return pages[0].astype(np.int8), pages[1].astype(np.int8), scales


def values(pages, kv_scales, which: int) -> np.ndarray:
    """A cache's K (which 0) or V (1) as numbers, [num_pages, Hkv, 16, D]."""
    return _np(pages) * _np(kv_scales)[:, :, which][:, :, None, None]


def attend_int8(q, k_pages, v_pages, kv_scales, block_table, lens, sinks, scale: float, window: int = 0,
                new: Optional[tuple] = None):
    """Attention over INT8 pages.  new None: a decode (q [B, Hq, D], lens the tokens each query
    sees).  new (k, v, cu_seqlens): a chunked prefill, lens the prefix lengths.  Returns out,
    lse, and vmax: the largest |v| that each query's head sees (for error bounds)."""
    q, bt, lens = _np(q), _np(block_table, np.int64), _np(lens, np.int64)
    hq, dim = q.shape[1:]
    hkv = k_pages.shape[1]
    group = hq // hkv
    cu = np.arange(len(lens) + 1) if new is None else _np(new[2], np.int64)
    kn, vn = (None, None) if new is None else (_np(new[0]), _np(new[1]))
    codes = [_np(k_pages), _np(v_pages)]
    sc = _np(kv_scales)
    sk = np.full(hq, -np.inf) if sinks is None else _np(sinks)
    out, lse, vmax = np.zeros(q.shape), np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    for b, held in enumerate(lens):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        if t0 == t1:
            continue
        at = bt[b, :(held + PAGE - 1) // PAGE]
        for g in range(hkv):
            kv = [(codes[i][at, g] * sc[at, g, i][:, None, None]).reshape(-1, dim)[:held] for i in range(2)]
            first = held - 1
            if new is not None:
                kv = [np.concatenate([kv[0], kn[t0:t1, g]]), np.concatenate([kv[1], vn[t0:t1, g]])]
                first = held
            j = np.arange(kv[0].shape[0])[None, :]
            pos = (first + np.arange(t1 - t0))[:, None]
            seen = j <= pos
            if window > 0:
                seen &= j > pos - window
            mag = np.abs(kv[1]).max(axis=1) if kv[1].shape[0] else np.zeros(0)
            top = np.where(seen, mag[None, :], 0.0).max(axis=1, initial=0.0)
            for h in range(g * group, (g + 1) * group):
                s = np.where(seen, (q[t0:t1, h] @ kv[0].T) * scale, -np.inf)
                m = np.maximum(s.max(axis=1, initial=-np.inf), sk[h])
                live = np.isfinite(m)
                m0 = np.where(live, m, 0.0)[:, None]
                p = np.exp(s - m0)
                den = p.sum(axis=1) + (np.exp(sk[h] - m0[:, 0]) if np.isfinite(sk[h]) else 0.0)
                out[t0:t1, h] = np.where(live[:, None], (p @ kv[1]) / np.where(den > 0, den, 1.0)[:, None], 0.0)
                with np.errstate(divide="ignore"):
                    lse[t0:t1, h] = np.where(live, m0[:, 0] + np.log(den), -np.inf)
                vmax[t0:t1, h] = top
    return out, lse, vmax


def rotary_rates(base: float, rotary_dim: int, factor: float = 1.0, scaling: str = "none",
                 original_context: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(theta [rotary_dim / 2], mscale)."""
    n = rotary_dim
    theta, mscale = np.empty(n // 2), 1.0
    for i in range(n // 2):
        w = base ** (-2.0 * i / n)
        if scaling == "linear":
            w = w / factor
        elif scaling == "yarn":
            c = [n * math.log(original_context / (2 * math.pi * r)) / (2 * math.log(base))
                 for r in (beta_fast, beta_slow)]
            lo, hi = max(0, math.floor(c[0])), min(n - 1, math.ceil(c[1]))
            y = min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
            w, mscale = (1 - y) * w + y * w / factor, 1 + 0.1 * math.log(factor)
        elif scaling == "wavelength":
            turns = original_context * w / (2 * math.pi)
            y = min(1.0, max(0.0, (beta_fast - turns) / (beta_fast - beta_slow)))
            w = (1 - y) * w + y * w / factor
        theta[i] = w
    return theta, mscale


def norm_rope(x, positions, weight=None, eps: float = 1e-6, rotary: Optional[dict] = None) -> np.ndarray:
    """One tensor [T, H, D] through the norm (weight given) and the rotation (rotary: the
    arguments of sinkattn.rotary_desc)."""
    x = _np(x).copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * _np(weight)
    if rotary is None:
        return x
    r = dict(rotary)
    inter = r.pop("interleaved", False)
    theta, ms = rotary_rates(**r)
    n = r["rotary_dim"]
    ang = _np(positions, np.float64)[:, None] * theta[None, :]
    co, si = (np.cos(ang) * ms)[:, None, :], (np.sin(ang) * ms)[:, None, :]
    ia, ib = (np.arange(0, n, 2), np.arange(1, n, 2)) if inter else (np.arange(n // 2), np.arange(n // 2, n))
    a, b = x[..., ia], x[..., ib]
    y = x.copy()
    y[..., ia], y[..., ib] = a * co - b * si, b * co + a * si
    return y
