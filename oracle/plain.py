"""Plain fp64 forms of the operators around the INT8 and the 4-bit KV cache, of the page plan and of
the query/key preparation, straight from their definitions in include/sinkattn.h: sequence by sequence, page by page, head by
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


def coded_int4(x):
    """Codes [..., D], z and s [..., D / 32] of rows x [..., D] in a 4-bit cache."""
    x = _np(x)
    x = x.reshape(*x.shape[:-1], -1, 32)
    fin = np.where(np.isfinite(x), x, 0.0)
    low, high = np.minimum(fin.min(axis=-1), 0.0), np.maximum(fin.max(axis=-1), 0.0)
    part, power = np.frexp((high - low) / 15.0)
    s = np.ldexp(np.ceil(part * 16.0) / 16.0, power)
    s = np.where(s < 2.0 ** -100, 0.0, s)
    by = np.where(s > 0, s, 1.0)
    z = np.where(s > 0, np.rint(-low / by), 0.0)
    with np.errstate(invalid="ignore"):
        codes = np.clip(np.rint(x / by[..., None] + z[..., None]), 0, 15)
    codes = np.where(np.isnan(x), z[..., None], codes)
    codes = np.where(s[..., None] > 0, codes, 0.0)
    return codes.reshape(*codes.shape[:-2], -1).astype(np.int64), z.astype(np.int64), s


def _word_int4(s, z):
    """The 16-bit word of a group: the upper half of s as a float, z in its low bits."""
    return (np.asarray(s, dtype=np.float32).view(np.uint32) >> 16).astype(np.int64) | z


def put_int4(rec, tok: int, x) -> None:
    """Row x [D] into place tok of one (page, head)'s K or V, bytes rec [9, D], in place."""
    flat, dim = rec.reshape(-1), rec.shape[-1]
    codes, z, s = coded_int4(x)
    for c in range(dim):
        i, e = c % 32 // 8, c % 8
        bit = 4 * (e // 2) + 16 * (e % 2)
        at = (c // 32 * PAGE + tok) * 16 + 4 * i + bit // 8
        flat[at] = (flat[at] & ~(15 << bit % 8)) | (int(codes[c]) << bit % 8)
    for g, w in enumerate(_word_int4(s, z)):
        at = 8 * dim + (g * PAGE + tok) * 2
        flat[at], flat[at + 1] = w & 255, w >> 8


def append_kv_int4(k, v, slots, kv_pages) -> np.ndarray:
    """The bytes of the cache after the append."""
    out = _np(kv_pages, np.int64).copy()
    rows = [_np(k), _np(v)]
    for t, slot in enumerate(_np(slots, np.int64)):
        if 0 <= slot < out.shape[0] * PAGE:
            for h in range(out.shape[1]):
                for i in range(2):
                    put_int4(out[slot // PAGE, h, i], int(slot % PAGE), rows[i][t, h])
    return out.astype(np.uint8)


def values_int4(kv_pages) -> list:
    """A 4-bit cache's K and V as numbers, each [num_pages, Hkv, 16, D]."""
    raw = _np(kv_pages, np.int64)
    n, h, _, _, dim = raw.shape
    flat = raw.reshape(n, h, 2, 9 * dim)
    tok = np.arange(PAGE)
    out = np.empty((2, n, h, PAGE, dim))
    for c in range(dim):
        i, e = c % 32 // 8, c % 8
        bit = 4 * (e // 2) + 16 * (e % 2)
        row = c // 32 * PAGE + tok
        code = (flat[..., row * 16 + 4 * i + bit // 8] >> bit % 8) & 15
        word = flat[..., 8 * dim + 2 * row] | flat[..., 8 * dim + 2 * row + 1] << 8
        s = ((word & 0xFFF0) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        out[..., c] = np.moveaxis((code - (word & 15)) * s, 2, 0)
    return [out[0], out[1]]


def attend_int4(q, kv_pages, block_table, lens, sinks, scale: float, window: int = 0, new: Optional[tuple] = None):
    """attend_int8 over the pages of a 4-bit cache."""
    k, v = values_int4(kv_pages)
    return attend_int8(q, k, v, np.ones((*k.shape[:2], 2)), block_table, lens, sinks, scale, window, new)


def plan_step(new_lens, seq_lens, block_table, free_pages, num_free: int, max_tokens: int) -> dict:
    """A step's plan, request by request: the list of free pages is a stack, taken from its top."""
    new, lens, table = _np(new_lens, np.int64), _np(seq_lens, np.int64), _np(block_table, np.int64).copy()
    free, num_pages = _np(free_pages, np.int64), len(free_pages)
    room = table.shape[1] * PAGE
    pos, slots = np.full(max_tokens, -1), np.full(max_tokens, -1)
    cu, after, t, short, long, bad = [0], [], 0, False, False, False
    left, wanted = num_free, 0
    for b, (n, have) in enumerate(zip(new, lens)):
        long |= n < 0
        n = max(int(n), 0)
        fits, rows = have >= 0 and have + n <= room, n == 0 or t + n <= max_tokens
        long |= not (fits and rows)
        first, last = -(-have // PAGE), -(-(have + n) // PAGE)
        need = int(last - first) if fits else 0
        wanted += need
        served = bool(fits and rows and (need == 0 or wanted <= num_free))
        short |= bool(fits and rows and not served)
        if served:
            for c in range(first, last):
                left -= 1
                table[b, c] = free[left]
            for i in range(n):
                p = have + i
                pg = table[b, p // PAGE]
                pos[t + i] = p
                if 0 <= pg < num_pages:
                    slots[t + i] = pg * PAGE + p % PAGE
                else:
                    bad = True
        after.append(have + n if served else have)
        t += n
        cu.append(min(t, max_tokens))
    return dict(cu_seqlens=np.array(cu), start_pos=lens, seq_lens=np.array(after), positions=pos, slots=slots,
                num_free=left, block_table=table, short=short, long=long, bad=bad)


def release_pages(done, seq_lens, block_table, free_pages, num_free: int):
    """Lengths, list and its size once the requests that are done have given their pages back."""
    lens, table, free = _np(seq_lens, np.int64).copy(), _np(block_table, np.int64), _np(free_pages, np.int64).copy()
    back = [table[b, c] for b in range(len(lens)) if done[b] for c in range(-(-lens[b] // PAGE))]
    free[num_free:num_free + len(back)] = back[::-1]
    lens[np.asarray(done, dtype=bool)] = 0
    return lens, free, num_free + len(back)


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
