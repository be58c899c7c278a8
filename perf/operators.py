"""Cases for the operators around an INT8 paged KV cache, and for the query/key preparation
before attention: what each one computes in plain torch, the calls of this library that compute
the same, the work of a pass and its result in 64 bits.

  rotate   per-head RMS norm of queries and keys with the position rotation in the same pass
  append   new K/V rows quantised into INT8 pages, one scale for each page and KV head
  decode   one query token per sequence over such a cache
  prefill  a chunk of new tokens over a prefix held in such a cache
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"
MAX_POS = 131072


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence's next token, gpt-oss heads, YaRN positions, no norm: latency
        dict(name="rotate_one_token", op="rotate", tokens=1, heads=64, kv_heads=8, dim=64, norm=False,
             rotary=64, interleaved=False, scaling="yarn", base=150000.0, factor=32.0),
        # a decode batch with normalised queries and keys, Qwen3-shape heads
        dict(name="rotate_decode_batch", op="rotate", tokens=128, heads=64, kv_heads=4, dim=128, norm=True,
             rotary=128, interleaved=False, scaling="none", base=1000000.0, factor=1.0),
        # a ragged prefill step: half of each head rotated, neighbours paired, odd token count
        dict(name="rotate_prefill", op="rotate", tokens=16381, heads=64, kv_heads=8, dim=64, norm=True,
             rotary=32, interleaved=True, scaling="linear", base=10000.0, factor=4.0),
        # a decode step's append: one token for each of 64 sequences, most in the middle of a page
        dict(name="append_decode_batch", op="append", seqs=64, new_lo=1, new_hi=1, start_lo=512, start_hi=8192,
             kv_heads=8, dim=64),
        # a mixed step: chunks and single tokens of Qwen3-shape heads, ragged starts
        dict(name="append_mixed", op="append", seqs=37, new_lo=1, new_hi=300, start_lo=0, start_hi=1000,
             kv_heads=4, dim=128),
        # the gpt-oss prefill batch's rows into empty pages and over page ends
        dict(name="append_prefill", op="append", seqs=4, new_lo=512, new_hi=4096, start_lo=0, start_hi=40,
             kv_heads=8, dim=64),
        # one user's next token: few rows, a medium context
        dict(name="decode_one", op="decode", seqs=1, len_lo=4097, len_hi=4097, log=False, heads=64, kv_heads=8,
             dim=64, window=0, sinks=True),
        # the Qwen3-shape batch: 16 query heads on each KV head, no sinks
        dict(name="decode_batch", op="decode", seqs=64, len_lo=1, len_hi=16384, log=False, heads=64, kv_heads=4,
             dim=128, window=0, sinks=False),
        # a long-context mix, gpt-oss heads
        dict(name="decode_long", op="decode", seqs=64, len_lo=128, len_hi=131072, log=True, heads=64, kv_heads=8,
             dim=64, window=0, sinks=True),
        # a short follow-up question over a cached conversation
        dict(name="prefill_short", op="prefill", seqs=1, new_lo=17, new_hi=17, pre_lo=1003, pre_hi=1003, heads=64,
             kv_heads=8, dim=64, window=0, sinks=True),
        # ragged chunks and prefixes (some empty) at head_dim 128
        dict(name="prefill_ragged", op="prefill", seqs=7, new_lo=1, new_hi=700, pre_lo=0, pre_hi=5000, heads=16,
             kv_heads=8, dim=128, window=0, sinks=False),
        # the long-context chunked prefill: 8 chunks of 512 tokens over 16384-token prefixes
        dict(name="prefill_long", op="prefill", seqs=8, new_lo=512, new_hi=512, pre_lo=16384, pre_hi=16384,
             heads=64, kv_heads=8, dim=64, window=0, sinks=True),
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "decode", "prefill"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8] if dim == 64 else [1, 2, 4])
    group = rng.choice([1, 2, 4, 8, 16])
    heads = min(64, kv_heads * group)
    if op == "rotate":
        scaling = rng.choice(["none", "linear", "yarn", "wavelength"])
        return dict(op=op, tokens=_log(rng, 1, 16000), heads=heads, kv_heads=kv_heads, dim=dim,
                    norm=rng.random() < 0.7, rotary=rng.choice(range(16, dim + 1, 16)),
                    interleaved=rng.random() < 0.5, scaling=scaling,
                    base=round(math.exp(rng.uniform(math.log(1e4), math.log(1e6))), 1),
                    factor=1.0 if scaling == "none" else round(rng.uniform(1.5, 40.0), 2))
    if op == "append":
        seqs = _log(rng, 1, 128)
        lo = rng.choice([0, 1])
        hi = max(1, _log(rng, 1, max(2, 8000 // seqs)))
        return dict(op=op, seqs=seqs, new_lo=min(lo, hi), new_hi=hi, start_lo=0, start_hi=_log(rng, 1, 8192),
                    kv_heads=kv_heads, dim=dim)
    window = rng.choice([0, 0, 0, _log(rng, 1, 5000)])
    if op == "decode":
        seqs = _log(rng, 1, 100)
        hi = _log(rng, 1, min(131072, 2000000 // seqs))
        log = rng.random() < 0.5 and hi > 16
        return dict(op=op, seqs=seqs, len_lo=min(hi, 16) if log else rng.choice([0, 1, hi // 2]), len_hi=hi, log=log,
                    heads=heads, kv_heads=kv_heads, dim=dim, window=window, sinks=rng.random() < 0.5)
    seqs = _log(rng, 1, 8)
    new = _log(rng, 1, 512)
    pre = _log(rng, 1, 16384)
    return dict(op=op, seqs=seqs, new_lo=rng.choice([0, 1, new]) if seqs > 1 else new, new_hi=new,
                pre_lo=rng.choice([0, 0, pre // 2, pre]), pre_hi=pre, heads=heads, kv_heads=kv_heads, dim=dim,
                window=window, sinks=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _ints(n, lo, hi, log=False, key=0):
    """Lengths of a case: they belong to the case, not to the seed, so that its work is known.
    The first is the range's top, so that every range is covered."""
    r = np.random.default_rng([n, lo, hi, int(log), key])
    v = np.exp(r.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)), n)).round() if log else r.integers(lo, hi + 1, n)
    v = np.clip(v.astype(np.int64), lo, hi)
    v[0] = hi
    return [int(x) for x in v]


def _lens(case):
    if case["op"] == "append":
        return (_ints(case["seqs"], case["new_lo"], case["new_hi"], key=1),
                _ints(case["seqs"], case["start_lo"], case["start_hi"], key=2))
    if case["op"] == "decode":
        return _ints(case["seqs"], case["len_lo"], case["len_hi"], case["log"], key=3)
    return (_ints(case["seqs"], case["new_lo"], case["new_hi"], key=4),
            _ints(case["seqs"], case["pre_lo"], case["pre_hi"], key=5))


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _gen(seed, key):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + key)


def _rows(shape, g, dim):
    """K or V rows: a standard deviation of its own for each channel, as a model's have."""
    ch = torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV))
    return torch.randn(shape, generator=g, device=DEV) * ch


def _scale_of(most):
    """The scale of a block whose largest magnitude is `most`: most / 127, rounded up to 8 significant
    bits, so that quotients of bf16 values by it are never within a rounding error of a tie."""
    bits = (most / 127.0).view(torch.int32)
    return ((bits + 0xFFFF) & -65536).view(torch.float32)


def _quantised(x):
    """Pages [n, Hkv, 16, D] as codes and scales [n, Hkv]."""
    s = _scale_of(x.abs().amax(dim=(2, 3)))
    return torch.round(x / s[:, :, None, None]).clamp_(-127, 127).to(torch.int8), s


def _cache(npages, kv_heads, dim, g):
    npages = max(npages, 1)
    k, ks = _quantised(_rows((npages, kv_heads, PAGE, dim), g, dim))
    v, vs = _quantised(_rows((npages, kv_heads, PAGE, dim), g, dim))
    return k, v, torch.stack([ks, vs], dim=-1).contiguous()


def _table(pages_of, npages, g, columns=None):
    """Block table over a shuffled pool; unused columns -1."""
    perm = torch.randperm(max(npages, 1), generator=g, device=DEV).to(torch.int32).cpu().numpy()
    columns = columns or max(1, max(pages_of))
    t = np.full((len(pages_of), columns), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages_of):
        t[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t).to(DEV)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rotary(case):
    scaling = case["scaling"]
    fast, slow = (32.0, 1.0) if scaling == "yarn" else (4.0, 1.0)
    return dict(base=case["base"], factor=case["factor"], scaling=scaling, original_context=4096, beta_fast=fast,
                beta_slow=slow, rotary_dim=case["rotary"], interleaved=case["interleaved"])


def prepare(case, seed):
    g = _gen(seed, 1)
    op, dim, hkv = case["op"], case["dim"], case["kv_heads"]
    s = dict(case=case, op=op)
    if op == "rotate":
        T, hq = case["tokens"], case["heads"]
        # one row holds a token's queries, keys and values, as a fused projection writes them
        qkv = torch.randn(T, (hq + 2 * hkv) * dim, generator=g, device=DEV).mul_(2.0).to(torch.bfloat16)
        s["q"] = qkv[:, :hq * dim].unflatten(1, (hq, dim))
        s["k"] = qkv[:, hq * dim:(hq + hkv) * dim].unflatten(1, (hkv, dim))
        if T <= 256:
            s["positions"] = torch.randint(0, MAX_POS, (T,), generator=g, device=DEV, dtype=torch.int32)
        else:  # chunks of sequences that start anywhere
            chunk = torch.arange(T, device=DEV) // 1021
            start = torch.randint(0, MAX_POS - 1021, (int(T // 1021) + 1,), generator=g, device=DEV)
            s["positions"] = (start[chunk] + torch.arange(T, device=DEV) % 1021).to(torch.int32)
        s["rotary"] = _rotary(case)
        s["wq"] = 1.0 + 0.2 * torch.randn(dim, generator=g, device=DEV) if case["norm"] else None
        s["wk"] = 1.0 + 0.2 * torch.randn(dim, generator=g, device=DEV) if case["norm"] else None
        s["eps"] = 1e-6
        if own:
            from paged_gqa_attention_head_gb300 import sinkattn
            s["desc"] = sinkattn.rotary_desc(**s["rotary"])
        return s
    if op == "append":
        new, start = _lens(case)
        # the pool holds the pages that this step writes to (a sequence's earlier pages are not touched)
        first = [p // PAGE for p in start]
        own_pages = [_pages(p + n) - f if n else 0 for p, n, f in zip(start, new, first)]
        npages = sum(own_pages) + 2
        s["k_pages"], s["v_pages"], s["scales"] = _cache(npages, hkv, dim, g)
        cols = max(1, max(_pages(p + n) for p, n in zip(start, new)))
        compact = _table(own_pages, npages, g).cpu().numpy()
        table = np.full((len(new), cols), -1, dtype=np.int32)
        for b, (f, n) in enumerate(zip(first, own_pages)):
            table[b, f:f + n] = compact[b, :n]
        s["table"] = torch.from_numpy(table).to(DEV)
        T = sum(new)
        qkv = torch.cat([_rows((T, hkv, dim), g, dim), _rows((T, hkv, dim), g, dim)], dim=1).to(torch.bfloat16)
        s["k"], s["v"] = qkv[:, :hkv].contiguous(), qkv[:, hkv:]  # the rotated keys, the projection's values
        s["cu"] = _i32(np.concatenate([[0], np.cumsum(new)]).tolist())
        s["start"] = _i32(start)
        # the plain form's plan: the touched pages, and for each of their slots the token it gets
        page, tok, keep = [], [], []
        t0 = 0
        for b, (p, n) in enumerate(zip(start, new)):
            for c in range(p // PAGE, _pages(p + n) if n else 0):
                page.append(int(table[b, c]))
                at = np.arange(PAGE) + c * PAGE
                tok.append(np.where((at >= p) & (at < p + n), at - p + t0, -1))
                keep.append(at < p)
            t0 += n
        s["page"] = torch.tensor(page, dtype=torch.int64, device=DEV)
        s["tok"] = torch.from_numpy(np.array(tok).reshape(-1, PAGE)).to(DEV)
        s["keep"] = torch.from_numpy(np.array(keep, dtype=bool).reshape(-1, PAGE)).to(DEV)
        return s
    hq = case["heads"]
    s["sinks"] = torch.randn(hq, generator=g, device=DEV) if case["sinks"] else None
    s["scale"] = 1.0 / math.sqrt(dim)
    if op == "decode":
        lens = _lens(case)
    else:
        new, lens = _lens(case)
    used = [_pages(n) for n in lens]
    npages = sum(used) + max(1, sum(used) // 20)  # some pages of the pool belong to nobody
    s["k_pages"], s["v_pages"], s["scales"] = _cache(npages, hkv, dim, g)
    s["table"] = _table(used, npages, g)
    s["lens"] = _i32(lens)
    T = len(lens) if op == "decode" else sum(new)
    s["q"] = torch.randn(T, hq, dim, generator=g, device=DEV).to(torch.bfloat16)
    if op == "prefill":
        s["k"] = _rows((T, hkv, dim), g, dim).to(torch.bfloat16)
        s["v"] = _rows((T, hkv, dim), g, dim).to(torch.bfloat16)
        cu = np.concatenate([[0], np.cumsum(new)])
        s["cu"] = _i32(cu.tolist())
        s["most"] = max(new)
        # the plain form's plan: each token's request and place in it
        s["req"] = torch.from_numpy(np.repeat(np.arange(len(new)), new)).to(DEV)
        s["at"] = torch.from_numpy(np.arange(T) - np.repeat(cu[:-1], new)).to(DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _theta(r):
    """The rate of each pair (its turn for one position), in 64 bits."""
    n, base = r["rotary_dim"], r["base"]
    i = torch.arange(n // 2, dtype=torch.float64, device=DEV)
    w = base ** (-2.0 * i / n)
    if r["scaling"] == "linear":
        return w / r["factor"], 1.0
    if r["scaling"] == "yarn":
        dim_of = lambda turns: n * math.log(r["original_context"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0.0, math.floor(dim_of(r["beta_fast"]))), min(n - 1.0, math.ceil(dim_of(r["beta_slow"])))
        y = ((i - lo) / max(0.001, hi - lo)).clamp(0, 1)
        return w * (1 - y) + w / r["factor"] * y, 1.0 + 0.1 * math.log(r["factor"])
    if r["scaling"] == "wavelength":
        turns = r["original_context"] * w / (2 * math.pi)  # of the pair over the original context
        y = ((turns - r["beta_slow"]) / (r["beta_fast"] - r["beta_slow"])).clamp(0, 1)
        return w * y + w / r["factor"] * (1 - y), 1.0
    return w, 1.0


def _plain_rotate(x, weight, s):
    r = s["rotary"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight
    theta, ms = _theta(r)
    angle = s["positions"].double()[:, None] * theta
    c, d = (torch.cos(angle) * ms).float()[:, None, :], (torch.sin(angle) * ms).float()[:, None, :]
    n = r["rotary_dim"]
    if r["interleaved"]:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack([a * c - b * d, b * c + a * d], dim=-1).flatten(-2)
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        turned = torch.cat([a * c - b * d, b * c + a * d], dim=-1)
    return torch.cat([turned, x[..., n:]], dim=-1).to(torch.bfloat16)


def _plain_append(x, pages, scales, s):
    """New rows [T, Hkv, D] into `pages`, their scales [num_pages, Hkv] with them, in place."""
    page, tok, keep = s["page"], s["tok"], s["keep"]
    live = tok >= 0
    rows = x[tok.clamp(min=0)].float().transpose(1, 2) * live[:, None, :, None]  # [touched, Hkv, 16, D]
    cand = _scale_of(rows.abs().amax(dim=(2, 3)))
    before = torch.where(keep.any(1)[:, None], scales[page], 0.0)
    after = torch.maximum(before, cand)
    by = torch.where(after > 0, after, 1.0)[:, :, None, None]
    codes = torch.round(rows / by).clamp(-127, 127)
    old = pages[page].float()
    moved = torch.where((after > before)[:, :, None, None], torch.round(old * before[:, :, None, None] / by), old)
    put = torch.where(live[:, None, :, None], codes, torch.where(keep[:, None, :, None], moved, old))
    pages[page] = put.to(torch.int8)
    scales[page] = after


def _rows_of(pages, scale, table):
    """Every table row's tokens in 32 bits: [B, Hkv, 16 * columns, D]."""
    at = table.clamp(min=0).long()
    x = pages[at].float() * scale[at][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _softmax_sum(scores, v, sinks):
    """scores [B, Hkv, G, Q, K] (hidden keys -inf), v [B, Hkv, K, D], sinks [Hkv, G] or None."""
    m = scores.amax(-1, keepdim=True)
    if sinks is not None:
        m = torch.maximum(m, sinks[None, :, :, None, None])
    zero = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = scores.sub_(zero).exp_()
    den = p.sum(-1, keepdim=True)
    if sinks is not None:
        den = den + torch.exp(sinks[None, :, :, None, None] - zero)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, p.shape[2:4]) / torch.where(den > 0, den, torch.ones_like(den))
    return out, (zero + torch.log(den)).squeeze(-1)


def _plain_attend(s):
    case = s["case"]
    hkv, dim = case["kv_heads"], case["dim"]
    group = case["heads"] // hkv
    sinks = None if s["sinks"] is None else s["sinks"].view(hkv, group)
    k = _rows_of(s["k_pages"], s["scales"][..., 0], s["table"])
    v = _rows_of(s["v_pages"], s["scales"][..., 1], s["table"])
    key = torch.arange(k.shape[2], device=DEV)
    lens = s["lens"].long()
    decode = s["op"] == "decode"
    if decode:
        q = s["q"].float().view(-1, hkv, group, 1, dim)
        pos = lens[:, None] - 1  # [B, 1]
        hidden = key[None, None, :] >= lens[:, None, None]
        kpos = key[None, None, :]
    else:
        n, most = lens.shape[0], s["most"]
        q = torch.zeros(n, most, case["heads"], dim, device=DEV)
        q[s["req"], s["at"]] = s["q"].float()
        q = q.view(n, most, hkv, group, dim).permute(0, 2, 3, 1, 4)
        kn = torch.zeros(n, most, hkv, dim, device=DEV)
        vn = torch.zeros(n, most, hkv, dim, device=DEV)
        kn[s["req"], s["at"]] = s["k"].float()
        vn[s["req"], s["at"]] = s["v"].float()
        k, v = torch.cat([k, kn.transpose(1, 2)], dim=2), torch.cat([v, vn.transpose(1, 2)], dim=2)
        t = torch.arange(most, device=DEV)
        pos = lens[:, None] + t  # [n, most]
        held = key.shape[0]
        kpos = torch.cat([key.expand(n, -1), lens[:, None] + t], dim=1)[:, None, :]  # [n, 1, K]
        hidden = torch.cat([(key[None, :] >= lens[:, None]).expand(n, held), torch.zeros(n, most, dtype=torch.bool, device=DEV)], dim=1)
        hidden = hidden[:, None, :] | (kpos > pos[:, :, None])
    if case["window"] > 0:
        hidden = hidden | (kpos <= pos[:, :, None] - case["window"])
    scores = torch.matmul((q * s["scale"]).flatten(2, 3), k.transpose(2, 3)).unflatten(2, (group, -1))
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    out, lse = _softmax_sum(scores, v, sinks)
    if decode:
        return out.flatten(1, 2).squeeze(2).to(torch.bfloat16), lse.flatten(1, 3)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["req"], s["at"]]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[s["req"], s["at"]]
    return out.to(torch.bfloat16), lse


def run(s):
    op = s["op"]
    if own:
        from paged_gqa_attention_head_gb300 import sinkattn
        if op == "rotate":
            return sinkattn.qk_norm_rope(s["q"], s["k"], s["positions"], s["desc"], q_weight=s["wq"], k_weight=s["wk"],
                                         eps=s["eps"])
        if op == "append":
            sinkattn.append_kv_int8(s["k"], s["v"], s["cu"], s["table"], s["start"], s["k_pages"], s["v_pages"], s["scales"])
        elif op == "decode":
            return sinkattn.decode_int8(s["q"], s["k_pages"], s["v_pages"], s["scales"], s["table"], s["lens"],
                                        sinks=s["sinks"], scale=s["scale"], window=s["case"]["window"])
        else:
            return sinkattn.prefill_int8(s["q"], s["k"], s["v"], s["cu"], s["k_pages"], s["v_pages"], s["scales"],
                                         s["table"], s["lens"], sinks=s["sinks"], scale=s["scale"],
                                         window=s["case"]["window"])
    elif op == "rotate":
        return _plain_rotate(s["q"], s["wq"], s), _plain_rotate(s["k"], s["wk"], s)
    elif op == "append":
        _plain_append(s["k"], s["k_pages"], s["scales"][..., 0], s)
        _plain_append(s["v"], s["v_pages"], s["scales"][..., 1], s)
    else:
        return _plain_attend(s)
    # the cache as the values it stands for
    return (s["k_pages"] * s["scales"][..., 0, None, None], s["v_pages"] * s["scales"][..., 1, None, None])


# ------------------------------------------------------------------ work
def _pairs(new, pre, window):
    n = 0
    for a, p in zip(new, pre):
        seen = np.arange(p + 1, p + a + 1, dtype=np.int64)
        n += int((np.minimum(seen, window) if window > 0 else seen).sum())
    return n


def work(case):
    dim, hkv = case["dim"], case["kv_heads"]
    if case["op"] == "rotate":
        rows = case["tokens"] * (case["heads"] + hkv)
        return {"bytes": rows * dim * 4 + case["tokens"] * 4, "flops": rows * (3 * case["rotary"] + (4 * dim if case["norm"] else 0))}
    if case["op"] == "append":
        new, start = _lens(case)
        pages = sum(_pages(p + n) - p // PAGE for p, n in zip(start, new) if n) + 2
        values = 2 * pages * hkv * PAGE * dim  # of the pool: codes read, values written
        return {"bytes": 2 * sum(new) * hkv * dim * 3 + values * 5 + pages * hkv * 8, "flops": 4 * 2 * sum(new) * hkv * dim}
    if case["op"] == "decode":
        lens = [min(n, case["window"]) if case["window"] > 0 else n for n in _lens(case)]
        return {"bytes": sum(lens) * 2 * hkv * dim + sum(_pages(n) for n in lens) * hkv * 8 + case["seqs"] * case["heads"] * (dim * 4 + 4),
                "flops": 4 * dim * case["heads"] * sum(lens)}
    new, pre = _lens(case)
    seen = [min(p, case["window"] + a) if case["window"] > 0 else p for a, p in zip(new, pre) if a]
    return {"bytes": sum(seen) * 2 * hkv * dim + sum(_pages(n) for n in seen) * hkv * 8
            + sum(new) * (case["heads"] * (dim * 4 + 4) + 2 * hkv * dim * 2),
            "flops": 4 * dim * case["heads"] * _pairs(new, pre, case["window"])}


# ------------------------------------------------------------------ 64 bits
def _exact_rotate(x, weight, s):
    r, case = s["rotary"], s["case"]
    x = x.double().cpu().numpy()
    p = s["positions"].cpu().numpy().astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / x.shape[-1] + s["eps"]) * weight.double().cpu().numpy()
    y = x.copy()
    n, f, ms = r["rotary_dim"], r["factor"], 1.0
    for i in range(n // 2):
        w = math.exp(-2.0 * i / n * math.log(r["base"]))
        if case["scaling"] == "linear":
            w /= f
        elif case["scaling"] == "yarn":
            place = [n * math.log(4096 / (2 * math.pi * b)) / (2 * math.log(r["base"])) for b in (32.0, 1.0)]
            lo, hi = max(0, math.floor(place[0])), min(n - 1, math.ceil(place[1]))
            ramp = min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
            w, ms = (1 - ramp) * w + ramp * w / f, 1 + 0.1 * math.log(f)
        elif case["scaling"] == "wavelength":
            length = 2 * math.pi / w
            if length > 4096 / 1.0:
                w /= f
            elif length >= 4096 / 4.0:
                part = (4096 / length - 1.0) / (4.0 - 1.0)
                w = (1 - part) * w / f + part * w
        i0, i1 = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + n // 2)
        co, si = (np.cos(p * w) * ms)[:, None], (np.sin(p * w) * ms)[:, None]
        y[..., i0], y[..., i1] = x[..., i0] * co - x[..., i1] * si, x[..., i0] * si + x[..., i1] * co
    return torch.from_numpy(y)


def _exact_append(x, pages, scales, s):
    """Sequence by sequence and page by page, from the definition."""
    x, pages = x.double().cpu().numpy(), pages.cpu().numpy().astype(np.float64)
    scales, table = scales.double().cpu().numpy().copy(), s["table"].cpu().numpy()
    cu, start = s["cu"].cpu().numpy(), s["start"].cpu().numpy()
    for b in range(len(start)):
        t, end = int(cu[b]), int(cu[b + 1])
        pos = int(start[b])
        while t < end:
            slot, pg = pos % PAGE, int(table[b, pos // PAGE])
            take = min(PAGE - slot, end - t)
            rows = x[t:t + take].transpose(1, 0, 2)
            was = scales[pg] if slot else np.zeros_like(scales[pg])
            part, power = np.frexp(np.abs(rows).max(axis=(1, 2)) / 127)
            now = np.maximum(was, np.ldexp(np.ceil(part * 256) / 256, power))  # 8 significant bits, upwards
            grown = now > was
            pages[pg, grown, :slot] = np.rint(pages[pg, grown, :slot] * was[grown][:, None, None] / now[grown][:, None, None])
            pages[pg, :, slot:slot + take] = np.clip(np.rint(rows / np.where(now > 0, now, 1)[:, None, None]), -127, 127)
            scales[pg] = now
            t, pos = t + take, pos + take
    return torch.from_numpy(pages * scales[:, :, None, None])


def _exact_attend(s):
    case = s["case"]
    hkv, dim, hq = case["kv_heads"], case["dim"], case["heads"]
    group, window = hq // hkv, case["window"]
    lens = s["lens"].tolist()
    cu = list(range(len(lens) + 1)) if s["op"] == "decode" else s["cu"].tolist()
    out = torch.zeros(cu[-1], hq, dim, dtype=torch.float64, device=DEV)
    lse = torch.full((cu[-1], hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, held in enumerate(lens):
        at = s["table"][b, :_pages(held)].long()
        rows = slice(cu[b], cu[b + 1])
        if cu[b] == cu[b + 1]:
            continue
        for h in range(hkv):
            k = (s["k_pages"][at, h].double() * s["scales"][at, h, 0].double()[:, None, None]).reshape(-1, dim)[:held]
            v = (s["v_pages"][at, h].double() * s["scales"][at, h, 1].double()[:, None, None]).reshape(-1, dim)[:held]
            first = held - 1  # position of the first query
            if s["op"] == "prefill":
                k, v, first = torch.cat([k, s["k"][rows, h].double()]), torch.cat([v, s["v"][rows, h].double()]), held
            ahead = torch.arange(k.shape[0], device=DEV)[None, :] - (first + torch.arange(cu[b + 1] - cu[b], device=DEV))[:, None]
            seen = ahead <= 0
            if window > 0:
                seen = seen & (ahead > -window)
            for e in range(h * group, (h + 1) * group):
                score = (s["q"][rows, e].double() @ k.T) * s["scale"]
                score = torch.where(seen, score, torch.full_like(score, -math.inf))
                if s["sinks"] is not None:  # a key of its own, without a value
                    score = torch.cat([score, s["sinks"][e].double().expand(score.shape[0], 1)], dim=1)
                if score.shape[1] == 0:
                    continue
                total = torch.logsumexp(score, dim=1)
                p = torch.exp(score - torch.where(torch.isinf(total), torch.zeros_like(total), total)[:, None])
                out[rows, e] = p[:, :k.shape[0]] @ v
                lse[rows, e] = total
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s["q"], s["wq"], s), _exact_rotate(s["k"], s["wk"], s)
    if case["op"] == "append":
        return (_exact_append(s["k"], s["k_pages"], s["scales"][..., 0], s),
                _exact_append(s["v"], s["v_pages"], s["scales"][..., 1], s))
    return _exact_attend(s)
