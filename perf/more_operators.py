"""Cases for a paged KV cache held in 4 bits and for the page plan of a serving step: what each
operator computes in plain torch, the calls of this library that compute the same, the work of a
pass and its result in 64 bits.

  plan     a step's block tables, slots, positions and lengths from the requests' lengths and a list
           of free pages
  release  the pages of finished requests back to that list
  append   new K/V rows quantised into their slots, and the pages as the values they stand for
  decode   one query token per sequence over such a cache
  prefill  a chunk of new tokens over a prefix held in such a cache

The cache: kv_pages uint8 [num_pages, kv_heads, 2 (K, V), 9, D].  The first 8 D bytes of a (page,
head, K or V) hold the codes [D / 32 groups of channels][16 tokens][16 bytes]; eight channels of a
token are a little-endian 32-bit word, channel c at bit 4 (c / 2) + 16 (c % 2).  The last D bytes are
16-bit words [D / 32][16], one for each token and group: a bf16 scale s of four significant bits with
the code z of the value 0 in its low four bits.  Value = s * (code - z).
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
GROUP = 32
DEV = "cuda"
BITS = (0, 16, 4, 20, 8, 24, 12, 28)  # of the eight channels of a word


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the next token of every sequence of a decode batch: one in sixteen needs a page
        dict(name="plan_decode_batch", op="plan", seqs=256, new_lo=1, new_hi=1, start_lo=0, start_hi=8192, columns=1024),
        # prompts of a prefill step, some continued, many pages each
        dict(name="plan_prompts", op="plan", seqs=24, new_lo=1, new_hi=8192, start_lo=0, start_hi=4096, columns=8192),
        # a few requests of a batch have ended
        dict(name="release_some", op="release", seqs=128, len_lo=1, len_hi=4096, done=0.1, columns=512),
        # a batch of long contexts is let go
        dict(name="release_long", op="release", seqs=64, len_lo=128, len_hi=131072, done=1.0, columns=8192),
        # a decode step's rows, gpt-oss heads: one token for each of 64 sequences, some of them padding
        dict(name="append_decode_batch", op="append", tokens=64, runs=64, padding=5, kv_heads=8, dim=64),
        # the rows of a prefill step, Qwen3-shape heads, ragged runs
        dict(name="append_prompts", op="append", tokens=16381, runs=7, padding=0, kv_heads=4, dim=128),
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
    op = rng.choice(["plan", "release", "append", "decode", "prefill"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8] if dim == 64 else [1, 2, 4])
    heads = min(64, kv_heads * rng.choice([1, 2, 4, 8, 16]))
    if op == "plan":
        seqs = _log(rng, 1, 1500)
        hi = _log(rng, 1, max(2, min(8192, 120000 // seqs)))
        start = _log(rng, 1, 16384)
        return dict(op=op, seqs=seqs, new_lo=rng.choice([0, 1]), new_hi=hi, start_lo=0, start_hi=start,
                    columns=(hi + start) // PAGE + rng.randint(1, 200))
    if op == "release":
        seqs = _log(rng, 1, 1500)
        hi = _log(rng, 1, max(2, min(131072, 2000000 // seqs)))
        return dict(op=op, seqs=seqs, len_lo=rng.choice([0, 1]), len_hi=hi, done=round(rng.random(), 2),
                    columns=hi // PAGE + rng.randint(1, 200))
    if op == "append":
        tokens = _log(rng, 1, 16000)
        return dict(op=op, tokens=tokens, runs=min(tokens, _log(rng, 1, 200)), padding=rng.choice([0, 0, rng.randint(1, 40)]),
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
    if case["op"] == "plan":
        return (_ints(case["seqs"], case["new_lo"], case["new_hi"], log=case["new_lo"] > 0, key=1),
                _ints(case["seqs"], case["start_lo"], case["start_hi"], key=2))
    if case["op"] == "release":
        lens = _ints(case["seqs"], case["len_lo"], case["len_hi"], log=case["len_lo"] > 0, key=6)
        done = np.random.default_rng([case["seqs"], 7]).random(case["seqs"]) < case["done"]
        done[0] = True
        return lens, [bool(d) for d in done]
    if case["op"] == "append":
        r = np.random.default_rng([case["tokens"], case["runs"], 8])
        cuts = np.sort(r.choice(np.arange(1, case["tokens"]), case["runs"] - 1, replace=False)) if case["runs"] > 1 else []
        new = np.diff(np.concatenate([[0], cuts, [case["tokens"]]]).astype(np.int64))
        return [int(n) for n in new], [int(x) for x in r.integers(0, 200, case["runs"])]
    if case["op"] == "decode":
        return _ints(case["seqs"], case["len_lo"], case["len_hi"], case["log"], key=3)
    return (_ints(case["seqs"], case["new_lo"], case["new_hi"], key=4),
            _ints(case["seqs"], case["pre_lo"], case["pre_hi"], key=5))


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _gen(seed, key):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + key)


def _rows(shape, g, dim):
    """K or V rows: a standard deviation and an offset of its own for each channel, as a model's have."""
    ch = torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV))
    off = torch.randn(dim, generator=g, device=DEV) * 0.5
    return torch.randn(shape, generator=g, device=DEV).add_(off).mul_(ch).to(torch.bfloat16)


def _pow2(n):
    """2^n in 64 bits, exactly."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _coded(x):
    """bf16 rows [..., D] as codes 0..15 and the words of their groups [..., D / 32], in 64 bits up to
    the scale: the smallest s of four significant bits with 15 s no less than the group's range (0
    counts as in it), z = -low / s rounded, codes x / s + z rounded, at most 15, ties to even."""
    x = x.unflatten(-1, (-1, GROUP)).double()
    low, high = x.amin(-1).clamp_(max=0.0), x.amax(-1).clamp_(min=0.0)
    part, power = torch.frexp((high - low) / 15.0)
    s = torch.ceil(part * 16.0) * _pow2(power - 4)
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    by = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.where(s > 0, torch.round(-low / by), torch.zeros_like(s))
    codes = torch.round(x / by[..., None] + z[..., None]).clamp_(0, 15)
    codes = torch.where(s[..., None] > 0, codes, torch.zeros_like(codes)).to(torch.int32).flatten(-2)
    words = (s.float().view(torch.int32) >> 16) + z.to(torch.int32)
    return codes, words


def _words32(codes):
    """Codes [..., D] as 32-bit words of eight channels [..., D / 8]."""
    c = codes.unflatten(-1, (-1, 8))
    w = torch.zeros(c.shape[:-1], dtype=torch.int32, device=c.device)
    for i, bit in enumerate(BITS):
        w |= c[..., i] << bit
    return w


def _packed(x):
    """Rows [n, heads, 16, D] of whole pages as bytes [n, heads, 9, D]."""
    n, h, _, dim = x.shape
    codes, words = _coded(x)
    w = _words32(codes).unflatten(-1, (dim // GROUP, 4)).transpose(2, 3).contiguous()  # [n, h, groups, 16, 4]
    p = words.to(torch.int16).transpose(2, 3).contiguous()
    return torch.cat([w.view(torch.uint8).view(n, h, 8, dim), p.view(torch.uint8).view(n, h, 1, dim)], dim=2)


def _cache(npages, kv_heads, dim, g):
    out = torch.empty(max(npages, 1), kv_heads, 2, 9, dim, dtype=torch.uint8, device=DEV)
    for i in range(2):
        for at in range(0, out.shape[0], 8192):
            n = min(8192, out.shape[0] - at)
            out[at:at + n, :, i] = _packed(_rows((n, kv_heads, PAGE, dim), g, dim))
    return out


def _table(pages_of, npages, g, columns=None):
    """Block table over a shuffled pool (unused columns -1), and the pages it leaves."""
    perm = torch.randperm(max(npages, 1), generator=g, device=DEV).to(torch.int32).cpu().numpy()
    columns = columns or max(1, max(pages_of))
    t = np.full((len(pages_of), columns), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages_of):
        t[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t).to(DEV), perm[at:]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed, 1)
    op = case["op"]
    s = dict(case=case, op=op)
    if op in ("plan", "release"):
        if op == "plan":
            new, held = _lens(case)
            take = sum(_pages(p + n) - _pages(p) for n, p in zip(new, held))
            s["new"], s["tokens"] = _i32(new), sum(new) + 3  # a few rows of padding behind the batch
        else:
            held, done = _lens(case)
            take = 0
            s["done"] = torch.tensor(done, device=DEV)
        used = [_pages(n) for n in held]
        npages = sum(used) + take + 17
        s["table"], left = _table(used, npages, g, case["columns"])
        free = np.zeros(npages, dtype=np.int32)
        free[:len(left)] = left
        s["free"], s["num_free"], s["held"] = torch.from_numpy(free).to(DEV), _i32([len(left)]), _i32(held)
        return s
    dim, hkv = case["dim"], case["kv_heads"]
    if op == "append":
        new, start = _lens(case)
        # the pool holds the pages that this step writes to, whole or in part, and two others
        first = [p // PAGE for p in start]
        used = [_pages(p + n) - f for p, n, f in zip(start, new, first)]
        npages = sum(used) + 2
        s["kv_pages"] = _cache(npages, hkv, dim, g)
        table = _table(used, npages, g)[0].cpu().numpy()
        slots = [np.arange(p, p + n) for p, n in zip(start, new)]
        slots = [table[b, at // PAGE - f].astype(np.int64) * PAGE + at % PAGE for b, (at, f) in enumerate(zip(slots, first))]
        slots = np.concatenate(slots + [np.full(case["padding"], -1, dtype=np.int64)])
        s["slots"] = torch.from_numpy(slots).to(DEV)
        T = len(slots)
        qkv = torch.cat([_rows((T, hkv, dim), g, dim), _rows((T, hkv, dim), g, dim)], dim=1)
        s["k"], s["v"] = qkv[:, :hkv].contiguous(), qkv[:, hkv:]  # the rotated keys, the projection's values
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
    s["kv_pages"] = _cache(npages, hkv, dim, g)
    s["table"] = _table(used, npages, g)[0]
    s["lens"] = _i32(lens)
    T = len(lens) if op == "decode" else sum(new)
    s["q"] = torch.randn(T, hq, dim, generator=g, device=DEV).to(torch.bfloat16)
    if op == "prefill":
        s["k"], s["v"] = _rows((T, hkv, dim), g, dim), _rows((T, hkv, dim), g, dim)
        cu = np.concatenate([[0], np.cumsum(new)])
        s["cu"] = _i32(cu.tolist())
        s["most"] = max(new)
        # the plain form's plan: each token's request and place in it
        s["req"] = torch.from_numpy(np.repeat(np.arange(len(new)), new)).to(DEV)
        s["at"] = torch.from_numpy(np.arange(T) - np.repeat(cu[:-1], new)).to(DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_plan(s):
    """Every request gets its pages here: the list holds enough of them."""
    new, held, table, free, T = s["new"].long(), s["held"].long(), s["table"], s["free"], s["tokens"]
    B = new.shape[0]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)])
    old, now = (held + PAGE - 1) // PAGE, (held + new + PAGE - 1) // PAGE
    before = torch.cumsum(now - old, 0) - (now - old)
    t = torch.arange(T, device=DEV)
    live = t < cu[-1]
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp_(max=B - 1)
    pos = held[req] + t - cu[req]
    page = pos // PAGE
    fresh = s["num_free"].long() - 1 - (before[req] + page - old[req])
    got = torch.where(page < old[req], table[req, page.clamp(max=table.shape[1] - 1)].long(), free[fresh.clamp(min=0)].long())
    begins = live & (pos % PAGE == 0)
    flat = torch.where(begins, req * table.shape[1] + page, torch.full_like(page, -1))
    at = flat[begins]
    table.view(-1)[at] = got[begins].to(torch.int32)
    gone = torch.full_like(pos, -1)
    return (cu.to(torch.int32), (held + new).to(torch.int32), torch.where(live, pos, gone).to(torch.int32),
            torch.where(live, got * PAGE + pos % PAGE, gone), (s["num_free"] - (now - old).sum()).to(torch.int32), table)


def _plain_release(s):
    held, done, table, free = s["held"].long(), s["done"], s["table"], s["free"]
    pages = torch.where(done, (held + PAGE - 1) // PAGE, torch.zeros_like(held))
    col = torch.arange(table.shape[1], device=DEV)
    which = table[col[None, :] < pages[:, None]]  # request by request, in the order of their tokens
    n = s["num_free"].long()
    free[n + which.shape[0] - 1 - torch.arange(which.shape[0], device=DEV)] = which
    return torch.where(done, torch.zeros_like(held), held).to(torch.int32), (n + which.shape[0]).to(torch.int32), free


def _values(pages):
    """Bytes [n, heads, 9, D] as the values they stand for, [n, heads, 16, D] in 32 bits."""
    n, h, _, dim = pages.shape
    groups = dim // GROUP
    w = pages[:, :, :8].reshape(n, h, 8 * dim).view(torch.int32).view(n, h, groups, PAGE, 4)
    p = pages[:, :, 8].reshape(n, h, dim).view(torch.int16).view(n, h, groups, PAGE).to(torch.int32) & 0xFFFF
    s, z = ((p & 0xFFF0) << 16).view(torch.float32), (p & 15).float()
    x = torch.empty(n, h, PAGE, groups, 4, 8, dtype=torch.float32, device=pages.device)
    for i, bit in enumerate(BITS):
        x[..., i] = (((w >> bit) & 15).float().sub_(z[..., None]).mul_(s[..., None])).transpose(2, 3)
    return x.view(n, h, PAGE, dim)


def _plain_append(s):
    kv, slots = s["kv_pages"], s["slots"]
    dim = kv.shape[-1]
    groups = dim // GROUP
    keep = slots >= 0
    page, tok = slots[keep] // PAGE, slots[keep] % PAGE
    codes_at = kv[:, :, :, :8].reshape(*kv.shape[:3], 8 * dim).view(torch.int32).view(*kv.shape[:3], groups, PAGE, 4)
    words_at = kv[:, :, :, 8].reshape(*kv.shape[:3], dim).view(torch.int16).view(*kv.shape[:3], groups, PAGE)
    for i, x in enumerate((s["k"], s["v"])):
        codes, words = _coded(x[keep])
        codes_at[page, :, i, :, tok] = _words32(codes).unflatten(-1, (groups, 4))
        words_at[page, :, i, :, tok] = words.to(torch.int16)
    kv[:, :, :, :8] = codes_at.reshape(*kv.shape[:3], groups * PAGE * 4).view(torch.uint8).view(*kv.shape[:3], 8, dim)
    kv[:, :, :, 8] = words_at.reshape(*kv.shape[:3], groups * PAGE).view(torch.uint8).view(*kv.shape[:3], dim)
    return _values(kv[:, :, 0]).to(torch.bfloat16), _values(kv[:, :, 1]).to(torch.bfloat16)


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


def _rows_of(values, table):
    """Every table row's tokens: [B, Hkv, 16 * columns, D]."""
    return values[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    case = s["case"]
    hkv, dim = case["kv_heads"], case["dim"]
    group = case["heads"] // hkv
    sinks = None if s["sinks"] is None else s["sinks"].view(hkv, group)
    k = _rows_of(_values(s["kv_pages"][:, :, 0]), s["table"])
    v = _rows_of(_values(s["kv_pages"][:, :, 1]), s["table"])
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
        if op == "plan":
            p = sinkattn.plan_step(s["new"], s["held"], s["table"], s["free"], s["num_free"], s["tokens"])
            return p.cu_seqlens, p.seq_lens, p.positions, p.slots, p.num_free, s["table"]
        if op == "release":
            return (*sinkattn.release_pages(s["done"], s["held"], s["table"], s["free"], s["num_free"]), s["free"])
        if op == "append":
            sinkattn.append_kv_int4(s["k"], s["v"], s["slots"], s["kv_pages"])
            return sinkattn.unpack_kv_int4(s["kv_pages"])
        if op == "decode":
            return sinkattn.decode_int4(s["q"], s["kv_pages"], s["table"], s["lens"], sinks=s["sinks"], scale=s["scale"],
                                        window=s["case"]["window"])
        return sinkattn.prefill_int4(s["q"], s["k"], s["v"], s["cu"], s["kv_pages"], s["table"], s["lens"],
                                     sinks=s["sinks"], scale=s["scale"], window=s["case"]["window"])
    if op == "plan":
        return _plain_plan(s)
    if op == "release":
        return _plain_release(s)
    return _plain_append(s) if op == "append" else _plain_attend(s)


# ------------------------------------------------------------------ work
def _pairs(new, pre, window):
    n = 0
    for a, p in zip(new, pre):
        seen = np.arange(p + 1, p + a + 1, dtype=np.int64)
        n += int((np.minimum(seen, window) if window > 0 else seen).sum())
    return n


def work(case):
    op = case["op"]
    if op == "plan":
        new, held = _lens(case)
        take = sum(_pages(p + n) - _pages(p) for n, p in zip(new, held))
        begun = sum(1 for n, p in zip(new, held) if n and p % PAGE)
        T = sum(new) + 3
        return {"bytes": 16 * case["seqs"] + 8 * take + 4 * begun + 12 * T, "flops": T}
    if op == "release":
        lens, done = _lens(case)
        pages = sum(_pages(n) for n, d in zip(lens, done) if d)
        return {"bytes": 9 * case["seqs"] + 8 * pages, "flops": pages}
    dim, hkv = case["dim"], case["kv_heads"]
    if op == "append":
        new, start = _lens(case)
        pages = sum(_pages(p + n) - p // PAGE for p, n in zip(start, new)) + 2
        row = 2 * hkv * dim  # K and V elements of a token
        return {"bytes": sum(new) * (row * 2 + row * 9 // 16 + 8) + pages * PAGE * row * (2 * 16 + 9) // 16, "flops": 4 * sum(new) * row}
    if op == "decode":
        lens = [min(n, case["window"]) if case["window"] > 0 else n for n in _lens(case)]
        return {"bytes": sum(lens) * hkv * dim * 9 // 8 + case["seqs"] * case["heads"] * (dim * 4 + 4),
                "flops": 4 * dim * case["heads"] * sum(lens)}
    new, pre = _lens(case)
    seen = [min(p, case["window"] + a) if case["window"] > 0 else p for a, p in zip(new, pre) if a]
    return {"bytes": sum(seen) * hkv * dim * 9 // 8 + sum(new) * (case["heads"] * (dim * 4 + 4) + 2 * hkv * dim * 2),
            "flops": 4 * dim * case["heads"] * _pairs(new, pre, case["window"])}


# ------------------------------------------------------------------ 64 bits
def _exact_plan(s):
    """Request by request: a stack of free pages, taken from its top."""
    new, held = s["new"].tolist(), s["held"].tolist()
    table, top = s["table"].cpu().numpy().copy(), int(s["num_free"][0])
    free = s["free"].cpu().numpy()
    pos = np.full(s["tokens"], -1, dtype=np.int32)
    slots = np.full(s["tokens"], -1, dtype=np.int64)
    cu, t = [0], 0
    for b, (n, p) in enumerate(zip(new, held)):
        for c in range(-(-p // PAGE), -(-(p + n) // PAGE)):
            top -= 1
            table[b, c] = free[top]
        at = np.arange(p, p + n)
        pos[t:t + n] = at
        slots[t:t + n] = table[b, at // PAGE].astype(np.int64) * PAGE + at % PAGE
        t += n
        cu.append(t)
    i32 = lambda v: torch.from_numpy(np.asarray(v, dtype=np.int32))  # noqa: E731
    return (i32(cu), i32([n + p for n, p in zip(new, held)]), torch.from_numpy(pos), torch.from_numpy(slots), i32([top]),
            torch.from_numpy(table))


def _exact_release(s):
    """What goes back lies so that requests planned last are taken apart first."""
    held, done, table = s["held"].tolist(), s["done"].tolist(), s["table"].cpu().numpy()
    free, n = s["free"].cpu().numpy().copy(), int(s["num_free"][0])
    back = [int(table[b, c]) for b in range(len(held)) if done[b] for c in range(-(-held[b] // PAGE))]
    free[n:n + len(back)] = back[::-1]
    lens = np.array([0 if d else x for x, d in zip(held, done)], dtype=np.int32)
    return torch.from_numpy(lens), torch.tensor([n + len(back)], dtype=torch.int32), torch.from_numpy(free)


def _decoded(raw):
    """Bytes [..., 9, D] as values [..., 16, D] in 64 bits, channel by channel from the layout."""
    raw = raw.cpu().numpy()
    dim = raw.shape[-1]
    flat = raw.reshape(*raw.shape[:-2], 9 * dim)
    out = np.empty((*raw.shape[:-2], PAGE, dim))
    tok = np.arange(PAGE)
    for c in range(dim):
        g, i = divmod(c, GROUP)
        word, e = divmod(i, 8)
        bit = 4 * (e // 2) + 16 * (e % 2)
        code = (flat[..., (g * PAGE + tok) * 16 + word * 4 + bit // 8] >> (bit % 8)) & 15
        lo = flat[..., 8 * dim + (g * PAGE + tok) * 2].astype(np.int64)
        hi = flat[..., 8 * dim + (g * PAGE + tok) * 2 + 1].astype(np.int64)
        p = hi * 256 + lo
        power, part = (p >> 7) & 255, (p >> 4) & 7
        s = np.where(power > 0, np.ldexp(1.0 + part / 8.0, power - 127), 0.0)
        out[..., c] = (code.astype(np.float64) - (p & 15)) * s
    return out


def _exact_append(s):
    """Group by group from the definition: the values that the rows' codes stand for, in their slots."""
    slots = s["slots"].cpu().numpy()
    keep = slots >= 0
    out = []
    for i, x in enumerate((s["k"], s["v"])):
        held = _decoded(s["kv_pages"][:, :, i])
        x = x.double().cpu().numpy()[keep]
        x = x.reshape(*x.shape[:2], -1, GROUP)
        low, high = np.minimum(x.min(-1), 0), np.maximum(x.max(-1), 0)
        step = np.zeros_like(low)
        # the candidates 8 .. 15 times a power of two around range / 15, smallest first
        want = (high - low) / 15
        power = np.floor(np.log2(np.where(want > 0, want, 1))) - 4
        for tries in range(24):
            cand = (8 + tries % 8) * np.exp2(power + tries // 8)
            step = np.where((step == 0) & (want > 0) & (cand >= want), cand, step)
        by = np.where(step > 0, step, 1)
        z = np.rint(-low / by)
        val = (np.clip(np.rint(x / by[..., None] + z[..., None]), 0, 15) - z[..., None]) * step[..., None]
        held[slots[keep] // PAGE, :, slots[keep] % PAGE] = val.reshape(*x.shape[:2], -1)
        out.append(torch.from_numpy(held))
    return tuple(out)


def _exact_attend(s):
    case = s["case"]
    hkv, hq = case["kv_heads"], case["heads"]
    group, window = hq // hkv, case["window"]
    lens = s["lens"].tolist()
    cu = list(range(len(lens) + 1)) if s["op"] == "decode" else s["cu"].tolist()
    out = torch.zeros(cu[-1], hq, case["dim"], dtype=torch.float64, device=DEV)
    lse = torch.full((cu[-1], hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, held in enumerate(lens):
        at = s["table"][b, :_pages(held)].long()
        rows = slice(cu[b], cu[b + 1])
        if cu[b] == cu[b + 1]:
            continue
        for h in range(hkv):
            k, v = (_unfolded(s["kv_pages"][at, h, i])[:held] for i in range(2))
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


def _unfolded(raw):
    """Bytes [n, 9, D] of one head as values [16 n, D] in 64 bits, on the device: low nibbles of a byte
    before its high ones, the bytes of a word in the order 0, 2, 1, 3."""
    n, _, dim = raw.shape
    groups = dim // GROUP
    b = raw[:, :8].reshape(n, groups, PAGE, 4, 2, 2)  # [..., word, channel parity, byte of the parity]
    nib = torch.stack([b % 16, b // 16], dim=-1)      # [..., word, parity, byte, nibble]
    code = nib.permute(0, 2, 1, 3, 5, 6, 4).reshape(n, PAGE, groups, GROUP).double()
    w = raw[:, 8].reshape(n, groups, PAGE, 2).double()
    p = (w[..., 0] + 256 * w[..., 1]).transpose(1, 2)  # [n, 16, groups]
    z = p % 16
    power = torch.floor(p / 128)
    s = torch.where(power > 0, (1.0 + torch.floor(p % 128 / 16) / 8.0) * _pow2(power - 127), torch.zeros_like(p))
    return ((code - z[..., None]) * s[..., None]).reshape(n * PAGE, dim)


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "release": _exact_release, "append": _exact_append}.get(case["op"], _exact_attend)(s)
