"""Cases for measuring the 4-bit KV cache and the batch plan built on the GPU.

The operators, by the ``kind`` of a case:

``store``   quantise new K/V rows into a paged pool of 4-bit rows and read
            the same rows back as bf16 values
``rope``    rotary embedding of q and k fused with that store, and the rows
            read back
``decode``  one query per sequence over a 4-bit paged cache
``prefill`` causal attention of packed new tokens over a 4-bit paged cache
``batch``   request lengths to boundaries, positions, slots and page table,
            with new pages taken from a free list

A pool row holds one token: groups of ``gs`` KV heads (the largest power of
two up to 8 that divides the head count), each group its heads' E2M1 codes
(two to a byte, the even element in the low nibble), then one E4M3 scale per
head and 16 elements, padded to a multiple of 16 bytes.  An element reads as
``code * block scale * head scale``; the store divides by ``block scale *
head scale`` and rounds to the nearest code.

``own`` selects the framework's calls; else ``run`` computes the plain form
with elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 512            # keys of a sequence taken together in the plain decode


# --------------------------------------------------------------- the format
def layout(hkv, d):
    """(groups, heads of a group, code bytes, scale bytes, group bytes) of a pool row."""
    gs = 8
    while hkv % gs:
        gs //= 2
    code, sc = gs * d // 2, gs * d // 16
    return hkv // gs, gs, code, sc, -(-(code + sc) // 16) * 16


def row_bytes(hkv, d):
    groups, _, _, _, gb = layout(hkv, d)
    return groups * gb


def quantise_rows(x, head_scale):
    """x fp32 [T, Hkv, d] to pool rows uint8 [T, row_bytes] (padding zero)."""
    T, hkv, d = x.shape
    groups, gs, code, sc, gb = layout(hkv, d)
    x = x.reshape(T, hkv, d // 16, 16)
    s8 = (x.abs().amax(-1) / head_scale[:, None] / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (s8.float() * head_scale[:, None])[..., None]
    z = torch.where(step > 0, x / step, torch.zeros_like(x))
    a = z.abs()
    c = (a > 0.25).to(torch.uint8)
    for edge, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= edge) if up else (a > edge)
    c += (z < 0).to(torch.uint8) * 8
    c = c.reshape(T, groups, gs * d)
    rows = torch.zeros((T, groups, gb), dtype=torch.uint8, device=x.device)
    rows[:, :, :code] = c[..., 0::2] | (c[..., 1::2] << 4)
    rows[:, :, code:code + sc] = s8.view(torch.uint8).reshape(T, groups, sc)
    return rows.reshape(T, groups * gb)


def values(rows, hkv, d, head_scale):
    """Pool rows uint8 [..., row_bytes] to the fp32 values [..., Hkv, d] they stand for."""
    groups, gs, code, sc, gb = layout(hkv, d)
    lead = rows.shape[:-1]
    r = rows.reshape(-1, groups, gb)
    b = r[:, :, :code]
    c = torch.stack((b & 15, b >> 4), -1).reshape(-1, hkv, d // 16, 16)
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                       device=rows.device)
    v = lut[c.int()]
    s = r[:, :, code:code + sc].contiguous().view(torch.float8_e4m3fn).float().reshape(-1, hkv, d // 16, 1)
    v *= s * head_scale[:, None, None]
    return v.reshape(*lead, hkv, d)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's new tokens, padded to a captured batch size
        {"name": "store 64 decode tokens", "kind": "store", "tokens": 64, "pad": 7, "hkv": 8, "d": 64, "page": 16, "mix": 1},
        # the prompts of sixteen requests of 512 tokens
        {"name": "store 8192 tokens", "kind": "store", "tokens": 8192, "pad": 0, "hkv": 8, "d": 128, "page": 16, "mix": 2},
        # a ragged chunk, half of each head rotated in interleaved pairs, six KV heads
        {"name": "rope store 333 ragged", "kind": "rope", "tokens": 333, "pad": 5, "hq": 12, "hkv": 6, "d": 64, "rot": 32, "pairs": True, "page": 1, "mix": 3},
        # the same sixteen prompts on their way from the projection into the cache
        {"name": "rope store 8192 tokens", "kind": "rope", "tokens": 8192, "pad": 0, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "pairs": False, "page": 16, "mix": 4},
        # one user's long conversation: latency of a single token
        {"name": "decode 1 x 20011", "kind": "decode", "seqs": 1, "lo": 20011, "hi": 20011, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "mix": 5},
        # short ragged contexts with a sliding window over a token-granular pool, an empty row among them
        {"name": "decode window odd heads", "kind": "decode", "seqs": 7, "lo": 0, "hi": 1500, "hq": 12, "hkv": 6, "d": 128, "page": 1, "window": 700, "mix": 6},
        # a batch of 64 sequences at head size 64
        {"name": "decode 64 x 4096 d64", "kind": "decode", "seqs": 64, "lo": 128, "hi": 4096, "hq": 32, "hkv": 8, "d": 64, "page": 16, "window": 0, "mix": 7},
        # a full serving batch of log-uniform contexts
        {"name": "decode 256 x 32768", "kind": "decode", "seqs": 256, "lo": 512, "hi": 32768, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "mix": 8},
        # a few ragged prompts over short cached prefixes
        {"name": "prefill 3 ragged d64", "kind": "prefill", "seqs": 3, "cached": 500, "lo": 1, "hi": 300, "hq": 8, "hkv": 2, "d": 64, "page": 1, "mix": 9},
        # eight requests extended over partly cached prompts
        {"name": "prefill 8 extend", "kind": "prefill", "seqs": 8, "cached": 4096, "lo": 64, "hi": 1024, "hq": 32, "hkv": 8, "d": 128, "page": 16, "mix": 10},
        # the plan of a decode step: one new token each, pages taken as they fill up
        {"name": "batch 256 decode", "kind": "batch", "seqs": 256, "cached_lo": 511, "cached_hi": 32767, "lo": 1, "hi": 1, "page": 16, "free": True, "slack": 0, "mix": 11},
        # the plan of a chunk of prompts over cached prefixes, into buffers of a fixed size
        {"name": "batch 1000 mixed", "kind": "batch", "seqs": 1000, "cached_lo": 0, "cached_hi": 8000, "lo": 0, "hi": 511, "page": 16, "free": False, "slack": 777, "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["store", "rope", "decode", "decode", "prefill", "prefill", "batch"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 6, 8, 8, 16])
    g = rng.choice([1, 2, 4, 4, 8])
    c = {"kind": kind, "page": rng.choice([1, 16, 16]), "mix": rng.randrange(1 << 30)}
    if kind == "store":
        t = _log(rng, 1, 8192)
        return {**c, "tokens": t, "pad": rng.randrange(0, 1 + t // 4), "hkv": hkv, "d": d}
    if kind == "rope":
        t = _log(rng, 1, 4096)
        return {**c, "tokens": t, "pad": rng.randrange(0, 1 + t // 4), "hq": hkv * g, "hkv": hkv, "d": d,
                "rot": rng.choice([16, 32, 64, d]), "pairs": rng.random() < 0.5}
    if kind == "decode":
        hi = _log(rng, 16, 32768)
        cost = 256 * 8000 * 8 * 128 // (hi * hkv * d)
        return {**c, "seqs": min(_log(rng, 1, 256), max(1, cost)), "lo": rng.choice([0, 1, max(1, hi // 64), hi]), "hi": hi,
                "hq": hkv * g, "hkv": hkv, "d": d, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}
    if kind == "prefill":
        hi = _log(rng, 1, 1024)
        cached = rng.choice([0, _log(rng, 1, 4096)])
        b = max(1, min(_log(rng, 1, 16), 8 * 1024 * 4096 * 32 // ((hi + 64) * (cached + hi) * hkv * g)))
        return {**c, "seqs": b, "cached": cached, "lo": rng.choice([1, max(1, hi // 8), hi]), "hi": hi, "hq": hkv * g, "hkv": hkv, "d": d}
    hi = rng.choice([1, _log(rng, 1, 512)])
    return {**c, "seqs": _log(rng, 1, 1000), "cached_lo": 0, "cached_hi": _log(rng, 1, 16384), "lo": rng.choice([0, hi]), "hi": hi,
            "free": rng.random() < 0.6, "slack": rng.choice([0, 1, rng.randrange(1000)])}


# Lengths belong to the case, not to the seed of its values.
def decode_lens(c):
    r = random.Random(c["mix"])
    lo, hi = c["lo"], c["hi"]
    if lo > 0 and hi > 32 * lo:
        return [min(hi, max(lo, _log(r, lo, hi))) for _ in range(c["seqs"])]
    lens = [r.randint(lo, hi) for _ in range(c["seqs"])]
    if lo == 0 and len(lens) > 2:
        lens[1] = 0
    return lens


def prefill_lens(c):
    r = random.Random(c["mix"])
    cached = [r.randint(0, c["cached"]) for _ in range(c["seqs"])]
    extend = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return cached, extend


def batch_lens(c):
    r = random.Random(c["mix"])
    lo, hi = c["cached_lo"], c["cached_hi"]
    cached = [min(hi, _log(r, lo, hi)) if lo > 0 and hi > 32 * lo else r.randint(lo, hi) for _ in range(c["seqs"])]
    extend = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    return cached, extend


# ----------------------------------------------------------------- prepare
def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def head_scales(g, hkv):
    """A head's largest magnitude (about 4.5 for these values) over 6 * 448."""
    return (3.5 + 2.0 * torch.rand(hkv, generator=g, device=DEV)) / 2688.0


def pages_of(g, lens, page):
    """A random page table [B, columns] for these lengths, the page past the
    used ones in every unused entry, and that page's number."""
    need = [-(-n // page) for n in lens]
    total, cols = sum(need), max(1, max(need))
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    n = torch.tensor(need, device=DEV)
    start = torch.cumsum(n, 0) - n
    c = torch.arange(cols, device=DEV)
    idx = (start[:, None] + c).clamp(max=max(0, total - 1))
    used = c < n[:, None]
    table = torch.where(used, perm[idx], torch.full_like(idx, total, dtype=torch.int32)) if total else \
        torch.zeros((len(lens), cols), dtype=torch.int32, device=DEV)
    return table.contiguous(), total


def filled_pool(g, pages, page, hkv, d, scale, lens, table):
    """A pool of quantised N(0, 1) rows; the last page and the slots that no
    request has written hold bytes that read as NaN."""
    slots = (pages + 1) * page
    pool = torch.full((slots, row_bytes(hkv, d)), 255, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hkv * d))
    for s in range(0, pages * page, step):
        e = min(pages * page, s + step)
        pool[s:e] = quantise_rows(torch.randn((e - s, hkv, d), generator=g, device=DEV).bfloat16().float(), scale)
    if page > 1:
        n = torch.tensor(lens, device=DEV)
        live = n % page != 0
        last = table[torch.arange(len(lens), device=DEV), ((n - 1).clamp(min=0) // page)].long()
        off = torch.arange(page, device=DEV)
        tail = (live[:, None] & (off >= (n % page)[:, None]))
        pool[(last[:, None] * page + off)[tail]] = 255
    return pool.view(pages + 1, page, -1)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = case, gen(seed)
    kind = c["kind"]
    s = {"case": c}
    if kind in ("store", "rope"):
        T, hkv, d, page = c["tokens"], c["hkv"], c["d"], c["page"]
        pages = -(-T * 5 // (4 * page)) + 1
        s["k"], s["v"] = normal(g, (T, hkv, d)), normal(g, (T, hkv, d))
        s["ks"], s["vs"] = head_scales(g, hkv), head_scales(g, hkv)
        slot = torch.randperm(pages * page, generator=g, device=DEV)[:T].to(torch.int32)
        slot[torch.randperm(T, generator=g, device=DEV)[:c["pad"]]] = -1
        s["slot"] = slot
        s["kc"] = torch.full((pages, page, row_bytes(hkv, d)), 255, dtype=torch.uint8, device=DEV)
        s["vc"] = s["kc"].clone()
        if kind == "rope":
            s["q"] = normal(g, (T, c["hq"], d))
            s["q_out"] = torch.empty_like(s["q"])
            far = 32768
            s["pos"] = torch.randint(0, far, (T,), generator=g, device=DEV, dtype=torch.int32)
            ang = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * \
                10000.0 ** (-2.0 * torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64) / c["rot"])
            s["cs"] = torch.cat((ang.cos(), ang.sin()), 1).float().contiguous()
    elif kind == "decode":
        lens, hkv, d, page = decode_lens(c), c["hkv"], c["d"], c["page"]
        s["table"], pages = pages_of(g, lens, page)
        s["ks"], s["vs"] = head_scales(g, hkv), head_scales(g, hkv)
        s["kc"] = filled_pool(g, pages, page, hkv, d, s["ks"], lens, s["table"])
        s["vc"] = filled_pool(g, pages, page, hkv, d, s["vs"], lens, s["table"])
        s["q"] = normal(g, (len(lens), c["hq"], d))
        s["lens"], s["max_k"] = i32(lens), max(1, max(lens))
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((len(lens), c["hq"]), dtype=torch.float32, device=DEV)
        W = c["window"]
        kept = [min(n, W) if W else n for n in lens]
        s["chunks"], s["most"] = sum(-(-n // CHUNK) for n in kept), max(1, max(-(-n // CHUNK) for n in kept))
    elif kind == "prefill":
        (cached, extend), hkv, d, page = prefill_lens(c), c["hkv"], c["d"], c["page"]
        lens = [a + b for a, b in zip(cached, extend)]
        s["table"], pages = pages_of(g, lens, page)
        s["ks"], s["vs"] = head_scales(g, hkv), head_scales(g, hkv)
        s["kc"] = filled_pool(g, pages, page, hkv, d, s["ks"], lens, s["table"])
        s["vc"] = filled_pool(g, pages, page, hkv, d, s["vs"], lens, s["table"])
        s["q"] = normal(g, (sum(extend), c["hq"], d))
        s["cu_q"] = i32([sum(extend[:i]) for i in range(len(extend) + 1)])
        s["cu_k"] = i32([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["max_q"], s["max_k"] = max(extend), max(lens)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((c["hq"], sum(extend)), dtype=torch.float32, device=DEV)
    else:
        cached, extend = batch_lens(c)
        B, page = len(cached), c["page"]
        lens = [a + b for a, b in zip(cached, extend)]
        s["max_k"] = max(1, max(lens))
        s["tokens"] = sum(extend) + c["slack"]
        table, pages = pages_of(g, lens, page)
        n = torch.arange(s["max_k"], device=DEV)
        rows = B + 3
        full = table[:, n // page] * page + (n % page).to(torch.int32)
        known = cached if c["free"] else lens
        full = torch.where(n < torch.tensor(known, device=DEV)[:, None], full, torch.full_like(full, pages * page))
        s["idx"] = torch.randperm(rows, generator=g, device=DEV)[:B].to(torch.int32)
        s["tokens_at"] = torch.full((rows, s["max_k"]), pages * page, dtype=torch.int32, device=DEV)
        s["tokens_at"][s["idx"].long()] = full
        s["cached"], s["extend"] = i32(cached), i32(extend)
        if c["free"]:
            used = sum(-(-a // page) for a in cached)
            s["free"] = torch.randperm(pages - used + 64, generator=g, device=DEV).to(torch.int32)
        s["columns"] = torch.full((B, -(-s["max_k"] // page)), -1, dtype=torch.int32, device=DEV)
    return s


# --------------------------------------------------------------- plain forms
def plain_store(s, k):
    c = s["case"]
    at = s["slot"].long()
    live = at >= 0
    got = []
    for x, pool, scale in ((k, s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        flat = pool.view(-1, pool.shape[-1])
        keep = torch.where(live, at, torch.zeros_like(at))
        rows = quantise_rows(x.float(), scale)
        flat[at[live]] = rows[live]
        back = values(flat[keep], c["hkv"], c["d"], scale)
        got.append(torch.where(live[:, None, None], back, torch.zeros_like(back)).bfloat16())
    return got


def rotate(x, cos, sin, rot, pairs):
    x = x.float()
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if pairs else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1).bfloat16()


def plain_rope(s):
    c = s["case"]
    h = c["rot"] // 2
    at = s["cs"][s["pos"].long()][:, None]
    q = rotate(s["q"], at[..., :h], at[..., h:], c["rot"], c["pairs"])
    k = rotate(s["k"], at[..., :h], at[..., h:], c["rot"], c["pairs"])
    return [q] + plain_store(s, k)


def plain_decode(s):
    c = s["case"]
    hkv, d, page, W = c["hkv"], c["d"], c["page"], c["window"]
    G, B, n = c["hq"] // hkv, c["seqs"], s["chunks"]
    q = s["q"].float().view(B, hkv, G, d)
    lens = s["lens"].long()
    first = (lens - W).clamp(min=0) if W else torch.zeros_like(lens)
    per = (lens - first + CHUNK - 1) // CHUNK
    start = torch.cumsum(per, 0) - per
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), per, output_size=n)
    at = first[seq] + (torch.arange(n, device=DEV) - start[seq]) * CHUNK
    pos = at[:, None] + torch.arange(CHUNK, device=DEV)
    seen = pos < lens[seq][:, None]
    pos = torch.minimum(pos, (lens[seq] - 1)[:, None])
    slot = s["table"][seq[:, None], pos // page].long() * page + pos % page
    k = values(s["kc"].view(-1, s["kc"].shape[-1])[slot], hkv, d, s["ks"])
    score = (k.permute(0, 2, 1, 3) @ q[seq].transpose(2, 3)) / math.sqrt(d)              # [n, Hkv, CHUNK, G]
    del k
    score = score.masked_fill(~seen[:, None, :, None], float("-inf"))
    place = (start[:, None] + torch.arange(s["most"], device=DEV)).clamp(max=max(0, n - 1))
    used = (torch.arange(s["most"], device=DEV) < per[:, None])[..., None, None]
    if n == 0:
        return [torch.zeros_like(s["q"]), torch.full_like(s["lse"], float("-inf"))]
    m = torch.where(used, score.amax(2)[place], torch.full((), float("-inf"), device=DEV)).amax(1)   # [B, Hkv, G]
    p = (score - m[seq][:, :, None]).exp()
    v = values(s["vc"].view(-1, s["vc"].shape[-1])[slot], hkv, d, s["vs"])
    o = p.transpose(2, 3) @ v.permute(0, 2, 1, 3)                                        # [n, Hkv, G, d]
    total = torch.where(used, p.sum(2)[place], torch.zeros((), device=DEV)).sum(1)
    o = torch.where(used[..., None], o[place], torch.zeros((), device=DEV)).sum(1)
    some = total > 0
    out = torch.where(some[..., None], o / total.clamp(min=1e-30)[..., None], torch.zeros((), device=DEV))
    lse = torch.where(some, m + total.clamp(min=1e-30).log(), torch.full((), float("-inf"), device=DEV))
    return [out.reshape(B, -1, d).bfloat16(), lse.reshape(B, -1)]


def plain_prefill(s):
    c = s["case"]
    hkv, d, page = c["hkv"], c["d"], c["page"]
    G, B, mq, mk = c["hq"] // hkv, c["seqs"], s["max_q"], s["max_k"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    row = torch.minimum(cu_q[:-1, None] + i, (cu_q[1:] - 1)[:, None])
    q = s["q"].float()[row].view(B, mq, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * mq, d)
    pos = torch.minimum(j.expand(B, -1), (lk - 1)[:, None])
    slot = s["table"][torch.arange(B, device=DEV)[:, None], pos // page].long() * page + pos % page
    k = values(s["kc"].view(-1, s["kc"].shape[-1])[slot], hkv, d, s["ks"]).permute(0, 2, 3, 1)
    score = ((q @ k) / math.sqrt(d)).view(B, hkv, G, mq, mk)
    hidden = j > (lk - lq)[:, None, None] + i[:, None]
    score = score.masked_fill(hidden[:, None, None], float("-inf"))
    m = score.amax(-1, keepdim=True)
    p = (score - m).exp()
    total = p.sum(-1, keepdim=True)
    v = values(s["vc"].view(-1, s["vc"].shape[-1])[slot], hkv, d, s["vs"]).permute(0, 2, 1, 3)
    o = (p.view(B, hkv, G * mq, mk) @ v).view(B, hkv, G, mq, d) / total
    lse = (m + total.log()).view(B, hkv * G, mq).permute(0, 2, 1)
    real = i < lq[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, mq, hkv * G, d)[real]
    return [out.bfloat16(), lse[real].t().contiguous()]


def plain_batch(s):
    c = s["case"]
    B, page = c["seqs"], c["page"]
    cached, extend = s["cached"].long(), s["extend"].long()
    lens = cached + extend
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    cu_q, cu_k = torch.cat((zero, extend.cumsum(0))), torch.cat((zero, lens.cumsum(0)))
    held = (cached + page - 1) // page
    need = (lens + page - 1) // page - held
    base = need.cumsum(0) - need
    t = torch.arange(s["tokens"], device=DEV)
    real = t < cu_q[-1]
    b = torch.searchsorted(cu_q[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = torch.where(real, cached[b] + t - cu_q[b], torch.zeros_like(t))
    row = s["idx"].long()
    at = s["tokens_at"]
    if c["free"]:
        fresh = pos // page - held[b]
        last = at[row[b], (cached[b] - 1).clamp(min=0)] // page
        new = s["free"][(base[b] + fresh).clamp(min=0, max=s["free"].numel() - 1)]
        slot = torch.where(fresh >= 0, new, last) * page + (pos % page).to(torch.int32)
        at[row[b][real], pos[real]] = slot[real]
    else:
        slot = at[row[b], pos]
    slot = torch.where(real, slot, torch.full_like(slot, -1))
    col = torch.arange(s["columns"].shape[1], device=DEV)
    mine = col * page < lens[:, None]
    cols = torch.where(mine, at[row][:, col * page] // page, s["columns"])
    s["columns"].copy_(cols)
    totals = torch.stack((cu_q[-1], extend.max(), lens.max(), need.sum() if c["free"] else zero[0]))
    got = [cu_q, cu_k, lens, pos, slot, cols, totals]
    return [x.to(torch.int32) for x in got] + ([at] if c["free"] else [])


# --------------------------------------------------------------- own calls
def own_run(s):
    import paged_kv_flashattention_gb300 as pa
    c, kind = s["case"], s["case"]["kind"]
    if kind == "store":
        pa.store_kv_fp4(s["k"], s["v"], s["slot"], s["kc"], s["vc"], s["ks"], s["vs"])
        return list(pa.load_kv_fp4(s["slot"], s["kc"], s["vc"], s["ks"], s["vs"], c["d"]))
    if kind == "rope":
        q = pa.rope_store_kv(s["q"], s["k"], s["v"], s["pos"], s["cs"], s["slot"], s["kc"], s["vc"], q_out=s["q_out"],
                             interleaved=c["pairs"], k_scale=s["ks"], v_scale=s["vs"], kv_dtype=pa.PA_KV_FP4)
        return [q] + list(pa.load_kv_fp4(s["slot"], s["kc"], s["vc"], s["ks"], s["vs"], c["d"]))
    if kind == "decode":
        if "work" not in s:
            need = pa.decode_workspace_size(s["q"].shape, s["kc"], s["max_k"], kv_dtype=pa.PA_KV_FP4, num_kv_heads=c["hkv"])
            s["work"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        pa.decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["max_k"], out=s["out"], lse=s["lse"], workspace=s["work"],
                  k_scale=s["ks"], v_scale=s["vs"], sliding_window=c["window"], kv_dtype=pa.PA_KV_FP4)
        return [s["out"], s["lse"]]
    if kind == "prefill":
        pa.prefill(s["q"], s["kc"], s["vc"], s["table"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], out=s["out"], lse=s["lse"],
                   k_scale=s["ks"], v_scale=s["vs"], kv_dtype=pa.PA_KV_FP4)
        return [s["out"], s["lse"]]
    if "plan" not in s:
        s["plan"] = pa.BatchPlanner(DEV, c["seqs"], s["tokens"], s["max_k"], c["page"])
    b = s["plan"].build(s["cached"], s["extend"], s["tokens_at"], s["idx"], free_pages=s.get("free"))
    got = [b.cu_seqlens_q, b.cu_seqlens_k, b.cache_seqlens, b.positions, b.slot_mapping, b.page_table, b.totals]
    return got + ([s["tokens_at"]] if c["free"] else [])


def run(state):
    if own:
        return own_run(state)
    kind = state["case"]["kind"]
    if kind == "store":
        return plain_store(state, state["k"])
    return {"rope": plain_rope, "decode": plain_decode, "prefill": plain_prefill, "batch": plain_batch}[kind](state)


# -------------------------------------------------------------------- work
def work(case):
    c, kind = case, case["kind"]
    if kind in ("store", "rope"):
        T, live, e = c["tokens"], c["tokens"] - c["pad"], c["hkv"] * c["d"]
        # rows in, the live tokens' 4-bit rows, the values read back, slots
        b = 2 * (2 * e * T + e * 9 // 16 * live + 2 * e * T) + 4 * T
        f = 2 * 4 * e * T
        if kind == "rope":
            b += 2 * 2 * c["hq"] * c["d"] * T + 4 * T + 4 * c["rot"] * T
            f += 3 * c["rot"] * (c["hq"] + c["hkv"]) * T
        return {"bytes": b, "flops": f}
    if kind == "decode":
        W = c["window"]
        keys = sum(min(n, W) if W else n for n in decode_lens(c))
        row = c["hkv"] * c["d"] * 9 // 16
        return {"bytes": 2 * row * keys + 4 * (keys // c["page"]) + c["seqs"] * c["hq"] * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["hq"] * keys}
    if kind == "prefill":
        cached, extend = prefill_lens(c)
        pairs = sum(e * a + e * (e + 1) // 2 for a, e in zip(cached, extend))
        row = c["hkv"] * c["d"] * 9 // 16
        return {"bytes": 2 * row * (sum(cached) + sum(extend)) + sum(extend) * c["hq"] * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["hq"] * pairs}
    cached, extend = batch_lens(c)
    cols = sum(-(-(a + e) // c["page"]) for a, e in zip(cached, extend))
    t = sum(extend)
    return {"bytes": 4 * (2 * cols + 2 * (t + c["slack"]) + (2 if c["free"] else 1) * t + 6 * c["seqs"]), "flops": 0}


# ------------------------------------------------------------------- exact
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3_table():
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return out


def nearest(x, table):
    """The table's entry (ascending, even places win ties) nearest to each x >= 0, in 64 bits."""
    t = torch.tensor(table, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(t, x).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    up = (t[hi] - x) - (x - t[lo])
    take = (up < 0) | ((up == 0) & (hi % 2 == 0)) | (hi == 0)
    return torch.where(x >= t[-1], t[-1], torch.where(take, t[hi], t[lo]))


def single(x):
    return x.float().double()


def exact_rows(x, head_scale):
    """What the store keeps of x [T, Hkv, d] (64 bits): the quotients are single-precision divisions, as the format says."""
    g = head_scale.double()[:, None, None]
    y = x.reshape(*x.shape[:-1], -1, 16)
    s = nearest(single(single(y.abs().amax(-1, keepdim=True) / g) / 6.0), e4m3_table())
    z = single(y / torch.where(s > 0, single(s * g), torch.ones_like(s)))
    kept = torch.where(s > 0, nearest(z.abs(), GRID) * torch.sign(z) * s, torch.zeros_like(z))
    return (kept * g).reshape(x.shape)


def exact_values(rows, hkv, d, head_scale):
    groups, gs, code, sc, gb = layout(hkv, d)
    r = rows.reshape(-1, groups, gb)
    b = r[..., :code].long()
    mag = torch.tensor(GRID + [-x for x in GRID], dtype=torch.float64, device=rows.device)
    v = torch.stack((mag[b % 16], mag[b // 16]), -1).reshape(-1, hkv, d // 16, 16)
    t = torch.tensor(e4m3_table(), dtype=torch.float64, device=rows.device)
    s = t[r[..., code:code + sc].long().clamp(max=126)].reshape(-1, hkv, d // 16, 1)
    return (v * s).reshape(-1, hkv, d) * head_scale.double()[:, None]


def exact_attention(q, k, v, first):
    """q [n, Hq, d], k, v [L, Hkv, d] in 64 bits; row i sees keys up to L - n + i, from `first` on."""
    n, hq, d = q.shape
    L, hkv, _ = k.shape
    k, v = k.repeat_interleave(hq // hkv, 1), v.repeat_interleave(hq // hkv, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(d)
    j, i = torch.arange(L, device=DEV), torch.arange(n, device=DEV)
    s = s.masked_fill((j[None] > (L - n + i)[:, None]) | (j < first)[None], float("-inf"))
    return torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v), torch.logsumexp(s, -1)


def exact(case, seed):
    c = case
    if c["kind"] == "batch":
        return None
    s = prepare(case, seed)
    hkv, d = c["hkv"], c["d"]
    if c["kind"] in ("store", "rope"):
        k, got = s["k"].double(), []
        if c["kind"] == "rope":
            rot, h = c["rot"], c["rot"] // 2
            w = torch.complex(s["cs"][s["pos"].long(), :h].double(), s["cs"][s["pos"].long(), h:].double())[:, None]
            for name in ("q", "k"):
                x = s[name].double()
                z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) if c["pairs"] else torch.complex(x[..., :h], x[..., h:rot])
                z = torch.view_as_real(z * w)
                x = torch.cat((z.flatten(-2) if c["pairs"] else torch.cat((z[..., 0], z[..., 1]), -1), x[..., rot:]), -1)
                if name == "q":
                    got.append(x)
            # the cache holds bf16 keys quantised: a key whose rounding to bf16 hangs on
            # 32-bit arithmetic has no single value here
            return got + [None, exact_rows(s["v"].double(), s["vs"]) * (s["slot"] >= 0)[:, None, None]]
        live = (s["slot"] >= 0)[:, None, None]
        return [exact_rows(k, s["ks"]) * live, exact_rows(s["v"].double(), s["vs"]) * live]
    kf, vf = s["kc"].view(-1, s["kc"].shape[-1]), s["vc"].view(-1, s["vc"].shape[-1])
    outs, lses = [], []
    if c["kind"] == "decode":
        lens = decode_lens(c)
        W = c["window"]
        starts = [max(0, n - W) if W else 0 for n in lens]
        queries = [s["q"][b:b + 1].double() for b in range(len(lens))]
    else:
        cached, extend = prefill_lens(c)
        lens = [a + e for a, e in zip(cached, extend)]
        starts = [0] * len(lens)
        queries = list(s["q"].double().split(extend))
    for b, L in enumerate(lens):
        if L == 0:
            outs.append(torch.zeros_like(queries[b]))
            lses.append(torch.full((c["hq"], 1), float("-inf"), dtype=torch.float64, device=DEV))
            continue
        j = torch.arange(starts[b], L, device=DEV)
        slot = s["table"][b, j // c["page"]].long() * c["page"] + j % c["page"]
        k, v = exact_values(kf[slot], hkv, d, s["ks"]), exact_values(vf[slot], hkv, d, s["vs"])
        o, l = exact_attention(queries[b], k, v, 0)
        outs.append(o)
        lses.append(l)
    lse = torch.cat(lses, 1)
    return [torch.cat(outs), lse.t().contiguous() if c["kind"] == "decode" else lse]
