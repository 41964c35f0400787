"""Cases for measuring decode over shared prefixes and beam search over a paged cache.

The operators, by the ``kind`` of a case:

``shared``  decode attention of sequences in groups that share a prefix: the
            prefix's keys are read through the row of the group's first
            sequence, the keys behind it through each sequence's own row
``select``  beam search's selection: the best continuations of each group of
            beams over beams and vocabulary, from logits and running scores
``reorder`` the states follow the selection: token-table rows and histories
            of the chosen parents, and the partly filled last pages copied

``own`` selects the framework's calls; else ``run`` computes the plain form
with elementary torch operations in 32 bits (the selection's totals, whose
order decides, in 64).
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------ 4-bit pool rows
def layout(hkv, d):
    """(groups, heads of a group, code bytes, scale bytes, group bytes) of a pool row."""
    gs = 8
    while hkv % gs:
        gs //= 2
    code, sc = gs * d // 2, gs * d // 16
    return hkv // gs, gs, code, sc, -(-(code + sc) // 16) * 16


def quantise_rows(x, head_scale):
    """x fp32 [T, Hkv, d] to 4-bit pool rows uint8 [T, row bytes] (padding zero)."""
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


def values(rows, c, scale):
    """Pool rows [..., row] of the case's type to the fp32 values [..., Hkv, d] they stand for."""
    hkv, d = c["hkv"], c["d"]
    if c["pool"] == "bf16":
        return rows.float().unflatten(-1, (hkv, d))
    if c["pool"] == "fp8":
        return rows.view(torch.float8_e4m3fn).float().unflatten(-1, (hkv, d)) * scale[:, None]
    groups, gs, code, sc, gb = layout(hkv, d)
    lead = rows.shape[:-1]
    r = rows.reshape(-1, groups, gb)
    b = r[:, :, :code]
    k = torch.stack((b & 15, b >> 4), -1).reshape(-1, hkv, d // 16, 16)
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                       device=rows.device)
    s = r[:, :, code:code + sc].contiguous().view(torch.float8_e4m3fn).float().reshape(-1, hkv, d // 16, 1)
    return (lut[k.int()] * s * scale[:, None, None]).reshape(*lead, hkv, d)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one request's four beams shortly after its prompt: latency of a step
        {"name": "shared 1 x 4 beams", "kind": "shared", "groups": 1, "lo": 4, "hi": 4, "loose": 0, "prefix_lo": 992, "prefix_hi": 992,
         "suffix_lo": 1, "suffix_hi": 40, "hq": 32, "hkv": 8, "d": 128, "page": 16, "pool": "bf16", "mix": 1},
        # 64 requests behind one system prompt
        {"name": "shared 64 x 8192", "kind": "shared", "groups": 1, "lo": 64, "hi": 64, "loose": 0, "prefix_lo": 8192, "prefix_hi": 8192,
         "suffix_lo": 16, "suffix_hi": 1024, "hq": 32, "hkv": 8, "d": 128, "page": 16, "pool": "bf16", "mix": 2},
        # a full serving batch behind one long document
        {"name": "shared 256 x 32768", "kind": "shared", "groups": 1, "lo": 256, "hi": 256, "loose": 0, "prefix_lo": 32768,
         "prefix_hi": 32768, "suffix_lo": 16, "suffix_hi": 512, "hq": 32, "hkv": 8, "d": 128, "page": 16, "pool": "bf16", "mix": 3},
        # eight beams of each of sixteen requests, head size 64, an FP8 cache
        {"name": "shared 16 x 8 beams fp8", "kind": "shared", "groups": 16, "lo": 8, "hi": 8, "loose": 0, "prefix_lo": 512,
         "prefix_hi": 8192, "suffix_lo": 1, "suffix_hi": 200, "hq": 32, "hkv": 8, "d": 64, "page": 16, "pool": "fp8", "mix": 4},
        # samples of a few requests over a 4-bit cache
        {"name": "shared 4 x 16 fp4", "kind": "shared", "groups": 4, "lo": 16, "hi": 16, "loose": 0, "prefix_lo": 16384,
         "prefix_hi": 16384, "suffix_lo": 1, "suffix_hi": 500, "hq": 32, "hkv": 8, "d": 128, "page": 16, "pool": "fp4", "mix": 5},
        # ragged groups, some empty, and sequences of none, over a token-granular pool of six heads
        {"name": "shared ragged", "kind": "shared", "groups": 7, "lo": 0, "hi": 21, "loose": 5, "prefix_lo": 0, "prefix_hi": 2500,
         "suffix_lo": 0, "suffix_hi": 333, "hq": 12, "hkv": 6, "d": 128, "page": 1, "pool": "bf16", "mix": 6},
        # one request's four beams over a small vocabulary
        {"name": "select 1 x 4 x 32000", "kind": "select", "groups": 1, "beams": 4, "vocab": 32000, "n": 4, "dtype": "bf16", "slack": 0,
         "done": 0.0, "masked": 0.0, "mix": 7},
        # a batch of requests over a large vocabulary, twice the beams kept for the hypotheses that end
        {"name": "select 64 x 4 x 128256", "kind": "select", "groups": 64, "beams": 4, "vocab": 128256, "n": 8, "dtype": "bf16",
         "slack": 0, "done": 0.0, "masked": 0.0, "mix": 8},
        # an odd vocabulary in padded rows of 32 bits, some beams done, some words banned
        {"name": "select 9 x 5 x 50257", "kind": "select", "groups": 9, "beams": 5, "vocab": 50257, "n": 10, "dtype": "fp32", "slack": 7,
         "done": 0.2, "masked": 0.3, "mix": 9},
        # one request's four beams, sixteen layers
        {"name": "reorder 1 x 4", "kind": "reorder", "groups": 1, "beams": 4, "prefix": 992, "suffix": 40, "layers": 16, "hkv": 8, "d": 64,
         "page": 16, "history": 64, "mix": 10},
        # a batch's beams, sixteen layers of the larger head
        {"name": "reorder 32 x 8", "kind": "reorder", "groups": 32, "beams": 8, "prefix": 4096, "suffix": 90, "layers": 16, "hkv": 8,
         "d": 128, "page": 16, "history": 512, "mix": 11},
        # a token-granular table: rows alone move
        {"name": "reorder 6 x 5 token table", "kind": "reorder", "groups": 6, "beams": 5, "prefix": 1000, "suffix": 1777, "layers": 3,
         "hkv": 6, "d": 128, "page": 1, "history": 0, "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["shared", "shared", "shared", "select", "select", "reorder"])
    mix = rng.randrange(1 << 30)
    hkv, d = rng.choice([1, 2, 4, 6, 8, 8, 16]), rng.choice([64, 128])
    if kind == "shared":
        g = rng.choice([1, 2, 4, 4, 8])
        groups, hi = _log(rng, 1, 64), _log(rng, 1, 256)
        groups = max(1, min(groups, 256 // hi))
        prefix, suffix = _log(rng, 1, 32768), _log(rng, 1, 1024)
        # no more work than the largest listed case
        while groups * hi * hkv * g * (prefix + 64) > 256 * 32 * 32768 // 4:
            prefix = max(1, prefix // 2)
        while groups * hi * hkv * d * suffix > 256 * 8 * 128 * 512:
            suffix = max(1, suffix // 2)
        return {"kind": kind, "groups": groups, "lo": rng.choice([0, 1, hi]), "hi": hi, "loose": rng.choice([0, 0, rng.randrange(9)]),
                "prefix_lo": rng.choice([0, max(1, prefix // 8), prefix]), "prefix_hi": prefix, "suffix_lo": rng.choice([0, 1]),
                "suffix_hi": suffix, "hq": hkv * g, "hkv": hkv, "d": d, "page": rng.choice([1, 16, 16]),
                "pool": rng.choice(["bf16", "bf16", "fp8", "fp4"]), "mix": mix}
    if kind == "select":
        beams, vocab = rng.choice([1, 2, 3, 4, 5, 8, 16]), _log(rng, 64, 128256)
        groups = min(_log(rng, 1, 256), max(1, 64 * 4 * 128256 // (beams * vocab)))
        return {"kind": kind, "groups": groups, "beams": beams, "vocab": vocab, "n": rng.choice([1, beams, 2 * beams, min(64, 4 * beams)]),
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "slack": rng.choice([0, 0, rng.randrange(1, 33)]),
                "done": rng.choice([0.0, 0.0, 0.3]), "masked": rng.choice([0.0, 0.0, 0.9]), "mix": mix}
    beams = rng.choice([2, 3, 4, 5, 8, 16])
    groups = max(1, min(_log(rng, 1, 64), 256 // beams))
    return {"kind": kind, "groups": groups, "beams": beams, "prefix": rng.choice([0, _log(rng, 1, 4096)]), "suffix": _log(rng, 1, 100),
            "layers": rng.choice([1, 2, 16]), "hkv": rng.choice([1, 2, 4, 6, 8]), "d": d, "page": rng.choice([1, 16, 16]),
            "history": rng.choice([0, 1, 300]), "mix": mix}


# Sizes and lengths belong to the case, not to the seed of its values.
def shared_lens(c):
    """(sizes of the groups, their prefixes, lengths behind the prefix per sequence)."""
    r = random.Random(c["mix"])
    sizes = [r.randint(c["lo"], c["hi"]) for _ in range(c["groups"])]
    if sum(sizes) + c["loose"] == 0:
        sizes[-1] = 1
    lo, hi = c["prefix_lo"], c["prefix_hi"]
    prefixes = [min(hi, _log(r, lo, hi)) if lo > 0 and hi > 4 * lo else r.randint(lo, hi) for _ in sizes]
    if c["page"] > 1 and c["mix"] % 2 == 0:          # whole pages shared
        prefixes = [p // c["page"] * c["page"] for p in prefixes]
    tails = [r.randint(c["suffix_lo"], c["suffix_hi"]) for _ in range(sum(sizes) + c["loose"])]
    return sizes, prefixes, tails


# ----------------------------------------------------------------- prepare
def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def pool_rows(g, n, c, scale):
    x = torch.randn((n, c["hkv"], c["d"]), generator=g, device=DEV)
    if c["pool"] == "bf16":
        return x.bfloat16().flatten(1)
    if c["pool"] == "fp8":
        return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
    return quantise_rows(x.bfloat16().float(), scale)


def prepare_shared(s, c, g):
    sizes, prefixes, tails = shared_lens(c)
    page, B = c["page"], len(tails)
    first = [p for p, n in zip(prefixes, sizes) for _ in range(n)] + [0] * c["loose"]
    lens = [p + t for p, t in zip(first, tails)]
    cols = max(1, max(-(-n // page) for n in lens))
    perm = torch.randperm(sum(p // page for p in prefixes) + sum(-(-n // page) for n in lens) + 1, generator=g, device=DEV).to(torch.int32)
    nothing = perm.numel() - 1
    table = torch.full((B, cols), int(perm[nothing]), dtype=torch.int32, device=DEV)
    used = b = 0
    copies = []                                      # the tail of a prefix lies on every sequence's own page
    for p, n in zip(prefixes, sizes):
        whole = p // page
        table[b:b + n, :whole] = perm[used:used + whole]
        used += whole
        copies += [(b, q, p) for q in range(b + 1, b + n) if p % page]
        b += n
    for q in range(B):
        whole = first[q] // page
        own_pages = -(-lens[q] // page) - whole
        table[q, whole:whole + own_pages] = perm[used:used + own_pages]
        used += own_pages
    slots = perm.numel() * page
    top = 4.5 / (448.0 if c["pool"] == "fp8" else 2688.0)
    s["ks"], s["vs"] = (top * (0.8 + 0.4 * torch.rand(c["hkv"], generator=g, device=DEV)) for _ in range(2))
    live = torch.zeros(slots, dtype=torch.bool, device=DEV)
    need = torch.tensor(lens, device=DEV)
    step = max(1, (1 << 26) // cols // page)
    for q in range(0, B, step):
        j = torch.arange(cols * page, device=DEV)
        at = table[q:q + step].long()[:, j // page] * page + j % page
        live[at[j < need[q:q + step, None]]] = True
    pools = []
    for scale in (s["ks"], s["vs"]):
        parts = [pool_rows(g, min(slots - k, 1 << 18), c, scale) for k in range(0, slots, 1 << 18)]
        pool = torch.cat(parts) if len(parts) > 1 else parts[0]
        for a, b, p in copies:                       # the same keys on each sequence's page
            j = torch.arange(p // page * page, p, device=DEV)
            pool[table[b, p // page].long() * page + j % page] = pool[table[a, p // page].long() * page + j % page]
        pool[~live] = float("nan") if c["pool"] == "bf16" else 255       # slots nothing has written
        shape = (-1, page, c["hkv"], c["d"]) if c["pool"] != "fp4" else (-1, page, pool.shape[-1])
        pools.append(pool.view(shape))
    s["kc"], s["vc"] = pools
    s["table"], s["lens"], s["first"] = table, i32(lens), i32(first)
    s["cu"] = i32([sum(sizes[:k]) for k in range(len(sizes) + 1)])
    s["max_k"], s["max_p"], s["max_s"], s["max_g"] = max(1, max(lens)), max(prefixes), max(tails), max(sizes)
    s["sizes"], s["prefixes"], s["tails"] = sizes, prefixes, tails
    s["q"] = normal(g, (B, c["hq"], c["d"]))
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((B, c["hq"]), dtype=torch.float32, device=DEV)


def prepare_select(s, c, g):
    rows, V = c["groups"] * c["beams"], c["vocab"]
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[c["dtype"]]
    wide = torch.randn((rows, V + c["slack"]), generator=g, device=DEV)
    wide = wide * (1.0 + 2.0 * torch.rand((rows, 1), generator=g, device=DEV))       # flat and peaked rows
    if c["masked"] > 0:
        wide[torch.rand(wide.shape, generator=g, device=DEV) < c["masked"]] = float("-inf")
    wide[:, V:] = float("nan")                       # behind the vocabulary: not read
    s["logits"] = wide.to(dtype)[:, :V]
    s["scores"] = -10.0 * torch.rand((c["groups"], c["beams"]), generator=g, device=DEV)
    s["done"] = None
    if c["done"] > 0:
        s["done"] = (torch.rand((c["groups"], c["beams"]), generator=g, device=DEV) < c["done"]).to(torch.uint8)
    s["pad"] = min(2, V - 1)


def prepare_reorder(s, c, g):
    G, K, page = c["groups"], c["beams"], c["page"]
    N, r = G * K, random.Random(c["mix"])
    shift = [r.randrange(page) for _ in range(G)] if page > 1 else [0] * G
    lens = [c["prefix"] + c["suffix"] + x for x in shift]
    width = max(lens) + 3
    s["first"] = [c["prefix"] // page * page] * G
    pages = [-(-n // page) for n in lens]
    kept = s["first"][0] // page
    own_pages = [p - kept for p in pages]
    total = G * kept + sum(K * p for p in own_pages) + N
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    rows = N + 2
    s["idx"] = torch.randperm(rows, generator=g, device=DEV)[:N].to(torch.int32)
    s["rows"] = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    at, used = s["idx"].long(), 0
    for k in range(G):
        head = perm[used:used + kept].repeat(K, 1)
        used += kept
        tail = perm[used:used + K * own_pages[k]].view(K, -1)
        used += K * own_pages[k]
        j = torch.arange(lens[k], device=DEV)
        s["rows"][at[k * K:(k + 1) * K], :lens[k]] = torch.cat((head, tail), 1)[:, j // page] * page + (j % page).to(torch.int32)
    s["spare"] = perm[used:used + N].contiguous()
    s["lens"], s["first"] = i32([n for n in lens for _ in range(K)]), i32([n for n in s["first"] for _ in range(K)])
    s["parents"] = torch.randint(0, K, (G, K), generator=g, device=DEV, dtype=torch.int32)
    s["kc"], s["vc"] = ([normal(g, (total, page, c["hkv"], c["d"])) for _ in range(c["layers"])] for _ in range(2))
    s["history"] = torch.randint(0, 32000, (N, c["history"]), generator=g, device=DEV, dtype=torch.int32) if c["history"] else None
    s["steps"] = max(lens)


def prepare(case, seed):
    s = {"case": case}
    {"shared": prepare_shared, "select": prepare_select, "reorder": prepare_reorder}[case["kind"]](s, case, gen(seed))
    return s


# --------------------------------------------------------------- plain forms
def plain_shared(s):
    c = s["case"]
    hkv, d, page = c["hkv"], c["d"], c["page"]
    G, B = c["hq"] // hkv, len(s["tails"])
    q = s["q"].float().view(B, hkv, G, d) / math.sqrt(d)
    kf, vf = (p.reshape(p.shape[0] * page, -1) for p in (s["kc"], s["vc"]))
    none = torch.full((), float("-inf"), device=DEV)
    m = torch.full((B, hkv, G), float("-inf"), device=DEV)
    total, acc = torch.zeros((B, hkv, G), device=DEV), torch.zeros((B, hkv, G, d), device=DEV)
    b = 0
    for n, p in zip(s["sizes"], s["prefixes"]):      # each prefix against all queries of its group
        if n and p:
            j = torch.arange(p, device=DEV)
            slot = s["table"][b].long()[j // page] * page + j % page
            k, v = values(kf[slot], c, s["ks"]).transpose(0, 1), values(vf[slot], c, s["vs"]).transpose(0, 1)     # [Hkv, p, d]
            x = q[b:b + n].permute(1, 0, 2, 3).reshape(hkv, n * G, d)
            score = x @ k.transpose(1, 2)
            top = score.amax(-1, keepdim=True)
            w = (score - top).exp_()
            m[b:b + n] = top.view(hkv, n, G).transpose(0, 1)
            total[b:b + n] = w.sum(-1).view(hkv, n, G).transpose(0, 1)
            acc[b:b + n] = (w @ v).view(hkv, n, G, d).transpose(0, 1)
            del score, w
        b += n
    if s["max_s"]:
        j = torch.arange(s["max_s"], device=DEV)
        pos = s["first"].long()[:, None] + j
        seen = pos < s["lens"][:, None]
        pos = torch.where(seen, pos, torch.zeros_like(pos))
        slot = s["table"].long().gather(1, pos // page) * page + pos % page
        slot = torch.where(seen, slot, torch.zeros_like(slot))
        k = values(kf[slot], c, s["ks"])                                                 # [B, max_s, Hkv, d]
        score = (q @ k.permute(0, 2, 3, 1)).masked_fill(~seen[:, None, None], float("-inf"))
        del k
        top = torch.maximum(m, score.amax(-1))
        ref = torch.where(top > none, top, torch.zeros_like(top))
        w = (score - ref[..., None]).exp()
        scale = (m - ref).exp()
        v = torch.where(seen[..., None, None], values(vf[slot], c, s["vs"]), torch.zeros((), device=DEV))
        acc = acc * scale[..., None] + w @ v.transpose(1, 2)
        total = total * scale + w.sum(-1)
        m = top
    some = total > 0
    out = torch.where(some[..., None], acc / total.clamp(min=1e-30)[..., None], torch.zeros((), device=DEV))
    lse = torch.where(some, m + total.clamp(min=1e-30).log(), none)
    return [out.reshape(B, c["hq"], d).bfloat16(), lse.reshape(B, c["hq"])]


def plain_select(s):
    c = s["case"]
    G, K, V, n = c["groups"], c["beams"], c["vocab"], c["n"]
    x = s["logits"].double()
    low = float("-inf")
    x = torch.where(torch.isnan(x) | (x == float("inf")), torch.full((), low, dtype=torch.float64, device=DEV), x)
    top = x.amax(1, keepdim=True)
    top = torch.where(top > low, top, torch.zeros_like(top))
    lse = top + (x - top).exp().sum(1, keepdim=True).log()
    total = s["scores"].double().view(-1, 1) + (x - lse)
    if s["done"] is not None:
        done = s["done"].view(-1, 1) != 0
        kept = torch.where(torch.arange(V, device=DEV) == s["pad"], s["scores"].double().view(-1, 1), torch.full((), low, dtype=torch.float64, device=DEV))
        total = torch.where(done, kept, total)
    total = torch.where(torch.isnan(total), torch.full_like(total, low), total).view(G, K * V)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    return [best.float(), (at // V).to(torch.int32), (at % V).to(torch.int32)]


def plain_reorder(s):
    c = s["case"]
    G, K, page = c["groups"], c["beams"], c["page"]
    N = G * K
    base = torch.arange(G, device=DEV)[:, None] * K
    parent = (base + s["parents"]).view(-1).long()
    moved = parent != torch.arange(N, device=DEV)
    idx, lens = s["idx"].long(), s["lens"].long()
    rows = s["rows"][idx]
    new = rows[parent]
    j = torch.arange(rows.shape[1], device=DEV)
    inside = moved[:, None] & (j >= s["first"].long()[:, None]) & (j < lens[:, None])
    if page > 1:
        part = lens % page
        at = (lens - 1).clamp(min=0)[:, None]
        last = rows.gather(1, at).view(-1) // page
        i = torch.arange(page, device=DEV)
        move = moved[:, None] & (i < part[:, None])
        src = (last[parent].long()[:, None] * page + i)[move]
        dst = (s["spare"].long()[:, None] * page + i)[move]
        for pool in s["kc"] + s["vc"]:
            flat = pool.view(-1, c["hkv"] * c["d"])
            flat[dst] = flat[src]
        tail = j >= (lens - part)[:, None]
        new = torch.where(tail, s["spare"][:, None] * page + (j % page).to(torch.int32), new)
        swap = moved & (part > 0)
        s["spare"].copy_(torch.where(swap, last, s["spare"]))
    s["rows"][idx] = torch.where(inside, new, rows)
    if s["history"] is not None:
        s["history"].copy_(s["history"][parent])
    return [s["rows"], s["spare"]] + ([] if s["history"] is None else [s["history"]]) + s["kc"] + s["vc"]


# --------------------------------------------------------------- own calls
def own_run(s):
    import paged_kv_flashattention_gb300 as pa
    c, kind = s["case"], s["case"]["kind"]
    if kind == "shared":
        kw = {"max_prefix": s["max_p"], "max_suffix": s["max_s"], "max_group": s["max_g"]}
        scales = {}
        if c["pool"] != "bf16":
            scales = {"k_scale": s["ks"], "v_scale": s["vs"], "kv_dtype": pa.PA_KV_FP8_E4M3 if c["pool"] == "fp8" else pa.PA_KV_FP4}
        if "work" not in s:
            need = pa.decode_shared_workspace_size(s["q"].shape, s["kc"], s["max_k"], s["cu"].numel() - 1, kv_dtype=scales.get("kv_dtype"),
                                                   num_kv_heads=c["hkv"], **kw)
            s["work"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        pa.decode_shared(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["max_k"], s["cu"], s["first"], out=s["out"], lse=s["lse"],
                         workspace=s["work"], **kw, **scales)
        return [s["out"], s["lse"]]
    if kind == "select":
        if "work" not in s:
            s["work"] = torch.empty(pa.beam_select_workspace_size(c["groups"], c["beams"], c["vocab"], c["n"]), dtype=torch.uint8, device=DEV)
        return list(pa.beam_select(s["logits"], s["scores"], c["n"], finished=s["done"], pad_token=s["pad"], workspace=s["work"]))
    pa.beam_reorder(s["parents"], s["rows"], s["idx"], s["lens"], s["spare"], s["kc"], s["vc"], prefix_lens=s["first"], history=s["history"],
                    max_seqlen_k=s["steps"])
    return [s["rows"], s["spare"]] + ([] if s["history"] is None else [s["history"]]) + s["kc"] + s["vc"]


def run(state):
    if own:
        return own_run(state)
    return {"shared": plain_shared, "select": plain_select, "reorder": plain_reorder}[state["case"]["kind"]](state)


# -------------------------------------------------------------------- work
def row_bytes(c):
    e = c["hkv"] * c["d"]
    return {"bf16": 2 * e, "fp8": e, "fp4": e * 9 // 16}[c["pool"]]


def work(case):
    c = case
    if c["kind"] == "shared":
        sizes, prefixes, tails = shared_lens(c)
        once = sum(p for p, n in zip(prefixes, sizes) if n) + sum(tails)
        seen = sum(p * n for p, n in zip(prefixes, sizes)) + sum(tails)
        return {"bytes": 2 * row_bytes(c) * once + 4 * (once // c["page"]) + len(tails) * c["hq"] * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["hq"] * seen}
    if c["kind"] == "select":
        cells = c["groups"] * c["beams"] * c["vocab"]
        return {"bytes": int(cells * (1.0 - c["done"])) * (4 if c["dtype"] == "fp32" else 2) + c["groups"] * (4 * c["beams"] + 12 * c["n"]),
                "flops": 3 * cells}
    r = random.Random(c["mix"])
    G, K, page = c["groups"], c["beams"], c["page"]
    part = [(c["prefix"] + c["suffix"] + (r.randrange(page) if page > 1 else 0)) for _ in range(G)]
    moved = K - 1                                    # of K beams with random parents, K - 1 on average have another one
    kept = c["prefix"] // page * page
    rows = sum(n % page for n in part) * moved
    cells = sum(n - kept for n in part) * moved + c["history"] * G * moved
    return {"bytes": 2 * (rows * 2 * c["layers"] * 2 * c["hkv"] * c["d"] + 4 * cells) + 16 * G * K, "flops": 0}


# ------------------------------------------------------------------- exact
def e4m3_table():
    out = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(math.nan if code & 127 == 127 else -v if code > 127 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def exact_rows(rows, c, scale):
    hkv, d = c["hkv"], c["d"]
    if c["pool"] == "bf16":
        return rows.double().view(-1, hkv, d)
    table = e4m3_table()
    if c["pool"] == "fp8":
        return table[rows.long()].view(-1, hkv, d) * scale.double()[:, None]
    groups, gs, code, sc, gb = layout(hkv, d)
    r = rows.reshape(-1, groups, gb).long()
    mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    mag = torch.tensor(mag + [-x for x in mag], dtype=torch.float64, device=DEV)
    b = r[..., :code]
    v = torch.stack((mag[b % 16], mag[b // 16]), -1).reshape(-1, hkv, d // 16, 16)
    return (v * table[r[..., code:code + sc]].reshape(-1, hkv, d // 16, 1)).reshape(-1, hkv, d) * scale.double()[:, None]


def exact_shared(s, c):
    hkv, d, page = c["hkv"], c["d"], c["page"]
    G = c["hq"] // hkv
    kf, vf = (p.reshape(p.shape[0] * page, -1) for p in (s["kc"], s["vc"]))
    outs, lses = [], []

    def keys(b, lo, hi):
        j = torch.arange(lo, hi, device=DEV)
        slot = s["table"][b, j // page].long() * page + j % page
        return [exact_rows(f[slot], c, x).permute(1, 0, 2) for f, x in ((kf, s["ks"]), (vf, s["vs"]))]

    b = 0
    for n, p in list(zip(s["sizes"], s["prefixes"])) + [(1, 0)] * c["loose"]:
        if n:
            pk, pv = keys(b, 0, p)
        for i in range(b, b + n):
            sk, sv = keys(i, p, p + s["tails"][i])
            q = s["q"][i].double().view(hkv, G, d)
            x = torch.cat((q @ pk.transpose(1, 2), q @ sk.transpose(1, 2)), -1) / math.sqrt(d)
            if x.shape[-1] == 0:
                outs.append(torch.zeros((hkv, G, d), dtype=torch.float64, device=DEV))
                lses.append(torch.full((hkv, G), float("-inf"), dtype=torch.float64, device=DEV))
                continue
            w = torch.softmax(x, -1)
            outs.append(w[..., :p] @ pv + w[..., p:] @ sv)
            lses.append(torch.logsumexp(x, -1))
        b += n
    return [torch.stack(outs).view(-1, c["hq"], d), torch.stack(lses).view(-1, c["hq"])]


def exact_select(s, c):
    G, K, V = c["groups"], c["beams"], c["vocab"]
    low, chosen = -1e300, float("-inf")              # nothing to choose; chosen already
    x = s["logits"].double().nan_to_num(nan=float("-inf"), posinf=float("-inf"), neginf=float("-inf"))
    total = (torch.log_softmax(x, 1).view(G, K, V) + s["scores"].double()[..., None]).nan_to_num(nan=low, neginf=low)
    if s["done"] is not None:
        for g, k in s["done"].nonzero().tolist():
            total[g, k] = low
            total[g, k, s["pad"]] = s["scores"][g, k].double()
    total = total.view(G, K * V)
    best, where = [], []
    for _ in range(c["n"]):
        v = total.amax(1, keepdim=True)
        at = (total == v).to(torch.int8).argmax(1, keepdim=True)
        total.scatter_(1, at, chosen)
        best.append(v)
        where.append(at)
    best, where = torch.cat(best, 1), torch.cat(where, 1)
    return [torch.where(best == low, torch.full_like(best, float("-inf")), best), (where // V).int(), (where % V).int()]


def exact(case, seed):
    if case["kind"] == "reorder":
        return None
    s = prepare(case, seed)
    return exact_shared(s, case) if case["kind"] == "shared" else exact_select(s, case)
