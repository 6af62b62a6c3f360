"""Operators around a paged FP4 latent cache, with their plain forms.

- norm_rope: the RMS norm of each head's query (or of a latent) and the rotation of
  its last channels by the token's position, in one pass.
- chunk_attn: attention of a chunk of new tokens of each sequence (one token, a part
  of a prompt, a whole one) over the entries that each token may see, which lie in
  pages of the cache.
- attn_mass: how much weight the queries gave to each entry, summed over heads and
  queries, on top of what earlier calls left.
- cache_evict: the entries of a sequence with the most weight (its first and last
  ones in any case), copied in order to other pages.
"""
import math
import random

import torch

own = False

D = 512           # latent width
G = 16            # channels per FP4 scale
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the queries of three decoding sequences, 16 heads: latency
        dict(name="rope_3x16", op="rope", n=3, heads=16, type="bf16", out="bf16", rot=64, halves=False, weight=True, extra=0),
        # a prompt chunk's latents from fp32, one slice of a wider projection, pairs half the rotated part apart
        dict(name="rope_latent_5003_f32", op="rope", n=5003, heads=1, type="f32", out="bf16", rot=64, halves=True, weight=True,
             extra=64),
        # the queries of a prompt chunk, 64 heads
        dict(name="rope_4096x64", op="rope", n=4096, heads=64, type="bf16", out="bf16", rot=64, halves=False, weight=False,
             extra=0),
        # one token of each of three short sequences, 16 heads: latency
        dict(name="chunk_3x1_1000", op="chunk", groups=3, nq=3, heads=16, n=1000, ragged=True, fresh=False, m=1, page=16,
             type="f16", part=1),
        # one token of each of 32 sequences over long contexts of very different lengths
        dict(name="chunk_32x1_65536", op="chunk", groups=32, nq=32, heads=64, n=65536, ragged=True, fresh=False, m=1, page=64,
             type="bf16", part=2),
        # chunks of four sequences' prompts behind what was cached before, two tokens to an entry
        dict(name="chunk_4x_601_30011", op="chunk", groups=4, nq=601, heads=20, n=30011, ragged=True, fresh=False, m=2, page=32,
             type="bf16", part=3),
        # a whole new prompt
        dict(name="chunk_prompt_2048", op="chunk", groups=1, nq=2048, heads=64, n=2048, ragged=False, fresh=True, m=1, page=128,
             type="bf16", part=4),
        # the weights of one token of each of three short sequences: latency
        dict(name="mass_3x1_1000", op="mass", groups=3, nq=3, heads=16, n=1000, ragged=True, fresh=False, m=1, page=16,
             type="bf16", part=5),
        # the weights of a decode step over long contexts
        dict(name="mass_32x1_65536", op="mass", groups=32, nq=32, heads=64, n=65536, ragged=False, fresh=False, m=1, page=64,
             type="bf16", part=6),
        # the weights that the last 64 tokens of a long prompt give to it
        dict(name="mass_64_32771", op="mass", groups=1, nq=64, heads=64, n=32771, ragged=False, fresh=False, m=1, page=64,
             type="f16", part=7),
        # five short sequences cut to 1,024 entries, one of them shorter than that
        dict(name="evict_5x4099", op="evict", groups=5, n=4099, keep=1024, first=4, last=128, d_idx=64, page=16, part=8),
        # eight long ones to a quarter, with their indexer keys
        dict(name="evict_8x131072", op="evict", groups=8, n=131072, keep=32768, first=64, last=1024, d_idx=128, page=64, part=9),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "mass", "evict"])
    part = rng.randrange(1 << 20)
    if op == "rope":
        heads = rng.choice([1, 1, 5, 16, 20, 64, 128])
        return dict(op=op, n=_spread(rng, 1, 262144 // heads), heads=heads, type=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f16", "f32"]), rot=rng.choice([0, 32, 64, 64, 128, 512]),
                    halves=rng.random() < 0.5, weight=rng.random() < 0.7, extra=rng.choice([0, 8, 64]))
    if op == "evict":
        groups = _spread(rng, 1, 32)
        n = _spread(rng, 2, 1048576 // groups)
        keep = _spread(rng, 1, max(1, min(n, 262144 // groups)))
        first = rng.randrange(0, keep // 2 + 1)
        return dict(op=op, groups=groups, n=n, keep=keep, first=first, last=rng.randrange(0, keep - first + 1),
                    d_idx=rng.choice([0, 64, 128]), page=rng.choice([16, 32, 64, 256]), part=part)
    heads = rng.choice([1, 5, 8, 16, 20, 32, 64, 64])
    groups = _spread(rng, 1, 32)
    nq = groups + _spread(rng, 1, 2000 if op == "chunk" else 64) - 1
    m = rng.choice([1, 1, 2])
    # at most the largest listed cases' products, entries and padded sizes of the plain form
    n = _spread(rng, 1, max(2, min((1 << 31) // (nq * heads * groups), 262144 // groups)))
    return dict(op=op, groups=groups, nq=nq, heads=heads, n=n, ragged=rng.random() < 0.7, fresh=rng.random() < 0.2, m=m,
                page=rng.choice([16, 32, 64, 256]), type=rng.choice(["bf16", "bf16", "f16"]), part=part)


def _layout(case):
    """New tokens, entries and first position of each group: the case alone says them."""
    g, r, m = case["groups"], random.Random(case["part"]), case["m"]
    if not case["ragged"]:
        each = [case["nq"] // g + (i < case["nq"] % g) for i in range(g)]
        lens = [case["n"]] * g
    else:
        cuts = sorted(r.sample(range(1, case["nq"]), g - 1)) if case["nq"] > 1 else []
        each = [b - a for a, b in zip([0] + cuts, cuts + [case["nq"]])]
        lens = [_spread(r, 1, case["n"]) for _ in range(g)]
        lens[r.randrange(g)] = case["n"]
    # a sequence holds its new tokens' entries; a fresh one holds no others
    lens = [c // m if case["fresh"] else max(k, c // m) for c, k in zip(each, lens)]
    pos = [max(0, k * m + r.randrange(m) - c) for c, k in zip(each, lens)]
    return each, lens, pos


def _kept_lens(case):
    r = random.Random(case["part"])
    lens = [_spread(r, max(1, case["n"] // 4), case["n"]) for _ in range(case["groups"])]
    lens[r.randrange(len(lens))] = case["n"]
    if len(lens) > 2:
        lens[r.randrange(len(lens))] = max(1, case["keep"] // 2)
    return lens


# ------------------------------------------------------------------ formats
def _e4m3(dtype):
    """Values of the bytes 0 .. 255 as E4M3."""
    return torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).to(dtype)


def _e2m1(dtype):
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-a for a in v], dtype=dtype, device=DEV)


def _decode(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], D // G, G)
    v = _e2m1(torch.float32)[c.int()] * _e4m3(torch.float32)[scales.int()].unsqueeze(-1)
    return v.reshape(codes.shape[0], D)


# ------------------------------------------------------------------ inputs
def _paged(case, gen, caps, keys):
    """A cache of random entries of about unit size in pages of a random order, of `caps` entries each."""
    p = case["page"]
    need = [-(-c // p) for c in caps]
    pages, most = sum(need), max(1, max(need))
    cap = max(8, -(-pages * p // 8) * 8)
    s = {"codes": torch.randint(0, 256, (cap, 256), dtype=torch.uint8, generator=gen, device=DEV),
         "scales": torch.randint(0x24, 0x34, (cap, 32), dtype=torch.uint8, generator=gen, device=DEV),
         "kidx": None, "kscale": None, "page": p}
    if keys:
        s["kidx"] = (torch.randn(cap, keys, generator=gen, device=DEV) * 100).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kscale"] = torch.exp2(torch.randint(-8, 0, (cap,), generator=gen, device=DEV).float())
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    first = torch.tensor([0] + need, device=DEV).cumsum(0)[:-1]
    at = first[:, None] + torch.arange(most, device=DEV)
    there = torch.arange(most, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    # (what lies behind a sequence's pages in the table is no page)
    s["table"] = torch.where(there, order[torch.where(there, at, 0)] if pages else -1, -1).to(torch.int32).contiguous()
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "rope":
        n, h, t = case["n"], case["heads"], TYPES[case["type"]]
        wide = torch.randn(n, h * D + case["extra"], generator=gen, device=DEV).mul_(3).to(t)
        x = wide[:, :h * D].unflatten(1, (h, D))              # one slice of a wider projection
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / max(1, half))
        # (positions of several sequences, up to a million tokens)
        start = torch.randint(0, 1 << 20, (1 + n // 64,), generator=gen, device=DEV)
        i = torch.arange(n, device=DEV)
        return {"op": "rope", "x": x, "out": torch.zeros(n, h, D, dtype=TYPES[case["out"]], device=DEV),
                "weight": 1 + 0.2 * torch.randn(D, generator=gen, device=DEV) if case["weight"] else None,
                "pos": (start[i // 64] + i % 64).to(torch.int32), "freq": freq.float(), "halves": case["halves"], "rot": case["rot"]}
    if case["op"] == "evict":
        lens, keep, g = _kept_lens(case), case["keep"], case["groups"]
        s = _paged(case, gen, lens + [min(n, keep) for n in lens], case["d_idx"])
        n = max(lens)
        # what accumulated weights look like: few large ones, many small, some exactly zero
        mass = torch.exp(2.5 * torch.randn(g, n, generator=gen, device=DEV) - 6)
        mass *= (torch.rand(g, n, generator=gen, device=DEV) > 0.05) * (torch.rand(g, n, generator=gen, device=DEV) > 0.05)
        most = min(n, keep)
        j = torch.arange(most, device=DEV)
        to = s["table"][g:].long().gather(1, (j // case["page"]).expand(g, most)) * case["page"] + j % case["page"]
        real = j < torch.tensor(lens, device=DEV).clamp(max=keep)[:, None]
        return s | {"op": "evict", "keep": keep, "first": case["first"], "last": case["last"], "mass": mass, "n": n,
                    "len": torch.tensor(lens, dtype=torch.int32, device=DEV), "to": s["table"][g:].contiguous(),
                    "table": s["table"][:g].contiguous(), "to_len": torch.zeros(g, dtype=torch.int32, device=DEV),
                    "kept": torch.full((g, keep), -1, dtype=torch.int32, device=DEV),
                    "mass_to": torch.zeros(g, keep, device=DEV), "rows": torch.where(real, to, -1).reshape(-1).contiguous(),
                    "back": torch.zeros(g * most, D, dtype=torch.bfloat16, device=DEV),
                    "key_back": torch.zeros(g * most, case["d_idx"], device=DEV) if case["d_idx"] else None}
    each, lens, pos = _layout(case)
    s = _paged(case, gen, lens, 0)
    nq, h, t = case["nq"], case["heads"], TYPES[case["type"]]
    off = [0]
    for c in each:
        off.append(off[-1] + c)
    s |= {"op": case["op"], "n": max(1, max(lens)), "most": max(each), "m": case["m"],
          "len": torch.tensor(lens, dtype=torch.int32, device=DEV), "seq": torch.arange(len(lens), dtype=torch.int32, device=DEV),
          "off": torch.tensor(off, dtype=torch.int32, device=DEV), "pos": torch.tensor(pos, dtype=torch.int32, device=DEV),
          # logits of standard deviation near 3
          "q": (torch.randn(nq, h, D, generator=gen, device=DEV) * (2.5 / math.sqrt(D))).to(t),
          "lse": torch.zeros(nq, h, device=DEV)}
    if case["op"] == "chunk":
        return s | {"out": torch.zeros(nq, h, D, dtype=t, device=DEV)}
    # each row's log sum as the attention leaves it, by the logits' spread
    i = torch.arange(nq, device=DEV)
    g = torch.searchsorted(s["off"][1:].long(), i, right=True)
    sees = ((s["pos"].long()[g] + i - s["off"].long()[g] + 1) // case["m"]).clamp(min=1).float()
    s["lse"] = (torch.log(sees) + 4.5)[:, None] + 0.2 * torch.randn(nq, h, generator=gen, device=DEV)
    s["prev"] = torch.rand(len(lens), s["n"], generator=gen, device=DEV) * 0.01
    return s | {"mass": torch.zeros(len(lens), s["n"], device=DEV), "decay": 0.9375}


# ------------------------------------------------------------------ one pass
def _own(s):
    import sparse_attention_decode_step_gb300 as csa
    if s["op"] == "rope":
        csa.norm_rope(s["x"], s["out"], weight=s["weight"], eps=1e-6, pos=s["pos"], inv_freq=s["freq"], halves=s["halves"])
        return [s["out"]]
    cache = csa.Cache.over(s["codes"], s["scales"], s["kidx"], s["kscale"], None, s["len"], s.get("m", 1))
    pages = csa.Pages(s["table"], s["page"])
    if s["op"] == "evict":
        to = csa.Cache.over(s["codes"], s["scales"], s["kidx"], s["kscale"], None, s["to_len"], 1)
        csa.cache_evict(cache, to, s["mass"], s["keep"], s["kept"], s["mass_to"], first=s["first"], last=s["last"], pages=pages,
                        to_pages=csa.Pages(s["to"], s["page"]))
        csa.cache_read(to, s["rows"], s["back"], s["key_back"])
        return {"kept": s["kept"], "len": s["to_len"], "mass": s["mass_to"], "x": s["back"], "key": s["key_back"]}
    groups = csa.Groups(s["seq"], s["off"])
    if s["op"] == "chunk":
        csa.chunk_attn(cache, groups, s["q"], s["out"], s["lse"], pos=s["pos"], pages=pages, max_n=s["n"])
        return {"out": s["out"], "lse": s["lse"]}
    csa.attn_mass(cache, groups, s["q"], s["lse"], s["mass"], pos=s["pos"], pages=pages, prev=s["prev"], decay=s["decay"], max_n=s["n"])
    return [s["mass"]]


def _rope(s):
    x, rot = s["x"].float(), s["rot"]
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    if s["weight"] is not None:
        y = y * s["weight"]
    if rot:
        a = s["pos"].double()[:, None, None] * s["freq"].double()
        c, b = torch.cos(a).float(), torch.sin(a).float()
        z = y[..., D - rot:]
        u, v = (z[..., :rot // 2], z[..., rot // 2:]) if s["halves"] else (z[..., 0::2], z[..., 1::2])
        u, v = u * c - v * b, u * b + v * c
        z = torch.cat([u, v], -1) if s["halves"] else torch.stack([u, v], -1).flatten(-2)
        y = torch.cat([y[..., :D - rot], z], -1)
    return [y.to(s["out"].dtype)]


def _evict(s):
    mass, n, keep = s["mass"], s["len"].long()[:, None], s["keep"]
    j = torch.arange(mass.shape[1], device=DEV)
    key = torch.where((j < s["first"]) | (j >= n - s["last"]), math.inf, mass)
    key = torch.where(j < n, key, -math.inf)
    top = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]      # (ties: the lower entry first)
    d = torch.arange(top.shape[1], device=DEV)
    real = d < n
    top = torch.sort(torch.where(real, top, mass.shape[1]), dim=1).values
    top = torch.where(real, top, 0)
    p = s["page"]
    src = (s["table"].long().gather(1, top // p) * p + top % p)[real]
    dst = (s["to"].long().gather(1, (d // p).expand_as(top)) * p + d % p)[real]
    for name in ("codes", "scales", "kidx", "kscale"):
        if s[name] is not None:
            s[name][dst] = s[name][src]
    kept, to = s["kept"].clone(), s["mass_to"].clone()
    kept[:, :top.shape[1]] = torch.where(real, top, -1).to(torch.int32)
    to[:, :top.shape[1]] = torch.where(real, mass.gather(1, top), 0.0)
    r, there = s["rows"].clamp(min=0), (s["rows"] >= 0)[:, None]
    x = torch.where(there, _decode(s["codes"][r], s["scales"][r]), 0.0).to(torch.bfloat16)
    key = None
    if s["kidx"] is not None:
        key = torch.where(there, _e4m3(torch.float32)[s["kidx"][r].int()] * s["kscale"][r].unsqueeze(-1), 0.0)
    return {"kept": kept, "len": s["len"].clamp(max=keep), "mass": to, "x": x, "key": key}


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "rope":
        return _rope(s)
    if s["op"] == "evict":
        return _evict(s)
    # groups padded to the longest: queries [g, most, h], entries [g, n]
    q, off, n, g = s["q"], s["off"].long(), s["len"].long(), s["len"].shape[0]
    most, h, p = s["most"], q.shape[1], s["page"]
    i = torch.arange(most, device=DEV)
    at = off[:-1, None] + i
    real = at < off[1:, None]
    at = torch.where(real, at, torch.zeros_like(at))
    j = torch.arange(s["n"], device=DEV)
    rows = torch.where(j < n[:, None], s["table"].long().gather(1, (j // p).expand(g, s["n"]).clamp(max=s["table"].shape[1] - 1)) * p + j % p, 0)
    v = _decode(s["codes"][rows.reshape(-1)], s["scales"][rows.reshape(-1)]).reshape(g, s["n"], D)
    x = (q.float()[at].reshape(g, most * h, D) @ v.transpose(1, 2)).reshape(g, most, h, s["n"])
    sees = torch.minimum((s["pos"].long()[:, None] + i + 1) // s["m"], n[:, None])
    seen = ((j < sees[..., None]) & real[..., None])[:, :, None]
    if s["op"] == "mass":
        w = torch.where(seen, torch.exp(x - s["lse"][at].unsqueeze(-1)), 0.0).sum((1, 2))
        return [torch.where(j < n[:, None], s["decay"] * s["prev"] + w, 0.0)]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(g, most * h, s["n"]) @ v).reshape(g, most, h, D) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": o[real].to(q.dtype), "lse": lse[real]}


def work(case):
    if case["op"] == "rope":
        rows = case["n"] * case["heads"]
        # squares, scaling, weight: 4 a channel; rotation 3 more
        return {"bytes": rows * D * (BYTES[case["type"]] + BYTES[case["out"]]) + case["n"] * 4, "flops": rows * (4 * D + 3 * case["rot"])}
    if case["op"] == "evict":
        lens, d = _kept_lens(case), case["d_idx"]
        kept = sum(min(n, case["keep"]) for n in lens)
        row = 288 + (d + 4 if d else 0)
        # weights, kept entries moved with their weights and numbers, and read back as values
        return {"bytes": sum(lens) * 4 + kept * (2 * row + 12 + row + 2 * D + 4 * d), "flops": 0}
    each, lens, pos = _layout(case)
    nq, h, e, m = case["nq"], case["heads"], BYTES[case["type"]], case["m"]
    sees = sum(min(n, (p + i + 1) // m) for c, n, p in zip(each, lens, pos) for i in range(c))
    if case["op"] == "mass":
        return {"bytes": sum(lens) * (288 + 8) + nq * h * (D * e + 4), "flops": 2 * D * h * sees}
    return {"bytes": sum(lens) * 288 + nq * h * (D * 2 * e + 4), "flops": 4 * D * h * sees}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _byte_value(b):
    """An E4M3 byte from its fields: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    v = [(1 + (i & 7) / 8) * 2.0 ** ((i >> 3) - 7) if i >> 3 else (i & 7) / 8 * 2.0 ** -6 for i in range(128)]
    return torch.tensor(v + [-a for a in v], dtype=torch.float64, device=DEV)[b.long()]


def _stored(codes, scales):
    c = torch.empty(codes.shape[0], D, dtype=torch.long, device=DEV)
    c[:, 0::2], c[:, 1::2] = (codes & 15).long(), (codes >> 4).long()
    v = [(1 + (i & 1) / 2) * 2.0 ** ((i >> 1) - 1) if i >> 1 else (i & 1) / 2 for i in range(8)]
    v = torch.tensor(v + [-a for a in v], dtype=torch.float64, device=DEV)
    return v[c] * _byte_value(scales).repeat_interleave(G, 1)


def _exact_rope(s):
    out = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
    rot = s["rot"]
    for k in range(0, out.shape[0], 512):            # some tokens at a time
        x = s["x"][k:k + 512].double()
        y = x / (x.pow(2).sum(2, keepdim=True) / D + 1e-6).sqrt()
        if s["weight"] is not None:
            y = y * s["weight"].double()
        if rot:
            angle = s["pos"][k:k + 512].double()[:, None] * s["freq"].double()[None]
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]
            tail = y[:, :, D - rot:]
            if s["halves"]:
                z = torch.complex(tail[:, :, :rot // 2].contiguous(), tail[:, :, rot // 2:].contiguous()) * turn
                y[:, :, D - rot:D - rot // 2], y[:, :, D - rot // 2:] = z.real, z.imag
            else:
                z = torch.view_as_complex(tail.unflatten(2, (rot // 2, 2)).contiguous()) * turn
                y[:, :, D - rot:] = torch.view_as_real(z).flatten(2)
        out[k:k + 512] = y
    return [out]


def _exact_evict(s, case):
    g, keep, p = s["len"].shape[0], case["keep"], case["page"]
    most = min(s["n"], keep)
    kept = torch.full((g, keep), -1, dtype=torch.int32, device=DEV)
    mass = torch.zeros(g, keep, dtype=torch.float64, device=DEV)
    x = torch.zeros(g, most, D, dtype=torch.float64, device=DEV)
    key = torch.zeros(g, most, case["d_idx"], dtype=torch.float64, device=DEV) if case["d_idx"] else None
    lens = _kept_lens(case)
    for b, n in enumerate(lens):
        inner = list(range(min(case["first"], n), max(min(case["first"], n), n - case["last"])))
        w = s["mass"][b].tolist()
        inner.sort(key=lambda j: (-w[j], j))
        outer = n - len(inner)
        chosen = sorted(set(range(n)) - set(inner) | set(inner[:max(0, min(n, keep) - outer)]))
        c = torch.tensor(chosen, device=DEV)
        kept[b, :len(chosen)] = c.to(torch.int32)
        mass[b, :len(chosen)] = s["mass"][b][c].double()
        r = s["table"][b].long()[torch.div(c, p, rounding_mode="floor")] * p + c % p
        x[b, :len(chosen)] = _stored(s["codes"][r], s["scales"][r])
        if key is not None:
            key[b, :len(chosen)] = _byte_value(s["kidx"][r]) * s["kscale"][r].double()[:, None]
    to_len = torch.tensor([min(n, keep) for n in lens], dtype=torch.int32, device=DEV)
    return {"kept": kept, "len": to_len, "mass": mass, "x": x.reshape(-1, D), "key": None if key is None else key.reshape(g * most, -1)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "evict":
        return _exact_evict(s, case)
    each, lens, pos = _layout(case)
    h, p, m = case["heads"], case["page"], case["m"]
    if case["op"] == "chunk":
        o = torch.zeros(case["nq"], h, D, dtype=torch.float64, device=DEV)
        lse = torch.full((case["nq"], h), -math.inf, dtype=torch.float64, device=DEV)
    else:
        mass = torch.zeros(len(lens), s["n"], dtype=torch.float64, device=DEV)
    at = 0
    for b, (c, n, first) in enumerate(zip(each, lens, pos)):
        j = torch.arange(n, device=DEV)
        r = s["table"][b].long()[j // p] * p + j % p
        v = _stored(s["codes"][r], s["scales"][r])
        for i in range(0, c, 8):                     # a few queries at a time
            k = min(c, i + 8)
            sees = torch.tensor([min(n, (first + t + 1) // m) for t in range(i, k)], device=DEV).repeat_interleave(h)
            x = s["q"][at + i:at + k].double().reshape(-1, D) @ v.T
            x = x.masked_fill(j[None] >= sees[:, None], -math.inf)
            if case["op"] == "mass":
                mass[b, :n] += torch.exp(x - s["lse"][at + i:at + k].double().reshape(-1, 1)).sum(0)
            elif n:
                l = torch.logsumexp(x, 1)
                w = torch.exp(x - l[:, None]).nan_to_num(0.0)
                o[at + i:at + k], lse[at + i:at + k] = (w @ v).reshape(k - i, h, D), l.reshape(k - i, h)
        if case["op"] == "mass":
            mass[b, :n] += 0.9375 * s["prev"][b, :n].double()
        at += c
    return [mass] if case["op"] == "mass" else {"out": o, "lse": lse}
