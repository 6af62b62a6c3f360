"""Operators over the FP4 latent cache, with their plain forms.

- cache_write / cache_read: latents (and FP8 indexer keys) quantised into given
  rows of a cache, and rows read back as the values they hold.
- dense_attn: attention of groups of queries over whole sequences of the cache.
  A group is either the queries of many sequences that share one prompt (its
  entries are read once for all of them, and the result is merged with each
  query's attention over its own entries), or the queries of one decoder
  sequence that attend to an encoder's entries of another length.
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
        # one new latent and key for each of 37 decoding sequences, read back at once: latency
        dict(name="write_37", op="write", n=37, cap=4096, type="bf16", d_idx=128, extra=128, part=1),
        # a prompt chunk's latents without keys (a cache that is only attended densely), f32
        dict(name="write_5003_f32", op="write", n=5003, cap=16384, type="f32", d_idx=0, extra=0, part=2),
        # a long prompt's latents, one slice of a wider projection, with narrow keys
        dict(name="write_65536", op="write", n=65536, cap=131072, type="bf16", d_idx=64, extra=64, part=3),
        # the window of one sequence replayed from the cache: latency
        dict(name="read_129", op="read", n=129, cap=8192, type="f16", d_idx=0, extra=0, part=4),
        # a whole long context in cache order, latents and keys
        dict(name="read_200003", op="read", n=200003, cap=262144, type="bf16", d_idx=128, extra=0, part=5),
        # two queries of 16 heads share a short prompt: latency
        dict(name="shared_2x16_700", op="dense", groups=1, nq=2, heads=16, n=700, ragged=False, prev=True, m=1,
             type="bf16", part=6),
        # a decode batch of 32 whose sequences all begin with the same 64K-token prompt
        dict(name="shared_32x64_65536", op="dense", groups=1, nq=32, heads=64, n=65536, ragged=False, prev=True, m=1,
             type="bf16", part=7),
        # 61 decoding sequences over 5 different prompts of 1 to 20,011 tokens
        dict(name="shared_61x64_5_prompts", op="dense", groups=5, nq=61, heads=64, n=20011, ragged=True, prev=True, m=1,
             type="bf16", part=8),
        # one token of each of 17 sequences to its encoder entries, m = 2, ragged lengths
        dict(name="cross_17x1_ragged", op="dense", groups=17, nq=17, heads=64, n=16384, ragged=True, prev=False, m=2,
             type="bf16", part=9),
        # one decoder query of a single sequence to a long encoder context
        dict(name="cross_1x1_131072", op="dense", groups=1, nq=1, heads=64, n=131072, ragged=False, prev=False, m=2,
             type="bf16", part=10),
        # four sequences' chunks of decoder queries, 20 heads, f16 queries and outputs
        dict(name="cross_4x_chunks", op="dense", groups=4, nq=601, heads=20, n=9001, ragged=True, prev=False, m=2,
             type="f16", part=11),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "dense", "dense"])
    part = rng.randrange(1 << 20)
    if op == "write":
        n = _spread(rng, 1, 65536)
        return dict(op=op, n=n, cap=n + _spread(rng, 1, 65536), type=rng.choice(["bf16", "f16", "f32"]),
                    d_idx=rng.choice([0, 64, 128]), extra=rng.choice([0, 8, 128]), part=part)
    if op == "read":
        n = _spread(rng, 1, 200000)
        return dict(op=op, n=n, cap=n + _spread(rng, 1, 60000), type=rng.choice(["bf16", "f16", "f32"]),
                    d_idx=rng.choice([0, 64, 128]), extra=rng.choice([0, 8, 128]), part=part)
    shared = rng.random() < 0.5
    heads = rng.choice([1, 5, 8, 16, 20, 32, 64, 64])
    groups = _spread(rng, 1, 6 if shared else 32)
    nq = groups + _spread(rng, 1, 64 if shared else 700) - 1
    # at most the largest listed case's products, and at most 131,072 entries in all
    n = _spread(rng, 1, max(2, min(65536 * 32 * 64 // (nq * heads), 131072 // groups)))
    return dict(op=op, groups=groups, nq=nq, heads=heads, n=n, ragged=rng.random() < 0.7, prev=shared,
                m=1 if shared else 2, type=rng.choice(["bf16", "bf16", "f16"]), part=part)


def _layout(case):
    """Queries and entries of each group of a dense case: the case alone says them."""
    g, r = case["groups"], random.Random(case["part"])
    if not case["ragged"]:
        each = [case["nq"] // g + (i < case["nq"] % g) for i in range(g)]
        return each, [case["n"]] * g
    cuts = sorted(r.sample(range(1, case["nq"]), g - 1)) if case["nq"] > 1 else []
    each = [b - a for a, b in zip([0] + cuts, cuts + [case["nq"]])]
    lens = [_spread(r, 1, case["n"]) for _ in range(g)]
    lens[r.randrange(g)] = case["n"]
    if g > 2:
        lens[r.randrange(g)] = 1
    return each, lens


# ------------------------------------------------------------------ formats
def _e4m3(dtype):
    """Values of the bytes 0 .. 255 as E4M3."""
    return torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).to(dtype)


def _e2m1(dtype):
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-a for a in v], dtype=dtype, device=DEV)


def _encode(x):
    """Rows of fp32 latents -> (codes, scales): per 16 channels the smallest E4M3 scale s with 6 s >= amax,
    each value to the nearest of s * {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code. All products are exact."""
    g = x.reshape(x.shape[0], D // G, G)
    a = g.abs()
    top = a.amax(-1, keepdim=True)
    steps = _e4m3(torch.float32)[1:127]
    at = torch.searchsorted(steps * 6.0, top).clamp(max=125)
    s = steps[at]
    c = ((a > 0.25 * s).to(torch.uint8) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) + (a > 2.5 * s)
         + (a >= 3.5 * s) + (a > 5.0 * s)).to(torch.uint8)
    c = torch.where((c > 0) & (g < 0), c + 8, c).reshape(x.shape[0], D // 2, 2)
    codes = c[..., 0] | (c[..., 1] << 4)
    scales = torch.where(top > 0, at + 1, 0).to(torch.uint8).reshape(x.shape[0], D // G)
    return codes, scales


def _decode(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], D // G, G)
    v = _e2m1(torch.float32)[c.int()] * _e4m3(torch.float32)[scales.int()].unsqueeze(-1)
    return v.reshape(codes.shape[0], D)


def _encode_key(k):
    """Rows of fp32 keys -> (E4M3 bytes, scale): the smallest power of two 2^e with 448 * 2^e >= amax (1 for zeros)."""
    top = k.abs().amax(-1)
    f, e = torch.frexp(top)                       # top = f * 2^e, f in [0.5, 1)
    e = torch.where(2 * f <= 1.75, e - 9, e - 8).int()
    s = ((e + 127) << 23).view(torch.float32)     # 2^e by its bits
    s = torch.where(top > 0, s, torch.ones_like(s))
    return (k / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8), s


# ------------------------------------------------------------------ inputs
def _cache(case, gen, base, m, filled):
    """The tensors of a cache; `filled`: with entries in every row."""
    cap, d = base[-1], case.get("d_idx", 0) or 64
    s = {"codes": torch.zeros(cap, 256, dtype=torch.uint8, device=DEV),
         "scales": torch.zeros(cap, 32, dtype=torch.uint8, device=DEV),
         "kidx": torch.zeros(cap, d, dtype=torch.uint8, device=DEV),
         "kscale": torch.ones(cap, device=DEV),
         "base": torch.tensor(base, dtype=torch.int64, device=DEV), "m": m}
    if filled:
        s["codes"], s["scales"] = _encode(torch.randn(cap, D, generator=gen, device=DEV))
        if case.get("d_idx"):
            s["kidx"], s["kscale"] = _encode_key(torch.randn(cap, d, generator=gen, device=DEV))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] in ("write", "read"):
        n, cap, t = case["n"], -(-case["cap"] // 8) * 8, TYPES[case["type"]]
        s = _cache(case, gen, [0, cap], 1, case["op"] == "read")
        s |= {"op": case["op"], "d_idx": case["d_idx"], "len": torch.full((1,), cap, dtype=torch.int32, device=DEV)}
        s["rows"] = torch.randperm(cap, generator=gen, device=DEV)[:n]
        wide = torch.zeros(n, D + case["extra"], dtype=t, device=DEV)
        s["x"] = wide[:, :D]                     # one slice of a wider row
        s["key"] = None
        if case["op"] == "write":
            s["x"].copy_(torch.randn(n, D, generator=gen, device=DEV))
            s["back"] = torch.zeros(n, D, dtype=t, device=DEV)
        if case["d_idx"]:
            s["key"] = torch.randn(n, case["d_idx"], generator=gen, device=DEV).to(t)
            s["key_back"] = torch.zeros(n, case["d_idx"], device=DEV)
        return s
    each, lens = _layout(case)
    base = [0]
    for c in lens:
        base.append(base[-1] + -(-c // 8) * 8)
    s = _cache(case, gen, base, case["m"], True)
    nq, h, t = case["nq"], case["heads"], TYPES[case["type"]]
    off = [0]
    for c in each:
        off.append(off[-1] + c)
    s |= {"op": "dense", "n": case["n"], "most": max(each), "len": torch.tensor(lens, dtype=torch.int32, device=DEV),
          "seq": torch.arange(len(lens), dtype=torch.int32, device=DEV),
          "off": torch.tensor(off, dtype=torch.int32, device=DEV),
          # logits of standard deviation 2.5 against latents of norm near sqrt(512)
          "q": (torch.randn(nq, h, D, generator=gen, device=DEV) * (2.5 / math.sqrt(D))).to(t),
          "out": torch.zeros(nq, h, D, dtype=t, device=DEV), "lse": torch.zeros(nq, h, device=DEV), "prev": None}
    if case["prev"]:
        # each query's attention over its own entries, as the sparse step leaves it
        s["prev"] = (torch.randn(nq, h, D, generator=gen, device=DEV) * 0.3,
                     torch.randn(nq, h, generator=gen, device=DEV) + 8.0)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        import sparse_attention_decode_step_gb300 as csa
        cache = csa.Cache.over(s["codes"], s["scales"], s["kidx"], s["kscale"], s["base"], s["len"], s["m"])
        if s["op"] == "write":
            csa.cache_write(cache, s["rows"], s["x"], s["key"])
            csa.cache_read(cache, s["rows"], s["back"], s["key_back"] if s["d_idx"] else None)
            return [s["back"], s["key_back"]] if s["d_idx"] else [s["back"]]
        if s["op"] == "read":
            csa.cache_read(cache, s["rows"], s["x"], s["key_back"] if s["d_idx"] else None)
            return [s["x"], s["key_back"]] if s["d_idx"] else [s["x"]]
        groups = csa.Groups(s["seq"], s["off"])
        csa.dense_attn(cache, groups, s["q"], s["out"], s["lse"], prev=s["prev"], max_n=s["n"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "write":
        r = s["rows"]
        s["codes"][r], s["scales"][r] = _encode(s["x"].float())
        if s["d_idx"]:
            s["kidx"][r], s["kscale"][r] = _encode_key(s["key"].float())
    if s["op"] in ("write", "read"):
        r = s["rows"]
        out = [_decode(s["codes"][r], s["scales"][r]).to(s["x"].dtype)]
        if s["d_idx"]:
            out.append(_e4m3(torch.float32)[s["kidx"][r].int()] * s["kscale"][r].unsqueeze(-1))
        return out
    # groups padded to the longest: queries [g, most, h], entries [g, n]
    q, off, n = s["q"], s["off"].long(), s["len"].long()
    most, h = s["most"], q.shape[1]
    at = off[:-1, None] + torch.arange(most, device=DEV)
    real = at < off[1:, None]
    at = torch.where(real, at, torch.zeros_like(at))
    j = torch.arange(s["n"], device=DEV)
    seen = j < n[:, None]
    rows = torch.where(seen, s["base"][:-1, None] + j, torch.zeros_like(j))
    v = _decode(s["codes"][rows.reshape(-1)], s["scales"][rows.reshape(-1)]).reshape(len(n), s["n"], D)
    x = q.float()[at].reshape(len(n), most * h, D) @ v.transpose(1, 2)
    x = torch.where(seen[:, None], x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = ((p @ v) / total).reshape(len(n), most, h, D)[real]
    lse = (top + torch.log(total)).reshape(len(n), most, h)[real]
    if s["prev"] is not None:
        po, pl = s["prev"]
        both = torch.maximum(lse, pl)
        a, b = torch.exp(lse - both), torch.exp(pl - both)
        o = (o * a.unsqueeze(-1) + po * b.unsqueeze(-1)) / (a + b).unsqueeze(-1)
        lse = both + torch.log(a + b)
    return {"out": o.to(q.dtype), "lse": lse}


def work(case):
    if case["op"] in ("write", "read"):
        n, d, e = case["n"], case["d_idx"], BYTES[case["type"]]
        stored = n * (288 + (d + 4 if d else 0) + 8)          # bytes of a row and its number
        out = n * (D * e + 4 * d)
        return {"bytes": stored + out + (n * (D + d) * e if case["op"] == "write" else 0), "flops": 0}
    each, lens = _layout(case)
    nq, h, e = case["nq"], case["heads"], BYTES[case["type"]]
    b = sum(lens) * 288 + nq * h * (D * 2 * e + 4) + (nq * h * (D + 1) * 4 if case["prev"] else 0)
    return {"bytes": b, "flops": 4 * D * h * sum(c * n for c, n in zip(each, lens))}


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


def _nearest(x):
    """The value that each latent is held as: the nearest of the group's eight, of two as near the even one."""
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    every = _byte_value(torch.arange(1, 127, device=DEV))
    out = torch.empty_like(x)
    for i in range(0, x.shape[0], 8192):
        g = x[i:i + 8192].reshape(-1, G)
        top = g.abs().amax(1)
        s = every[(every[None] * 6 < top[:, None]).sum(1).clamp(max=125)]
        far = (g.abs()[..., None] - levels * s[:, None, None]).abs()
        even, odd = far[..., 0::2].min(-1), far[..., 1::2].min(-1)
        k = torch.where(even.values <= odd.values, 2 * even.indices, 2 * odd.indices + 1)
        out[i:i + 8192] = (levels[k] * s[:, None] * g.sign()).reshape(-1, D)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        out = [_nearest(s["x"].double())]
        if case["d_idx"]:
            k = s["key"].double()
            power = torch.tensor([2.0 ** i for i in range(-140, 130)], dtype=torch.float64, device=DEV)
            scale = power[(448 * power < k.abs().amax(1, keepdim=True)).sum(1)]
            y = k / scale[:, None]
            # steps of 2^-9 below 2^-6, else an eighth of the power of two below
            below = power[torch.searchsorted(power, y.abs(), right=True).clamp(min=1) - 1].clamp(min=2.0 ** -6)
            out.append(torch.round(y / below * 8) / 8 * below * scale[:, None])
        return out
    if case["op"] == "read":
        r = s["rows"]
        out = [_stored(s["codes"][r], s["scales"][r])]
        if case["d_idx"]:
            out.append(_byte_value(s["kidx"][r]) * s["kscale"][r].double()[:, None])
        return out
    each, lens = _layout(case)
    o = torch.empty(case["nq"], case["heads"], D, dtype=torch.float64, device=DEV)
    lse = torch.empty(case["nq"], case["heads"], dtype=torch.float64, device=DEV)
    at, row = 0, 0
    for c, n in zip(each, lens):
        v = _stored(s["codes"][row:row + n], s["scales"][row:row + n])
        for i in range(at, at + c, 8):           # a few queries at a time
            k = min(at + c, i + 8)
            x = s["q"][i:k].double().reshape(-1, D) @ v.T
            l = torch.logsumexp(x, 1)
            z = torch.exp(x - l[:, None]) @ v
            if s["prev"] is not None:
                pl = s["prev"][1][i:k].double().reshape(-1)
                both = torch.logaddexp(l, pl)
                z = z * torch.exp(l - both)[:, None] + s["prev"][0][i:k].double().reshape(-1, D) * torch.exp(pl - both)[:, None]
                l = both
            o[i:k], lse[i:k] = z.reshape(k - i, -1, D), l.reshape(k - i, -1)
        at, row = at + c, row + -(-n // 8) * 8
    return {"out": o, "lse": lse}
