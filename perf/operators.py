"""The 4-bit operators: what is measured of them, and their plain forms.

Weights (nib): W[n, k] = mu[n, k / group] + scale[n, k / group] (c[n, k] - 8), c in 0 .. 15, fp16 scale and
optional fp16 mu per (row, group), group 32, 64 or 128. Held as
  codes  int32 [ceil(N / 16), K / 128, 256]: word ((h 8 + g) 4 + q) 4 + j of a block holds row 8 h + g of the strip,
         columns 32 j + 8 q .. + 7 of the 128; nibble p of a word is column 2 (p % 4) + p / 4 of its eight;
  scale, mu  fp16 [ceil(N / 16), K / group, 16], row r of the strip at 2 (r % 8) + r / 8.
Operators: fit (dense fp16 W to this form, and back to fp16), linear (y = x W^T).

Cache: K and V of past tokens in pages, 4-bit codes c with fp16 scale s and zero z per token and 64 entries of a
head: value = z + s c. uint8 pool [pages, kv heads, page / 16, 18 D]: 16 tokens as K codes, V codes (8 D bytes each),
K scales, V scales (D bytes each):
  K codes  word ((h 8 + g) 4 + q) D / 32 + j: token 8 h + g, entries 32 j + 8 q .. + 7 (nibbles as above);
  V codes  word ((h 8 + g) 4 + q) D / 32 + j: tokens 8 h + 2 q (nibbles p = 0 .. 3) and 8 h + 2 q + 1 (nibbles p + 4),
           entry 16 (2 j + p / 2) + 8 (p % 2) + g;
  K scales fp16 [16 tokens, D / 64, 2] (s, z);
  V scales fp16 [4 q, D / 64, 2 (s, z), 4]: tokens 2 q, 2 q + 1, 2 q + 8, 2 q + 9.
Operators: append (quantise new K and V into the pages; read back as fp16), attention (of the last tokens of each
sequence over its pages, with an optional window and always visible first tokens)."""
import math

import torch

own = False

F16, F32, F64 = torch.float16, torch.float32, torch.float64


def listed():
    return [
        # a small projection of a 2560-wide model quantised on load
        {"name": "fit 1024x2560", "op": "fit", "N": 1024, "K": 2560, "group": 128, "offset": True},
        # the largest projection of a 4096-wide model, small groups, no offset
        {"name": "fit 4096x12288 g64", "op": "fit", "N": 4096, "K": 12288, "group": 64, "offset": False},
        # one decoded token through the smallest projection: latency
        {"name": "linear 1x1024x2560", "op": "linear", "M": 1, "N": 1024, "K": 2560, "group": 128, "offset": False},
        # one decoded token through the widest projection
        {"name": "linear 1x12288x4096", "op": "linear", "M": 1, "N": 12288, "K": 4096, "group": 128, "offset": True},
        # an output head with an odd number of rows, a few sequences at once, the smallest groups
        {"name": "linear 6x65543x2560 g32", "op": "linear", "M": 6, "N": 65543, "K": 2560, "group": 32, "offset": True},
        # a prompt through the widest projection
        {"name": "linear 2048x12288x4096", "op": "linear", "M": 2048, "N": 12288, "K": 4096, "group": 128, "offset": False},
        # one new token of each of 64 sequences
        {"name": "append 64x1", "op": "append", "B": 64, "T": 1, "Hk": 8, "D": 128, "page": 64, "cap": 4096},
        # four prompts of different lengths
        {"name": "append 4x4000", "op": "append", "B": 4, "T": 4000, "Hk": 8, "D": 128, "page": 64, "cap": 8192},
        # a chat that has just begun, small heads: latency
        {"name": "attention 2 of 500", "op": "attention", "B": 2, "T": 1, "G": 4, "Hk": 8, "D": 64, "page": 16, "longest": 500, "window": 0, "sinks": 0},
        # serving 64 sequences of all lengths
        {"name": "attention 64 to 8192", "op": "attention", "B": 64, "T": 1, "G": 4, "Hk": 8, "D": 128, "page": 64, "longest": 8192, "window": 0, "sinks": 0},
        # one very long document, four drafted tokens to verify
        {"name": "attention 1 of 131072 drafts", "op": "attention", "B": 1, "T": 4, "G": 4, "Hk": 8, "D": 128, "page": 128, "longest": 131072, "window": 0, "sinks": 0},
        # streaming over long texts: a window and four first tokens
        {"name": "attention 32 window 1000", "op": "attention", "B": 32, "T": 1, "G": 8, "Hk": 4, "D": 128, "page": 32, "longest": 16384, "window": 1000, "sinks": 4},
    ]


def spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("fit", "linear", "linear", "append", "attention", "attention"))
    if op == "fit":
        return {"op": op, "N": spread(rng, 64, 8192), "K": 128 * spread(rng, 4, 48), "group": rng.choice((32, 64, 128)), "offset": rng.random() < 0.5}
    if op == "linear":
        M = rng.choice((1, spread(rng, 2, 16), spread(rng, 17, 128), spread(rng, 129, 2000)))
        return {"op": op, "M": M, "N": spread(rng, 64, 12000), "K": 128 * spread(rng, 4, 32), "group": rng.choice((32, 64, 128)), "offset": rng.random() < 0.5}
    Hk, D, page = rng.choice((1, 2, 4, 8)), rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
    B = spread(rng, 1, 64)
    if op == "append":
        T = spread(rng, 1, 4000 // B + 1)
        return {"op": op, "B": B, "T": T, "Hk": Hk, "D": D, "page": page, "cap": -(-(T + rng.randrange(1, 2000)) // page) * page}
    longest = spread(rng, 40, max(41, 131072 // B))
    window = rng.choice((0, spread(rng, 16, 4000)))
    return {"op": op, "B": B, "T": rng.choice((1, 1, rng.randrange(2, 9))), "G": rng.choice((1, 2, 3, 4, 8)), "Hk": Hk, "D": D, "page": page, "longest": longest,
            "window": window, "sinks": rng.choice((0, rng.randrange(1, 40))) if window else 0}


def work(case):
    c = case
    if c["op"] == "fit":
        n, g = c["N"] * c["K"], c["N"] * (c["K"] // c["group"])
        held = n / 2 + 2 * g * (2 if c["offset"] else 1)
        return {"bytes": 2 * n + held + held + 2 * n, "flops": 6 * n}
    if c["op"] == "linear":
        n, g = c["N"] * c["K"], c["N"] * (c["K"] // c["group"])
        return {"bytes": n / 2 + 2 * g * (2 if c["offset"] else 1) + 2 * c["M"] * (c["K"] + c["N"]), "flops": 2 * c["M"] * n}
    if c["op"] == "append":
        n = sum(counts_of(c))
        values = 2 * n * c["Hk"] * c["D"]
        held = n * c["Hk"] * 18 * c["D"] / 16
        return {"bytes": 2 * values + held + held + 2 * 2 * c["B"] * c["T"] * c["Hk"] * c["D"], "flops": 6 * values}
    pairs = tokens = 0
    for n in lens_of(c):
        first = max(c["sinks"], n - c["T"] + 1 - c["window"]) if c["window"] else 0
        tokens += n - first + min(c["sinks"], n, first)
        for i in range(max(0, n - c["T"]), n):
            seen = i + 1
            if c["window"]:
                seen = min(c["window"], i + 1) + max(0, min(c["sinks"], i + 1 - c["window"]))
            pairs += seen
    H = c["Hk"] * c["G"]
    return {"bytes": tokens * c["Hk"] * 18 * c["D"] / 16 + 4 * c["B"] * c["T"] * H * c["D"], "flops": 4 * pairs * H * c["D"]}


def counts_of(c):
    """New tokens of each sequence of a padded batch: all T of the first, fewer of the others where T > 1."""
    return [c["T"] if b == 0 or c["T"] == 1 else max(1, c["T"] - (c["T"] * ((7 * b) % 16)) // 32) for b in range(c["B"])]


def lens_of(c):
    """Cached tokens of each sequence, its new ones among them: the longest, and a spread of shorter ones."""
    return [c["longest"] if b == 0 else max(c["T"], (c["longest"] * (1 + (11 * b) % 16)) // 16 - (5 * b) % 13) for b in range(c["B"])]


def tables(sizes, page, width, gen):
    """Page tables [B, width] over a shuffled pool, -1 where a sequence has no page, and the pool's pages."""
    need = [-(-n // page) for n in sizes]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int64)
    have = torch.tensor(need, device="cuda")[:, None]
    at = torch.cumsum(have, 0) - have + torch.arange(width, device="cuda")[None]
    return torch.where(torch.arange(width, device="cuda")[None] < have, order[at.clamp(max=pages - 1)], -1).to(torch.int32), pages


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=F32)

    def words(*shape):
        return torch.randint(-(1 << 31), 1 << 31, shape, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)

    def uniform(lo, hi, *shape):
        return (torch.rand(shape, generator=gen, device="cuda", dtype=F32) * (hi - lo) + lo).to(F16)

    s = {"case": dict(c)}
    if c["op"] == "fit":
        s["W"] = (normal(c["N"], c["K"]) * 0.02).to(F16)
    elif c["op"] == "linear":
        N, K, strips = c["N"], c["K"], -(-c["N"] // 16)
        s["codes"] = words(strips, K // 128, 256)
        s["scale"] = uniform(0.005, 0.02, strips, K // c["group"], 16)
        s["mu"] = uniform(-0.01, 0.01, strips, K // c["group"], 16) if c["offset"] else None
        s["x"] = normal(c["M"], K).to(F16)
    elif c["op"] == "append":
        B, T, Hk, D, page = (c[k] for k in ("B", "T", "Hk", "D", "page"))
        counts = counts_of(c)
        start = [(37 * b + seed) % (c["cap"] - T + 1) for b in range(B)]
        s["table"], pages = tables([a + n for a, n in zip(start, counts)], page, c["cap"] // page, gen)
        s["start"], s["counts"] = (torch.tensor(v, device="cuda", dtype=torch.int32) for v in (start, counts))
        s["k"], s["v"] = ((normal(B, T, Hk, D) * (0.5 + torch.rand(Hk, D, generator=gen, device="cuda"))).to(F16) for _ in range(2))
        s["pool"] = torch.zeros(pages, Hk, page // 16, 18 * D, device="cuda", dtype=torch.uint8)
    else:
        B, T, Hk, D, page = (c[k] for k in ("B", "T", "Hk", "D", "page"))
        lens = lens_of(c)
        s["table"], pages = tables(lens, page, -(-max(lens) // page), gen)
        s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        units = pages * Hk * (page // 16)
        # codes of all values; scales as a head of unit spread has them, zeros near the range's lower end
        s["pool"] = words(units, 9 * D // 2).view(torch.uint8).view(pages, Hk, page // 16, 18 * D)
        scales = s["pool"].view(F16).view(units, 9 * D)
        step, zero = uniform(0.1, 0.4, units, D // 2), uniform(0.8, 1.2, units, D // 2)
        zero = (step.float() * -7.5 * zero.float()).to(F16)
        scales[:, 8 * D:8 * D + D // 2].view(units, 16, D // 64, 2).copy_(torch.stack([step[:, :D // 4], zero[:, :D // 4]], -1).view(units, 16, D // 64, 2))
        scales[:, 8 * D + D // 2:].view(units, 4, D // 64, 2, 4).copy_(torch.stack([step[:, D // 4:].view(units, 4, D // 64, 4), zero[:, D // 4:].view(units, 4, D // 64, 4)], 3))
        s["q"] = normal(B, T, Hk * c["G"], D).to(F16)
    if own:
        from ternary_weight_only_tern_b200 import api

        if c["op"] == "linear":
            s["w"] = api.NibWeight(c["N"], c["K"], c["group"], s["codes"], s["scale"], s["mu"], static=True)
        elif c["op"] in ("append", "attention"):
            s["cache"] = api.PagedCache(s["pool"])
    return s


# ------------------------------------------------------------------------------ the layouts, in torch

def nibbles(words):
    """int32 [...] -> the 8 nibbles [..., 8] of each word."""
    return (words[..., None] >> torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)) & 15


def rows_of(tiles, entries):
    """Words [..., 128 * entries / 64] of 16 rows of `entries` (32 j + 8 q + i) -> codes [..., 16, entries]."""
    j = entries // 32
    n = nibbles(tiles.reshape(*tiles.shape[:-1], 16, 4, j))                      # [..., row, q, j, p]
    n = n.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-2)                    # [..., row, q, j, i]
    return n.transpose(-2, -3).flatten(-3)                                       # [..., row, j q i]


def weight_codes(words, N):
    t = rows_of(words, 128)                                                      # [strips, K / 128, 16, 128]
    return t.transpose(1, 2).flatten(2).flatten(0, 1)[:N]


def weight_scales(scale, N, to):
    return scale.unflatten(-1, (8, 2)).transpose(-1, -2).flatten(-2).transpose(1, 2).flatten(0, 1)[:N].to(to)


def dequant_weight(s, to):
    c = s["case"]
    w = (weight_codes(s["codes"], c["N"]) - 8).to(to).unflatten(1, (-1, c["group"])) * weight_scales(s["scale"], c["N"], to)[..., None]
    if s["mu"] is not None:
        w += weight_scales(s["mu"], c["N"], to)[..., None]
    return w.flatten(1)


def unit_values(units, D, to):
    """uint8 [n, 18 D] blocks of 16 tokens -> K, V [n, 16, D]."""
    w = units.view(torch.int32)
    sc = units.view(F16)[:, 8 * D:]
    ks = sc[:, :D // 2].reshape(-1, 16, D // 64, 2).to(to)
    K = rows_of(w[:, :2 * D], D).to(to).unflatten(-1, (D // 64, 64)) * ks[..., :1] + ks[..., 1:]
    n = nibbles(w[:, 2 * D:4 * D].reshape(-1, 2, 8, 4, D // 32)).unflatten(-1, (2, 2, 2))  # [n, h, g, q, j, odd, p / 2, p % 2]
    vc = n.permute(0, 1, 3, 5, 4, 6, 7, 2).reshape(-1, 16, D)
    vs = sc[:, D // 2:].reshape(-1, 4, D // 64, 2, 2, 2).permute(0, 4, 1, 5, 2, 3).reshape(-1, 16, D // 64, 2).to(to)  # [n, q, grp, sz, h, odd] -> token
    V = vc.to(to).unflatten(-1, (D // 64, 64)) * vs[..., :1] + vs[..., 1:]
    return K.flatten(-2), V.flatten(-2)


def cached(s, L, to):
    """K, V [B, Hk, L, D] of the first L tokens of every sequence (zero where there is no page)."""
    c = s["case"]
    page, D, Hk, pool, table = c["page"], c["D"], c["Hk"], s["pool"], s["table"]
    P = -(-L // page)
    units = pool[table[:, :P].clamp(min=0).long()]                               # [B, P, Hk, page / 16, 18 D]
    units = units.transpose(1, 2).reshape(-1, 18 * D)
    K, V = unit_values(units, D, to)
    return tuple(t.view(-1, Hk, P * page, D)[:, :, :L] for t in (K, V))


# ------------------------------------------------------------------------------ quantising, in `to`

def quantise(x, lo, scale, bias, to):
    """Codes of x [..., g] for fp16 scale and zero (value = zero + scale (c - bias))."""
    s, z = scale.to(to)[..., None], lo.to(to)[..., None]
    return torch.where(s > 0, torch.round((x - z) / torch.where(s > 0, s, 1)) + bias, bias).clamp(0, 15)


def fit(W, group, offset, to):
    w = W.to(to).unflatten(1, (-1, group))
    if offset:
        lo, hi = w.amin(-1), w.amax(-1)
        s = ((hi - lo) / torch.full_like(lo, 15)).to(F16)
        mu = (lo + 8 * s.to(to)).to(F16)
    else:
        s = w.abs().amax(-1)
        s = (s / torch.full_like(s, 7)).to(F16)
        mu = torch.zeros_like(s)
    c = quantise(w, mu, s, 8, to)
    return (mu.to(to)[..., None] + s.to(to)[..., None] * (c - 8)).flatten(1)


def store(x, to):
    """What the cache holds of x [..., D]."""
    g = x.to(to).unflatten(-1, (-1, 64))
    lo, hi = g.amin(-1), g.amax(-1)
    s, z = ((hi - lo) / torch.full_like(lo, 15)).to(F16), lo.to(F16)
    return (z.to(to)[..., None] + s.to(to)[..., None] * quantise(g, z, s, 0, to)).flatten(-2)


def attend(q, K, V, s, to):
    """softmax(q K^T / sqrt(D)) V over the visible tokens; q [B, T, H, D], K and V [B, Hk, L, D]."""
    c = s["case"]
    B, T, Hk, G, D, L = c["B"], c["T"], c["Hk"], c["G"], c["D"], K.shape[2]
    x = q.to(to).view(B, T, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * T, D)
    p = (x @ K.transpose(-1, -2)) * (1 / math.sqrt(D))
    at = s["lens"].long()[:, None] - T + torch.arange(T, device=q.device)[None]  # [B, T] the queries' places
    j = torch.arange(L, device=q.device)
    seen = j <= at[..., None]
    if c["window"]:
        seen &= (j > at[..., None] - c["window"]) | (j < c["sinks"])
    p = p.view(B, Hk, G, T, L).masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    o = p.view(B, Hk, G * T, L) @ V
    return o.view(B, Hk, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, Hk * G, D)


def padded(v, counts):
    """v [B, T, ...] with zeros behind each sequence's tokens."""
    here = torch.arange(v.shape[1], device=v.device)[None] < counts[:, None]
    return torch.where(here[..., None, None], v, 0)


# ------------------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if own:
        from ternary_weight_only_tern_b200 import api

        if c["op"] == "fit":
            return api.nib_dequant(api.nib_fit(s["W"], group=c["group"], offset=c["offset"]))
        if c["op"] == "linear":
            return api.nib_linear(s["x"], s["w"])
        if c["op"] == "append":
            api.cache_append(s["cache"], s["k"], s["v"], s["table"], s["start"], s["counts"])
            return api.cache_read(s["cache"], s["table"], s["start"], c["T"], s["counts"])
        return api.cache_attention(s["q"], s["cache"], s["table"], s["lens"], window=c["window"], sinks=c["sinks"])
    if c["op"] == "fit":
        return fit(s["W"], c["group"], c["offset"], F32).to(F16)
    if c["op"] == "linear":
        return (s["x"].to(F32) @ dequant_weight(s, F32).t()).to(F16)
    if c["op"] == "append":
        return tuple(padded(store(t, F32), s["counts"]).to(F16) for t in (s["k"], s["v"]))
    K, V = cached(s, c["longest"], F32)
    return attend(s["q"], K, V, s, F32).to(F16)


# ------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits, one row, head or sequence at a time."""
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "fit":
        G, out = c["group"], []
        for rows in s["W"].split(256):
            w = rows.double().reshape(len(rows), -1, G)
            if c["offset"]:
                step = ((w.max(-1)[0] - w.min(-1)[0]) / 15).half().double().unsqueeze(-1)
                mid = (w.min(-1, keepdim=True)[0] + 8 * step).half().double()
            else:
                step = (w.abs().max(-1)[0] / 7).half().double().unsqueeze(-1)
                mid = torch.zeros_like(step)
            level = torch.clamp(torch.nan_to_num(torch.round((w - mid) / step)), -8, 7)
            out.append((mid + step * level).reshape(len(rows), -1))
        return torch.cat(out)
    if c["op"] == "linear":
        N, K, G = c["N"], c["K"], c["group"]
        x, out = s["x"].double(), torch.empty(c["M"], N, device="cuda", dtype=F64)
        # where row r, column k of a strip's 128 lies: word, shift, scale
        k = torch.arange(128, device="cuda")
        j, q, i = k // 32, k % 32 // 8, k % 8
        shift = (4 * (i // 2 + 4 * (i % 2))).to(torch.int32)
        for r in range(16):
            word = ((r // 8 * 8 + r % 8) * 4 + q) * 4 + j
            place = 2 * (r % 8) + r // 8
            rows = (N - r + 15) // 16
            if rows <= 0:
                continue
            for part in torch.arange(rows, device="cuda").split(1024):
                code = (s["codes"][part][:, :, word] >> shift) & 15                # [rows, K / 128, 128]
                w = (code.double() - 8).reshape(len(part), K // G, G) * s["scale"][part][:, :, place].double()[..., None]
                if s["mu"] is not None:
                    w = w + s["mu"][part][:, :, place].double()[..., None]
                out[:, part * 16 + r] = x @ w.reshape(len(part), K).t()
        return out
    if c["op"] == "append":
        out = []
        for t in (s["k"], s["v"]):
            o = torch.zeros(t.shape, device="cuda", dtype=F64)
            for b, n in enumerate(counts_of(c)):
                for d in range(0, c["D"], 64):
                    y = t[b, :n, :, d:d + 64].double()
                    z = y.min(-1, keepdim=True)[0]
                    step = ((y.max(-1, keepdim=True)[0] - z) / 15).half().double()
                    o[b, :n, :, d:d + 64] = z + step * torch.clamp(torch.nan_to_num(torch.round((y - z) / step)), 0, 15)
            out.append(o)
        return tuple(out)
    B, T, Hk, G, D, page = (c[k] for k in ("B", "T", "Hk", "G", "D", "page"))
    out = torch.zeros(B, T, Hk * G, D, device="cuda", dtype=F64)
    d = torch.arange(D, device="cuda")
    jk, qk, ik = d // 32, d % 32 // 8, d % 8
    tile, half, gv = d // 16, d % 16 // 8, d % 8
    for b, n in enumerate(lens_of(c)):
        t = torch.arange(n, device="cuda")
        pages = s["table"][b].long()[t // page]
        for h in range(Hk):
            K, V = (torch.empty(n, D, device="cuda", dtype=F64) for _ in range(2))
            for a in range(0, n, 20000):
                tt = t[a:a + 20000]
                u = s["pool"][pages[a:a + 20000], h, tt % page // 16].contiguous()
                r = (tt % 16)[:, None]
                w, f = u.view(torch.int32), u.view(F16)
                kc = w.gather(1, ((r * 4 + qk) * (D // 32) + jk).long()) >> (4 * (ik // 2 + 4 * (ik % 2))).to(torch.int32) & 15
                vword = 2 * D + ((r // 8 * 8 + gv) * 4 + r % 8 // 2) * (D // 32) + tile // 2
                vc = w.gather(1, vword.long()) >> (4 * (2 * (tile % 2) + half) + 16 * (r % 2)).to(torch.int32) & 15
                ka = 8 * D + (r * (D // 64) + d // 64) * 2
                va = 8 * D + D // 2 + ((r % 8 // 2) * (D // 64) + d // 64) * 8 + r // 8 * 2 + r % 2
                K[a:a + 20000] = f.gather(1, ka + 1).double() + f.gather(1, ka).double() * kc.double()
                V[a:a + 20000] = f.gather(1, va + 4).double() + f.gather(1, va).double() * vc.double()
            for i in range(T):
                place = n - T + i
                see = t <= place
                if c["window"]:
                    see = see & ((t > place - c["window"]) | (t < c["sinks"]))
                q = s["q"][b, i, h * G:(h + 1) * G].double()
                out[b, i, h * G:(h + 1) * G] = torch.softmax(q @ K[see].t() / math.sqrt(D), -1) @ V[see]
    return out
