"""Cases, plain forms and exact values of the paged 4-bit cache's operators.

The cache holds keys and values as the codec holds them: random signs and a
Walsh-Hadamard transform over head_dim, then 4-bit codes with an fp16 scale and
zero per group. Four operators work on it:

  write   quantises new tokens' keys and values into slots of the cache
  read    gives the stored rows back, inverse transform included
  attend  attention of query tokens over the requests' pages
  load    puts the codes of a compressed stream into slots, as they are

A write and a load leave 4-bit state behind, so their passes end with a read of
the rows they stored: the values are what is compared.

Layout of the pool, [layers][pages][2 (K, V)][kv_heads][block], bytes: a block
holds page_tokens / 16 tiles of 16 tokens; a tile holds the 16 tokens' codes
(head_dim / 2 bytes each, low nibble first), then their group meta (fp16 scale,
fp16 zero per group), both x 2^-k, k = 3. A key's 4-byte words and a value's
2-byte halfwords, in channel order [groups of 32 channels][4 or 8], are stored
transposed: [4 or 8][groups of 32 channels].
"""
import math
import random

import torch

own = False

K_SCALE = 8.0  # meta is stored x 2^-3 for head_dim 64 and 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a decode step's new tokens: 64 requests, one layer, ASYM g128 (the 8B shape)
        case("write step", op="write", layers=1, heads=8, dim=128, group=128, tokens=64, pages=4096,
             page=16, dtype="bf16"),
        # a 4096-token prompt entering all 32 layers
        case("write prompt", op="write", layers=32, heads=8, dim=128, group=128, tokens=4096,
             pages=300, page=16, dtype="bf16"),
        # head_dim 64, fp16 slices of a fused qkv, some padding tokens, ragged count
        case("write d64 fused", op="write", layers=6, heads=5, dim=64, group=32, tokens=1733,
             pages=90, page=32, dtype="fp16", quant=1, signs=1, fused=True, skip=7),
        # one short request read back for another engine's use
        case("read short", op="read", layers=1, heads=5, dim=64, group=64, tokens=203, pages=40,
             page=32, dtype="fp16", quant=1),
        # 16 requests of 512..8192 tokens in 16-token pages (the paged batch), 4 layers
        case("read batch", op="read", layers=4, heads=8, dim=128, group=64, tokens=69632, pages=4600,
             page=16, dtype="bf16"),
        # one request's decode step, 4096 tokens, 32 query / 8 kv heads
        case("decode one", op="attend", layers=1, heads=8, dim=128, group=128, reqs=1, length=4096,
             qpk=4, page=16, dtype="bf16"),
        # a serving batch: 64 ragged requests up to 8192 tokens, 8 query heads per kv head
        case("decode batch", op="attend", layers=1, heads=8, dim=128, group=64, reqs=64, length=8192,
             ragged=True, qpk=8, page=16, dtype="bf16"),
        # one long context, 28 query / 4 kv heads, group 32
        case("decode long", op="attend", layers=1, heads=4, dim=128, group=32, reqs=1, length=131072,
             qpk=7, page=64, dtype="fp16"),
        # verifying 5 drafted tokens per request, sliding window, head_dim 64, an empty request
        case("verify window", op="attend", layers=2, heads=6, dim=64, group=64, reqs=17, length=2500,
             ragged=True, queries=5, window=1000, qpk=4, page=32, dtype="bf16", quant=1, signs=1),
        # a 1024-token chunk of a prompt after 8192 cached tokens
        case("prompt chunk", op="attend", layers=1, heads=8, dim=128, group=128, reqs=1, length=9216,
             queries=1024, qpk=4, page=16, dtype="bf16"),
        # one small layer group arriving
        case("load slice", op="load", layers=2, heads=4, dim=128, group=32, tokens=1001, pages=70,
             page=16, dtype="bf16"),
        # a whole 8B-shaped cache arriving from the prefill side
        case("load cache", op="load", layers=32, heads=8, dim=128, group=128, tokens=4096, pages=300,
             page=16, dtype="bf16"),
    ]


def case(name=None, **more):
    c = {"op": "", "layers": 1, "heads": 1, "dim": 128, "group": 128, "page": 16, "dtype": "bf16",
         "quant": 0, "signs": 0}
    if more["op"] in ("write", "read", "load"):
        c |= {"tokens": 1, "pages": 1}
        if more["op"] == "write":
            c |= {"fused": False, "skip": 0}
    else:
        c |= {"reqs": 1, "length": 1, "ragged": False, "queries": 1, "window": 0, "qpk": 1,
              "causal": True}
    c |= more
    if name:
        c["name"] = name
    return c


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "read", "attend", "attend", "attend", "load"])
    dim = rng.choice([64, 128, 128])
    c = {"op": op, "dim": dim, "group": rng.choice([g for g in (32, 64, 128) if g <= dim]),
         "heads": rng.choice([1, 2, 4, 5, 8, 8]), "page": rng.choice([16, 16, 32, 64, 256]),
         "dtype": rng.choice(["bf16", "fp16"]), "quant": rng.choice([0, 0, 1]),
         "signs": rng.choice([0, 0, 1])}
    if op != "attend":
        c["layers"] = log(1, 32)
        most = min(60000, 1000000 // (c["layers"] * c["heads"]))
        c["tokens"] = log(1, most)
        c["pages"] = (c["tokens"] + c["page"] - 1) // c["page"] + rng.randrange(1, 40)
        if op == "write":
            c["fused"] = rng.random() < 0.5
            c["skip"] = rng.choice([0, 0, 5, 13])
        return case(**c)
    c["layers"] = rng.choice([1, 1, 2, 4])
    c["qpk"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    c["ragged"] = rng.random() < 0.7
    if rng.random() < 0.75:  # decode and verification
        c["reqs"] = log(1, 64)
        c["length"] = log(1, max(2, min(100000, 1600000 // (c["layers"] * c["heads"] * c["reqs"]))))
        c["queries"] = rng.choice([1, 1, 1, 2, 3, 6])
    else:  # pieces of prompts
        c["reqs"] = log(1, 4)
        c["queries"] = log(16, 700)
        c["length"] = min(9000, c["queries"] + log(1, 4000))
        while c["layers"] * c["heads"] * c["qpk"] * c["reqs"] * c["queries"] * c["length"] > 1.2e8:
            c["queries"] = max(2, c["queries"] // 2)
            c["length"] = max(c["queries"], c["length"] // 2 + rng.randrange(3))
    c["window"] = rng.choice([0, 0, 0, log(1, 2000)])
    c["causal"] = True if c["window"] else rng.random() < 0.85
    return case(**c)


def lengths(c):
    """Tokens in the cache per request, the new ones among them."""
    if not c["ragged"]:
        return [c["length"]] * c["reqs"]
    r = random.Random(c["reqs"] * 1000003 + c["length"])
    v = [r.randint(1, c["length"]) for _ in range(c["reqs"])]
    if c["reqs"] > 2:
        v[1] = c["length"]
        v[c["reqs"] // 2] = 0  # a request that has nothing in the cache
    return v


def queries(c, lens):
    """Query tokens per request: at most `queries`, at most its length; none for an empty one."""
    r = random.Random(c["reqs"] * 7919 + c["queries"])
    return [min(n, c["queries"] if not c["ragged"] or i == 1 else r.randint(1, c["queries"]))
            if n else (1 if c["queries"] == 1 else 0) for i, n in enumerate(lens)]


# ------------------------------------------------------------- plain form --
def sign_values(seed, c):
    """The +-1 diagonals as floats [layers, 2, heads, dim]."""
    words = c["dim"] // 64
    count = words * (c["layers"] * 2 * c["heads"] if c["signs"] else 1)
    state, out = seed, []
    for _ in range(count):
        state = (state + 0x9E3779B97F4A7C15) & (2 ** 64 - 1)
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & (2 ** 64 - 1)
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & (2 ** 64 - 1)
        z ^= z >> 31
        out += [-1.0 if z >> i & 1 else 1.0 for i in range(64)]
    s = torch.tensor(out, dtype=torch.float32).reshape(-1, c["dim"])
    if not c["signs"]:
        s = s.expand(c["layers"] * 2 * c["heads"], c["dim"])
    return s.reshape(c["layers"], 2, c["heads"], c["dim"]).cuda()


def butterfly(y):
    """Unnormalised Walsh-Hadamard transform of the last dimension, strides ascending."""
    d = y.shape[-1]
    for h in (1, 2, 4, 8, 16, 32, 64)[: d.bit_length() - 1]:
        p = y.unflatten(-1, (d // (2 * h), 2, h))
        a, b = p[..., 0, :], p[..., 1, :]
        y = torch.stack((a + b, a - b), -2).flatten(-3)
    return y


def half_toward(x, up):
    """fp32 -> fp16, rounded up or down."""
    h = x.half()
    bits = h.view(torch.int16).int()
    o = torch.where(bits < 0, -(bits & 0x7FFF), bits)
    o = o + ((h.float() < x).int() if up else -(h.float() > x).int())
    return torch.where(o < 0, -o - 0x8000, o).short().view(torch.float16)


def quantise(y, c):
    """Transformed vectors [..., dim] -> codes uint8 [..., dim / 2], meta int32 [..., groups]."""
    y = y.unflatten(-1, (-1, c["group"]))
    mn, mx = y.amin(-1, keepdim=True) + 0.0, y.amax(-1, keepdim=True) + 0.0
    if c["quant"]:
        scale = half_toward(torch.maximum(mn.abs(), mx.abs()) / mn.new_tensor(7.0) / K_SCALE, True)
        zero = half_toward(scale.float() * -8.0 + 0.0, False)
    else:
        zero = half_toward(mn / K_SCALE, False)
        scale = half_toward((mx - zero.float() * K_SCALE) / mn.new_tensor(15.0) / K_SCALE, True)
    sf = scale.float() * K_SCALE
    r = torch.where(sf == 0, sf, sf.reciprocal())
    if c["quant"]:
        q = torch.round(y * r).clamp(-7, 7) + 8
    else:
        q = torch.round((y - zero.float() * K_SCALE) * r).clamp(0, 15)
    q = q.flatten(-2).to(torch.uint8).unflatten(-1, (-1, 2))
    meta = (scale.view(torch.int16).int() & 0xFFFF) | (zero.view(torch.int16).int() << 16)
    return q[..., 0] | q[..., 1] << 4, meta.squeeze(-1)


def dequantise(codes, meta, c):
    """Codes [..., dim / 2], meta [..., groups] -> transformed values, fp32."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, c["group"]))
    scale = (meta & 0xFFFF).short().view(torch.float16).float()[..., None] * K_SCALE
    zero = (meta >> 16).short().view(torch.float16).float()[..., None] * K_SCALE
    return (zero + q * scale).flatten(-2)


def tiles(pool, c):
    """Views of the pool: codes [L, P, 2, H, tiles, 16, dim / 2] and meta, int32, [..., 16, groups]."""
    cb, mb = c["dim"] // 2, c["dim"] // c["group"] * 4
    p = pool.unflatten(-1, (c["page"] // 16, 16 * (cb + mb)))
    meta = pool.view(torch.int32).unflatten(-1, (c["page"] // 16, 4 * (cb + mb)))
    return p[..., : 16 * cb].unflatten(-1, (16, cb)), meta[..., 4 * cb:].unflatten(-1, (16, mb // 4))


def places(slots, c):
    inside = slots % c["page"]
    return slots // c["page"], inside // 16, inside % 16


def turned(codes, kv_dim, stored):
    """Codes in channel order to their stored order (stored) or back, keys and values along kv_dim."""
    blocks = codes.shape[-1] // 16  # of 32 channels
    k, v = codes.unbind(kv_dim)
    k = k.unflatten(-1, (blocks, 4, 4) if stored else (4, blocks, 4)).transpose(-3, -2).flatten(-3)
    v = v.unflatten(-1, (blocks, 8, 2) if stored else (8, blocks, 2)).transpose(-3, -2).flatten(-3)
    return torch.stack((k, v), kv_dim)


def store(pool, codes, meta, slots, c):
    """Rows [L, 2, H, N, ...] to N slots."""
    page, tile, lane = places(slots, c)
    cv, mv = tiles(pool, c)
    cv[:, page, :, :, tile, lane] = turned(codes, -4, True).permute(3, 0, 1, 2, 4)
    mv[:, page, :, :, tile, lane] = meta.permute(3, 0, 1, 2, 4)


def fetch(pool, slots, c):
    """The slots' transformed values, fp32 [N, L, 2, H, dim]."""
    page, tile, lane = places(slots, c)
    cv, mv = tiles(pool, c)
    codes = turned(cv[:, page, :, :, tile, lane], -3, False)
    return dequantise(codes, mv[:, page, :, :, tile, lane], c)


def plain_read(s, c):
    keep = s["slots"] >= 0
    x = butterfly(fetch(s["pool"], s["slots"][keep], c)) * (1.0 / c["dim"]) * s["signs"]
    for n, name in enumerate(("k_out", "v_out")):
        s[name][:, keep] = x[:, :, n].transpose(0, 1).to(s[name].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def plain_write(s, c):
    keep = s["slots"] >= 0
    x = torch.stack((s["k"][:, keep], s["v"][:, keep]), 1).float().transpose(2, 3)  # [L, 2, H, N, dim]
    codes, meta = quantise(butterfly(x * s["signs"][:, :, :, None]), c)
    store(s["pool"], codes, meta, s["slots"][keep], c)
    return plain_read(s, c)


def plain_load(s, c):
    layers, heads, n = c["layers"], c["heads"], c["tokens"]
    vectors = layers * 2 * heads * n
    cb, groups = c["dim"] // 2, c["dim"] // c["group"]
    base = s["data_base"]
    codes = s["stream"][base: base + vectors * cb].view(layers, 2, heads, n, cb)
    at = base + -(-vectors * cb // 16) * 16
    meta = s["stream"][at: at + vectors * groups * 4].view(torch.int32).view(layers, 2, heads, n, groups)
    store(s["pool"], codes, meta, s["slots"], c)
    return plain_read(s, c)


def plain_attend(s, c):
    reach = s["page_table"].shape[1] * c["page"]
    lens, starts = s["seq_lens"].long(), s["q_starts"].long()
    t = torch.arange(reach, device="cuda")
    there = t < lens[:, None]  # [R, T]
    slots = s["page_table"].long().clamp(min=0)[:, t // c["page"]] * c["page"] + t % c["page"]
    x = butterfly(fetch(s["pool"], torch.where(there, slots, 0), c)) * (1.0 / c["dim"]) * s["signs"]
    x = torch.where(there[..., None, None, None, None], x, 0.0)  # [R, T, L, 2, H, dim]
    k, v = x[:, :, :, 0].permute(2, 0, 3, 4, 1), x[:, :, :, 1].permute(2, 0, 3, 1, 4)
    i = torch.arange(c["queries"], device="cuda")
    count = starts[1:] - starts[:-1]
    asked = i < count[:, None]  # [R, Q]
    rows = torch.where(asked, starts[:-1, None] + i, 0)
    at = (lens - count)[:, None] + i if c["causal"] else (lens - 1)[:, None].expand(-1, c["queries"])
    seen = there[:, None] & (t <= at[..., None])  # [R, Q, T]
    if c["window"]:
        seen = seen & (t > at[..., None] - c["window"])
    q = s["q"].float()[:, rows].unflatten(3, (c["heads"], c["qpk"]))  # [L, R, Q, H, g, dim]
    q = q.permute(0, 1, 3, 2, 4, 5).flatten(3, 4)
    score = torch.matmul(q, k).unflatten(3, (c["queries"], c["qpk"])) * s["scale"]
    score = torch.where(seen[:, None, :, None], score, -math.inf)  # [L, R, H, Q, g, T]
    most = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(most == -math.inf, 0.0, most))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(3, 4), v).unflatten(3, (c["queries"], c["qpk"]))
    o = torch.where(total > 0, o / total, 0.0)
    lse = (most + total.log()).squeeze(-1)
    pick = asked.flatten().nonzero().squeeze(1)
    o = o.permute(1, 3, 0, 2, 4, 5).flatten(0, 1)[pick]  # [T, L, H, g, dim]
    lse = lse.permute(1, 3, 0, 2, 4).flatten(0, 1)[pick]
    s["out"].copy_(o.transpose(0, 1).flatten(2, 3))
    s["lse"].copy_(lse.transpose(0, 1).flatten(2, 3))
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ state --
def values(c, n, gen):
    """Keys [L, n, H, dim] with strong per-channel scales, values near Gaussian: fp32."""
    shape = (c["layers"], n, c["heads"], c["dim"])
    k = torch.randn(shape, device="cuda", generator=gen)
    scale = torch.randn((c["layers"], 1, c["heads"], c["dim"]), device="cuda", generator=gen)
    k *= torch.exp(0.5 * scale)
    return k, torch.randn(shape, device="cuda", generator=gen)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    sign_seed = random.Random(int(seed)).getrandbits(63)
    dtype = DTYPES[c["dtype"]]
    s = {"case": c, "sign_seed": sign_seed, "signs": sign_values(sign_seed, c)}
    block = c["page"] * (c["dim"] // 2 + c["dim"] // c["group"] * 4)
    if c["op"] == "attend":
        lens = lengths(c)
        n, need = sum(lens), [-(-x // c["page"]) for x in lens]
        pages = sum(need) + 3
    else:
        n, pages = c["tokens"], c["pages"]
    # slots that nothing has written hold anything, NaN patterns among it
    s["pool"] = torch.randint(0, 256, (c["layers"], pages, 2, c["heads"], block), device="cuda",
                              generator=gen, dtype=torch.uint8)
    s["num_pages"] = pages
    order = torch.randperm(pages, device="cuda", generator=gen)
    if c["op"] == "attend":
        table = torch.full((c["reqs"], max(max(need), 1)), -1, dtype=torch.int32)
        at, slots = 0, [torch.empty(0, dtype=torch.long, device="cuda")]
        for r, x in enumerate(need):
            table[r, :x] = order[at: at + x].int().cpu()
            t = torch.arange(lens[r], device="cuda")
            slots.append(order[at + t // c["page"]] * c["page"] + t % c["page"])
            at += x
        slots = torch.cat(slots)
        asked = queries(c, lens)
        starts = [sum(asked[:r]) for r in range(c["reqs"] + 1)]
        s["page_table"], s["seq_lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        s["q_starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
        s["scale"] = c["dim"] ** -0.5
        shape = (c["layers"], starts[-1], c["heads"] * c["qpk"], c["dim"])
        s["q"] = torch.randn(shape, device="cuda", generator=gen).to(dtype)
        s["out"] = torch.zeros(shape, dtype=dtype, device="cuda")
        s["lse"] = torch.zeros(shape[:3], dtype=torch.float32, device="cuda")
    else:
        t = torch.arange(n, device="cuda")
        slots = order[t // c["page"]] * c["page"] + t % c["page"]
        if c["op"] == "read" and n > 1:  # some of the rows, in another order, a few left out
            slots = slots[torch.randperm(n, device="cuda", generator=gen)] if n < 5000 else slots
        shape = (c["layers"], n, c["heads"], c["dim"])
        s["k_out"] = torch.zeros(shape, dtype=dtype, device="cuda")
        s["v_out"] = torch.zeros(shape, dtype=dtype, device="cuda")
    k, v = values(c, n, gen)
    if c["op"] == "write":
        if c["fused"]:  # keys and values as slices of a fused projection's output
            both = torch.cat((k, v, k), 2).to(dtype)
            s["k"], s["v"] = both[:, :, : c["heads"]], both[:, :, c["heads"]: 2 * c["heads"]]
        else:
            s["k"], s["v"] = k.to(dtype), v.to(dtype)
        if c["skip"]:  # padding tokens
            slots[:: c["skip"]] = -1
        s["slots"] = slots
        return s
    x = torch.stack((k, v), 1).to(torch.bfloat16).float().transpose(2, 3)  # [L, 2, H, N, dim]
    del k, v
    codes, meta = quantise(butterfly(x * s["signs"][:, :, :, None]), c)
    if c["op"] == "load":
        s |= stream_of(codes, meta, sign_seed, c)
    else:
        store(s["pool"], codes, meta, slots, c)
    if c["op"] != "attend":
        s["slots"] = slots
    return s


def stream_of(codes, meta, sign_seed, c):
    """The codes and meta as a compressed stream whose chunks are stored raw."""
    regions = [codes.contiguous().view(-1), meta.contiguous().view(torch.uint8).view(-1)]
    entries, at = [], 0
    for r in regions:
        for x in range(0, r.numel(), 16384):
            size = min(16384, r.numel() - x)
            entries.append(size | at // 16 << 16)
            at += -(-size // 16) * 16
    base = -(-(64 + 8 * len(entries) + 4) // 16) * 16
    head = bytearray(base)
    fields = [(0, 4, 0x3143564B), (4, 2, 1), (6, 2, 64), (8, 1, 4), (9, 1, 3),
              (11, 1, c["quant"] << 1 | c["signs"] << 3), (12, 4, c["group"]), (16, 4, c["layers"]),
              (20, 4, 2), (24, 4, c["heads"]), (28, 4, c["dim"]), (32, 8, c["tokens"]),
              (40, 8, sign_seed), (48, 4, 1), (52, 4, len(entries)), (56, 8, base + at)]
    for where, size, value in fields + [(64 + 8 * i, 8, e) for i, e in enumerate(entries)]:
        head[where: where + size] = value.to_bytes(size, "little")
    head[64 + 8 * len(entries): 68 + 8 * len(entries)] = c["tokens"].to_bytes(4, "little")
    out = torch.zeros(base + at, dtype=torch.uint8, device="cuda")
    out[:base] = torch.frombuffer(head, dtype=torch.uint8).cuda()
    out[base: base + regions[0].numel()] = regions[0]
    at = base + -(-regions[0].numel() // 16) * 16
    out[at: at + regions[1].numel()] = regions[1]
    return {"stream": out, "nbytes": out.numel(), "data_base": base}


# -------------------------------------------------------------------- run --
def handle(s):
    """The cache object that a serving program keeps for its pool."""
    import kv_cache_compression_04_b200 as kvc
    if "cache" not in s:
        c = s["case"]
        s["cache"] = kvc.PagedCache(c["layers"], c["heads"], c["dim"], s["num_pages"],
                                    page_tokens=c["page"], group=c["group"],
                                    sign_seed=s["sign_seed"], quant=c["quant"], signs=c["signs"],
                                    pool=s["pool"])
    return s["cache"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"write": plain_write, "read": plain_read, "load": plain_load,
                "attend": plain_attend}[c["op"]](s, c)
    cache = handle(s)
    if c["op"] == "attend":
        cache.attend(s["q"], s["page_table"], s["seq_lens"], q_starts=s["q_starts"],
                     max_q=c["queries"], out=s["out"], lse=s["lse"], scale=s["scale"],
                     causal=c["causal"], window=c["window"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "write":
        cache.write(s["k"], s["v"], s["slots"])
    elif c["op"] == "load":
        cache.load(s["stream"], s["nbytes"], s["slots"], [c["tokens"]])
    cache.read(s["slots"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    row = c["dim"] // 2 + c["dim"] // c["group"] * 4  # a stored vector
    if c["op"] != "attend":
        n = c["tokens"]
        if c["op"] == "write" and c["skip"]:
            n -= -(-n // c["skip"])
        vectors = c["layers"] * 2 * c["heads"] * n
        # write: bf16 in, stored out, and read back; load: the stream's share in its place
        moved = {"write": 2 * c["dim"] + 2 * row, "read": row, "load": 3 * row}[c["op"]]
        stages = c["dim"].bit_length() - 1
        adds = (2 if c["op"] == "write" else 1) * (stages + 2) * c["dim"]
        return {"bytes": vectors * (moved + 2 * c["dim"]), "flops": vectors * adds}
    lens = lengths(c)
    pairs = read = asked = 0
    for n, m in zip(lens, queries(c, lens)):
        asked += m
        first = n  # the first key that some query sees
        for i in range(m):
            end = n - m + i + 1 if c["causal"] else n
            lo = max(0, end - c["window"]) if c["window"] else 0
            pairs += end - lo
            first = min(first, lo)
        read += n - first if m else 0
    heads = c["layers"] * c["heads"]
    out = asked * heads * c["qpk"]
    return {"bytes": heads * read * 2 * row + out * (4 * c["dim"] + 4),
            "flops": 4 * c["dim"] * heads * c["qpk"] * pairs}


# ------------------------------------------------------------------ exact --
def hadamard(d):
    """Sylvester's matrix in 64 bits."""
    i = torch.arange(d, device="cuda")
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> k) & 1 for k in range(7)) % 2
    return 1.0 - 2.0 * odd.double()


def exact_rows(pool, slots, c, signs, h):
    """The rows of `slots` in 64 bits [N, L, 2, H, dim], from the pool's bytes."""
    cb, groups = c["dim"] // 2, c["dim"] // c["group"]
    tile = 16 * (cb + 4 * groups)
    page, rest = slots // c["page"], slots % c["page"]
    got = pool[:, page].transpose(0, 1)  # [N, L, 2, H, block]
    got = got.reshape(slots.numel(), -1, c["page"] // 16, tile)
    n = torch.arange(slots.numel(), device=slots.device)
    got = got[n, :, rest // 16]  # [N, L*2*H, tile]
    lane = (rest % 16)[:, None, None]
    i = torch.arange(cb, device=slots.device)  # byte i of a row in channel order is stored at:
    at_k = (i // 4 % 4) * (cb // 4) + i // 16 * 4 + i % 4
    at_v = (i // 2 % 8) * (cb // 8) + i // 16 * 2 + i % 2
    at = torch.stack((at_k, at_v)).repeat_interleave(c["heads"], 0).repeat(c["layers"], 1)
    byte = got.gather(2, lane * cb + at)
    where = 16 * cb + lane * 4 * groups + torch.arange(4 * groups, device=slots.device)
    half = got.gather(2, where.expand(-1, got.shape[1], -1)).contiguous().view(torch.float16).double()
    q = torch.empty(*byte.shape[:2], c["dim"], dtype=torch.float64, device=slots.device)
    q[..., 0::2], q[..., 1::2] = (byte % 16).double(), (byte // 16).double()
    scale = half[..., 0::2].repeat_interleave(c["group"], -1)
    zero = half[..., 1::2].repeat_interleave(c["group"], -1)
    y = (q * scale + zero) * 8.0
    return (y @ h / c["dim"]).view(-1, c["layers"], 2, c["heads"], c["dim"]) * signs.double()


def exact_half(x, up):
    """64-bit values to the fp16 grid, toward +inf or -inf."""
    step = torch.pow(2.0, torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14))).clamp(min=-14) - 10)
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def exact_stored(x, c, signs, h):
    """What the cache stands for after writing x [..., H, dim] (64 bits)."""
    y = ((x * signs) @ h).unflatten(-1, (-1, c["group"]))
    if c["quant"]:
        s = exact_half(y.abs().amax(-1, keepdim=True) / 7.0 / 8.0, True) * 8.0
        got = torch.round(y / torch.where(s == 0, 1.0, s)) * s
    else:
        z = exact_half(y.amin(-1, keepdim=True) / 8.0, False) * 8.0
        s = exact_half((y.amax(-1, keepdim=True) - z) / 15.0 / 8.0, True) * 8.0
        got = torch.round((y - z) / torch.where(s == 0, 1.0, s)) * s + z
    return got.flatten(-2) @ h / c["dim"] * signs


def exact(case, seed):
    c, s = case, prepare(case, seed)
    h = hadamard(c["dim"])
    signs = s["signs"].double()
    if c["op"] == "attend":
        return exact_attend(s, c, signs, h)
    outs = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    if c["op"] == "load":
        size = c["layers"] * 2 * c["heads"] * c["tokens"]
        cb, groups = c["dim"] // 2, c["dim"] // c["group"]
        at = s["data_base"] + (size * cb + 15) // 16 * 16
        byte = s["stream"][s["data_base"]: s["data_base"] + size * cb].view(c["layers"], 2, c["heads"], -1, cb)
        half = s["stream"][at: at + size * groups * 4].view(torch.float16)
        half = half.view(c["layers"], 2, c["heads"], -1, groups, 2).double()
        for layer in range(c["layers"]):
            for n in range(2):
                b = byte[layer, n]
                q = torch.stack((b % 16, b // 16), -1).flatten(-2).double().unflatten(-1, (groups, -1))
                y = (q * half[layer, n, ..., :1] + half[layer, n, ..., 1:]).flatten(-2) * 8.0
                x = y @ h / c["dim"] * signs[layer, n][:, None]
                outs[n][layer] = x.transpose(0, 1)
        return {"k": outs[0], "v": outs[1]}
    keep = s["slots"] >= 0
    if c["op"] == "write":
        for layer in range(c["layers"]):
            for n, name in enumerate(("k", "v")):
                outs[n][layer, keep] = exact_stored(s[name][layer, keep].double(), c, signs[layer, n], h)
        return {"k": outs[0], "v": outs[1]}
    at = keep.nonzero().squeeze(1)
    for piece in at.split(4096):
        x = exact_rows(s["pool"], s["slots"][piece], c, signs, h)
        for n in range(2):
            outs[n][:, piece] = x[:, :, n].transpose(0, 1)
    return {"k": outs[0], "v": outs[1]}


def exact_attend(s, c, signs, h):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    lens, starts = s["seq_lens"].tolist(), s["q_starts"].tolist()
    q = s["q"].double().unflatten(2, (c["heads"], c["qpk"]))
    for r, n in enumerate(lens):
        m = starts[r + 1] - starts[r]
        if not n or not m:
            continue
        t = torch.arange(n, device="cuda")
        slots = s["page_table"][r].long()[t // c["page"]] * c["page"] + t % c["page"]
        x = torch.cat([exact_rows(s["pool"], p, c, signs, h) for p in slots.split(4096)])
        i = torch.arange(m, device="cuda")[:, None]
        hide = t > n - m + i if c["causal"] else (t < 0).expand(m, -1)
        if c["window"]:
            hide = hide | (t <= n - m + i - c["window"])
        for layer in range(c["layers"]):
            for head in range(c["heads"]):
                rows = q[layer, starts[r]: starts[r + 1], head]  # [m, g, dim]
                sc = (rows @ x[:, layer, 0, head].T) * s["scale"]
                sc = sc.masked_fill(hide[:, None], -math.inf)
                z = torch.logsumexp(sc, -1, keepdim=True)
                p = torch.exp(sc - torch.where(z == -math.inf, 0.0, z))
                at = slice(head * c["qpk"], (head + 1) * c["qpk"])
                out[layer, starts[r]: starts[r + 1], at] = p @ x[:, layer, 1, head]
                lse[layer, starts[r]: starts[r + 1], at] = z.squeeze(-1)
    return {"out": out, "lse": lse}
