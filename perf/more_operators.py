"""The operators of a decode step over an 8-bit paged cache as they are measured: cases, inputs, and each operator in plain torch.

Four operators stand between a layer's projection and its output for one new token a request:

  rope    norms of the query and key heads and their rotation by position     (lmoe_qk_norm_rope)
  write   K/V rows -> E4M3 codes and a power-of-two scale in their slots       (lmoe_kv_write_fp8)
  read    rows of requests out of the cache again, as bf16                     (lmoe_kv_read_fp8)
  decode  attention of one new token a request over the cache                  (lmoe_decode_attention_fp8)

The cache is [block][kv head][slot][head width] in E4M3 with an E8M0 scale byte for each [block][kv head][slot]: the
element is code * 2^(byte - 127).  A row's scale is the smallest power of two that brings its largest magnitude to 448
or less.  A request's position p is in block block_table[request][p // block_size], slot p % block_size.

A case fixes the shapes (lengths come from its own "shape" number); the values, the positions and the block order come
from the seed.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # the queries and keys of one user's next token: latency of the smallest call
        dict(name="rope_one_token", op="rope", tokens=1, q_heads=64, kv_heads=8, width=128, rotated=128, axes=1,
             interleaved=False, norm=True, far=131072),
        # a prompt of 16384 tokens in one call
        dict(name="rope_prompt", op="rope", tokens=16384, q_heads=64, kv_heads=8, width=128, rotated=128, axes=1,
             interleaved=False, norm=True, far=16384),
        # a video's patches with positions in time, height and width, a part of each head rotated, neighbours as pairs
        dict(name="rope_video", op="rope", tokens=5003, q_heads=16, kv_heads=16, width=80, rotated=64, axes=3,
             interleaved=True, norm=True, far=2000),
        # the next token of 64 requests enters the cache
        dict(name="write_step", op="write", tokens=64, rows=64, kv_heads=8, width=128, block=16, blocks=2048,
             gather=False),
        # a prompt of 16384 tokens enters the cache
        dict(name="write_prompt", op="write", tokens=16384, rows=16384, kv_heads=8, width=128, block=64, blocks=512,
             gather=False),
        # one request's prefix back as rows, for a call that takes bf16
        dict(name="read_one_request", op="read", shape=1, requests=1, len_lo=1021, len_hi=1021, kv_heads=8, width=128,
             block=16),
        # the prefixes of 16 long requests
        dict(name="read_batch", op="read", shape=2, requests=16, len_lo=500, len_hi=8191, kv_heads=8, width=128,
             block=32),
        # one user's next token early in a chat
        dict(name="decode_one_user", op="decode", shape=3, requests=1, len_lo=1021, len_hi=1021, q_heads=64,
             kv_heads=8, width=128, block=16, window=0),
        # the next token of a batch of 64 requests of mixed length
        dict(name="decode_batch", op="decode", shape=4, requests=64, len_lo=512, len_hi=8191, q_heads=64, kv_heads=8,
             width=128, block=64, window=0),
        # a large server: 256 requests from a few tokens to thousands, five query heads to a key head
        dict(name="decode_large_server", op="decode", shape=5, requests=256, len_lo=20, len_hi=8191, q_heads=40,
             kv_heads=8, width=128, block=32, window=0),
        # one request far into a long document: the prefix has to be split over the whole card
        dict(name="decode_long_document", op="decode", shape=6, requests=1, len_lo=131071, len_hi=131071, q_heads=64,
             kv_heads=8, width=128, block=64, window=0),
        # a sliding-window layer of 48 long requests, heads of 64
        dict(name="decode_window_layer", op="decode", shape=7, requests=48, len_lo=300, len_hi=32768, q_heads=24,
             kv_heads=8, width=64, block=16, window=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "read", "decode", "decode", "decode"])
    shape = rng.randrange(1 << 30)
    if op == "rope":
        q_heads, kv_heads, width = rng.choice([(64, 8, 128), (40, 8, 128), (32, 4, 128), (24, 8, 64), (16, 16, 80),
                                               (8, 1, 256), (12, 2, 96)])
        return dict(op=op, tokens=_log(rng, 1, 16384 * 72 * 128 // ((q_heads + kv_heads) * max(width, 128))),
                    q_heads=q_heads, kv_heads=kv_heads, width=width,
                    rotated=rng.choice([width, width, width // 32 * 16]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8, far=_log(rng, 100, 1000000))
    if op == "write":
        gather = rng.random() < 0.5
        tokens = _log(rng, 1, 16384)
        block = rng.choice([16, 32, 64, 128])
        return dict(op=op, tokens=tokens, rows=tokens + (rng.randint(0, tokens) if gather else 0),
                    kv_heads=rng.choice([1, 3, 8]), width=rng.choice([64, 128]), block=block,
                    blocks=tokens // block + rng.randint(1, 64), gather=gather)
    kv_heads, width = rng.choice([(8, 128), (4, 128), (16, 64), (1, 128), (8, 64)])
    # no more than the listed cases read from the cache
    room = (30000 if op == "read" else 100000) * 1024 // (kv_heads * width)
    len_hi = min(_log(rng, 4, 16384 if op == "read" else 131072), room)
    case = dict(op=op, shape=shape, requests=_log(rng, 1, max(1, min(256, room // len_hi))),
                len_lo=rng.randint(0, len_hi), len_hi=len_hi, kv_heads=kv_heads, width=width,
                block=rng.choice([16, 32, 64, 128]))
    if op == "decode":
        case |= dict(q_heads=kv_heads * rng.choice([1, 3, 4, 5, 8, 8, 16]), window=rng.choice([0, 0, 0, 1024, 333]))
    return case


def _lengths(case):
    """Tokens that each request holds."""
    r = random.Random(case["shape"])
    lo, hi = case["len_lo"], case["len_hi"]
    lens = [int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1 for _ in range(case["requests"])]
    lens[0] = hi
    return lens


# ---------------------------------------------------------------------------------------------
# what the operators cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    d, hk = case["width"], case["kv_heads"]
    if case["op"] == "rope":
        t, heads = case["tokens"], case["q_heads"] + hk
        return {"bytes": 2 * 2 * t * heads * d + 4 * t * case["axes"] + 2 * case["rotated"] + 4 * d * case["norm"],
                "flops": t * heads * (3 * d * case["norm"] + 3 * case["rotated"])}
    if case["op"] == "write":
        return {"bytes": case["tokens"] * (2 * hk * (2 * d + d + 1) + (8 if case["gather"] else 4)), "flops": 0}
    lens = _lengths(case)
    if case["op"] == "read":
        return {"bytes": sum(lens) * 2 * hk * (d + 1 + 2 * d) + 4 * sum(-(-x // case["block"]) for x in lens), "flops": 0}
    hq, w = case["q_heads"], case["window"]
    seen = [min(x, w) if w else x for x in lens]
    return {"bytes": sum(seen) * 2 * hk * (d + 1) + len(lens) * (2 * 2 * hq * d + 4 * hq + 4)
            + 4 * sum(-(-x // case["block"]) for x in seen), "flops": 4 * d * hq * sum(seen)}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _two_to(e):
    """2^e in fp32 for whole numbers -126 <= e <= 127; 0 for -127, the scale of rows of zeros alone here."""
    return (e + 127 << 23).view(torch.float32)


def _quantise(x):
    """E4M3 codes (as bytes) and E8M0 bytes of rows [..., width]: the smallest 2^e with max |x| <= 448 * 2^e."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(dim=-1))  # m * 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -127).clamp(-127, 127)
    codes = (x * _two_to(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scale):
    """fp32 values of E4M3 codes [..., width] and E8M0 bytes [...]."""
    return codes.view(torch.float8_e4m3fn).float() * _two_to(scale.int() - 127)[..., None]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    s = {"case": case}
    hk, d = case["kv_heads"], case["width"]

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] == "rope":
        t, hq, half = case["tokens"], case["q_heads"], case["rotated"] // 2
        # the rows of a fused projection: queries, keys and values of a token side by side
        qkv = normal(t, (hq + 2 * hk) * d).bfloat16()
        q, k, _ = qkv.split([hq * d, hk * d, hk * d], dim=1)
        gain = (1 + 0.2 * normal(2, d)).bfloat16() if case["norm"] else (None, None)
        # the frequencies' axes in turn, as equal shares of every axis have them
        axis = dev((np.arange(half) % case["axes"]).astype(np.int32)) if case["axes"] > 1 else None
        s |= {"q": q.unflatten(1, (hq, d)), "k": k.unflatten(1, (hk, d)), "q_gain": gain[0], "k_gain": gain[1],
              "pos": dev(rs.randint(0, case["far"], (case["axes"], t)).astype(np.int32)), "axis": axis,
              "freq": dev((500000.0 ** (-np.arange(half) / half)).astype(np.float32)), "eps": 1e-6}
        return s
    if case["op"] == "write":
        bs, t = case["block"], case["tokens"]
        kv = (normal(case["rows"], 2 * hk * d) * torch.exp2(2 * normal(case["rows"], 1))).bfloat16()
        kn, vn = kv.split([hk * d, hk * d], dim=1)
        slots = rs.permutation(case["blocks"] * bs)[:t].astype(np.int32) if case["gather"] else \
            (rs.permutation(case["blocks"])[:, None] * bs + np.arange(bs)).reshape(-1)[:t].astype(np.int32)
        if t > 8:
            slots[rs.randint(t)] = -1  # a token whose request had no room
        src = dev(np.sort(rs.permutation(case["rows"])[:t]).astype(np.int32)) if case["gather"] else None
        s |= {"k_new": kn.unflatten(1, (hk, d)), "v_new": vn.unflatten(1, (hk, d)), "slots": dev(slots), "src": src}
        blocks = case["blocks"]
    else:
        lens, bs = _lengths(case), case["block"]
        held = [-(-x // bs) for x in lens]
        blocks, wide = sum(held) + 3, max(1, max(held))
        order, at = rs.permutation(blocks).astype(np.int32), 0
        table = np.zeros((len(lens), wide), np.int32)
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        s |= {"block_table": dev(table), "lens": dev(np.array(lens, np.int32)), "len_max": max(lens),
              "token_offsets": dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)), "tokens": sum(lens)}
        if case["op"] == "decode":
            hq = case["q_heads"]
            qkv = normal(len(lens), (hq + 2 * hk) * d).bfloat16()
            s |= {"q": qkv[:, :hq * d].unflatten(1, (hq, d)), "scale": d ** -0.5}
    # keys with channels of unequal size, as projections have them; tokens of unequal size
    size = torch.empty(hk, 1, d, device="cuda").uniform_(0.5, 1.5, generator=g)
    s["k"], s["k_scale"] = _quantise(normal(blocks, hk, bs, d) * size)
    s["v"], s["v_scale"] = _quantise(normal(blocks, hk, bs, d) * torch.exp2(0.5 * normal(blocks, hk, bs, 1)))
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _plain_rope(s):
    case = s["case"]
    n = case["rotated"]
    pos = s["pos"][s["axis"].long()].T if s["axis"] is not None else s["pos"].T  # [tokens, half or 1]
    angle = pos.double() * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, gain):
        x = x.float()
        if case["norm"]:
            x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + s["eps"]) * gain.float()
        a, b = (x[..., 0:n:2], x[..., 1:n:2]) if case["interleaved"] else (x[..., :n // 2], x[..., n // 2:n])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([a, b], dim=-1).flatten(-2) if case["interleaved"] else torch.cat([a, b], dim=-1)
        return torch.cat([r, x[..., n:]], dim=-1).bfloat16()

    return {"q": turned(s["q"], s["q_gain"]), "k": turned(s["k"], s["k_gain"])}


def _own_rope(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:  # what a serving loop holds from step to step
        case = s["case"]
        s["kept"] = (lm.rope_dims_of(case["tokens"], case["q_heads"], case["kv_heads"], case["width"],
                                     case["rotated"], n_axes=case["axes"], interleaved=case["interleaved"],
                                     norm=case["norm"], eps=s["eps"]),
                     torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda"))
    dims, q, k = s["kept"]
    lm.lmoe_qk_norm_rope(dims, s["q"], s["k"], s["q_gain"], s["k_gain"], s["pos"], s["freq"], s["axis"], q, k)
    return {"q": q, "k": k}


def _cache(s):
    """The cache as an output: codes as the E4M3 values that they are, scales as E8M0 bytes."""
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _plain_write(s):
    bs = s["case"]["block"]
    keep = (s["slots"] >= 0).nonzero(as_tuple=True)[0]
    slot = s["slots"].long()[keep]
    src = s["src"].long()[keep] if s["src"] is not None else keep
    for at, rows in (("k", s["k_new"]), ("v", s["v_new"])):
        codes, scale = _quantise(rows[src])
        s[at][slot // bs, :, slot % bs] = codes
        s[at + "_scale"][slot // bs, :, slot % bs] = scale
    return _cache(s)


def _own_write(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:
        s["kept"] = lm.kv_cache_fp8_of(s["k"], s["v"], s["k_scale"], s["v_scale"])
    lm.lmoe_kv_write_fp8(s["kept"], s["k_new"], s["v_new"], s["src"], s["slots"])
    return _cache(s)


def _plain_read(s):
    bs, off = s["case"]["block"], s["token_offsets"].long()
    t = torch.arange(s["tokens"], device=off.device)
    b = torch.searchsorted(off, t, right=True) - 1
    p = t - off[b]
    block = s["block_table"].long()[b, p // bs]
    return {at: _values(s[at][block, :, p % bs], s[at + "_scale"][block, :, p % bs]).bfloat16() for at in ("k", "v")}


def _own_read(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:
        shape = (s["tokens"], s["case"]["kv_heads"], s["case"]["width"])
        s["kept"] = (lm.kv_cache_fp8_of(s["k"], s["v"], s["k_scale"], s["v_scale"]),
                     torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    cache, k, v = s["kept"]
    lm.lmoe_kv_read_fp8(cache, s["token_offsets"], None, s["block_table"], k, v)
    return {"k": k, "v": v}


def _plain_decode(s):
    case = s["case"]
    hq, hk, d, bs, w = case["q_heads"], case["kv_heads"], case["width"], case["block"], case["window"]
    lens = s["lens"].long()
    # the positions that a window leaves, padded to the longest
    span = min(s["len_max"], w) if w else s["len_max"]
    p = (lens - span).clamp(min=0)[:, None] + torch.arange(span, device=lens.device)
    held = p < lens[:, None]
    p = torch.where(held, p, 0)
    block = torch.gather(s["block_table"].long(), 1, p // bs)

    def rows(at):
        x = _values(s[at][block, :, p % bs], s[at + "_scale"][block, :, p % bs])
        return x.masked_fill(~held[:, :, None, None], 0.0).transpose(1, 2)

    q = s["q"].float().unflatten(1, (hk, hq // hk))
    x = (torch.matmul(q, rows("k").transpose(2, 3)) * s["scale"]).masked_fill(~held[:, None, None], -math.inf)
    top = x.amax(dim=3, keepdim=True) if span else x.new_full((*x.shape[:3], 1), -math.inf)
    top = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(dim=3, keepdim=True)
    o = torch.matmul(e, rows("v")) / torch.where(total > 0, total, 1.0)
    return {"out": o.flatten(1, 2).bfloat16(), "lse": (torch.log(total) + top)[..., 0].flatten(1, 2)}


def _own_decode(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:
        case, q = s["case"], s["q"]
        cache = lm.kv_cache_fp8_of(s["k"], s["v"], s["k_scale"], s["v_scale"])
        dims = lm.decode_dims_of(case["requests"], case["q_heads"], s["block_table"].shape[1], s["scale"],
                                 window=case["window"])
        s["kept"] = (dims, cache, torch.empty(q.shape, dtype=q.dtype, device=q.device),
                     torch.empty(q.shape[:2], dtype=torch.float32, device=q.device),
                     torch.empty(lm.lmoe_decode_attention_fp8_workspace_bytes(dims, cache), dtype=torch.uint8,
                                 device=q.device))
    dims, cache, out, lse, ws = s["kept"]
    lm.lmoe_decode_attention_fp8(dims, cache, s["q"], s["lens"], s["block_table"], out, lse, ws)
    return {"out": out, "lse": lse}


_PLAIN = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "decode": _plain_decode}
_OWN = {"rope": _own_rope, "write": _own_write, "read": _own_read, "decode": _own_decode}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _e4m3_table():
    """The value of each byte as E4M3: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    out = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = math.nan if c & 127 == 127 else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out.append(-x if c & 128 else x)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _exact_codes(x):
    """Values of the E4M3 codes of rows in 64 bits, and the E8M0 bytes."""
    top = x.abs().amax(dim=-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448.0))
    for _ in range(2):  # the logarithm's own rounding
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e))
    e = torch.where(top > 0, e.clamp(-127, 127), -127.0)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.round(y / step) * step, (e[..., 0] + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        half, out = case["rotated"] // 2, {}
        for name in ("q", "k"):
            x = s[name].double()
            if case["norm"]:
                x = x / torch.sqrt((x * x).sum(dim=2, keepdim=True) / case["width"] + s["eps"]) * s[name + "_gain"].double()
            y = x.clone()
            for i in range(half):
                p = s["pos"][i % case["axes"]].double() * s["freq"][i].double()
                c, z = torch.cos(p)[:, None], torch.sin(p)[:, None]
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                y[:, :, a] = x[:, :, a] * c - x[:, :, b] * z
                y[:, :, b] = x[:, :, a] * z + x[:, :, b] * c
            out[name] = y
        return out
    bs = case["block"]
    if case["op"] == "write":
        # whole numbers (the scales) have no computed value here
        value = _e4m3_table()
        out = {"k": value[s["k"].int()], "v": value[s["v"].int()], "k_scale": None, "v_scale": None}
        slots = s["slots"].tolist()
        src = s["src"].tolist() if case["gather"] else list(range(len(slots)))
        to = torch.tensor([(a // bs, a % bs, b) for a, b in zip(slots, src) if a >= 0], device="cuda").T
        for name in ("k", "v"):
            out[name].transpose(1, 2)[to[0], to[1]] = _exact_codes(s[name + "_new"].double()[to[2]])[0]
        return out
    value, lens = _e4m3_table(), _lengths(case)
    flat = {n: s[n].transpose(1, 2).reshape(-1, case["kv_heads"], case["width"]) for n in ("k", "v")}
    size = {n: s[n + "_scale"].transpose(1, 2).reshape(-1, case["kv_heads"]) for n in ("k", "v")}

    def rows(n, b, lo, hi):
        t = torch.arange(lo, hi, device="cuda")
        at = s["block_table"][b].long()[t // bs] * bs + t % bs
        return value[flat[n][at].int()] * torch.exp2(size[n][at].double() - 127)[..., None]

    if case["op"] == "read":
        return {n: torch.cat([rows(n, b, 0, x) for b, x in enumerate(lens)]) for n in ("k", "v")}
    hq, hk, w = case["q_heads"], case["kv_heads"], case["window"]
    out = torch.zeros(len(lens), hq, case["width"], dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        lo = max(0, n - w) if w else 0
        k, v = rows("k", b, lo, n), rows("v", b, lo, n)
        for h in range(hk):
            of = slice(h * (hq // hk), (h + 1) * (hq // hk))
            x = s["q"][b, of].double() @ k[:, h].T * s["scale"]
            lse[b, of] = torch.logsumexp(x, dim=1)
            out[b, of] = torch.exp(x - lse[b, of, None]) @ v[:, h]
    return {"out": out, "lse": lse}
