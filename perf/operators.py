"""The speculative-decoding operators as they are measured: cases, inputs, and each operator in plain torch.

Four operators make one verification step of a serving loop over a paged key/value cache:

  masks   parents of drafted tokens -> ancestor bit masks and positions      (lmoe_tree_masks)
  attend  attention of the drafted tokens over the cached prefix and the     (lmoe_tree_attention)
          tree of drafts
  plan    request lengths -> block tables, slot maps, free blocks            (lmoe_kv_plan)
  write   accepted (or prompt) K/V rows -> their slots in the cache          (lmoe_kv_write)

The cache is [block][kv head][slot][head width]; a request's position p is in
block block_table[request][p // block_size], slot p % block_size.  Requests are
ragged: token_offsets[b] .. token_offsets[b + 1] are request b's rows.

A case fixes the shapes (lengths come from its own "shape" number); the values,
the block order and the trees come from the seed.
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
        # one user, eight drafted tokens, a chat's first turns: latency of the smallest call
        dict(name="attend_one_user", op="attend", shape=1, requests=1, n_lo=8, n_hi=8, len_lo=1021, len_hi=1021,
             q_heads=64, kv_heads=8, width=128, block=16, window=0),
        # plain decoding of a full batch, one token for each of 64 requests of mixed length
        dict(name="attend_decode_batch", op="attend", shape=2, requests=64, n_lo=1, n_hi=1, len_lo=512, len_hi=8191,
             q_heads=64, kv_heads=8, width=128, block=64, window=0),
        # verification of up to eight drafted tokens for 16 requests, short and long ones together
        dict(name="attend_verify_batch", op="attend", shape=3, requests=16, n_lo=2, n_hi=8, len_lo=1000,
             len_hi=32768, q_heads=64, kv_heads=8, width=128, block=32, window=0),
        # one request far into a long document: the prefix has to be split over the whole card
        dict(name="attend_long_document", op="attend", shape=4, requests=1, n_lo=8, n_hi=8, len_lo=131071,
             len_hi=131071, q_heads=64, kv_heads=8, width=128, block=64, window=0),
        # wide trees (33 to 64 drafts) for 32 requests: enough rows for the tensor cores to bind
        dict(name="attend_wide_trees", op="attend", shape=5, requests=32, n_lo=33, n_hi=64, len_lo=1024, len_hi=8192,
             q_heads=64, kv_heads=8, width=128, block=32, window=0),
        # a sliding-window layer: 48 long requests, 2048 tokens each in sight, three query heads to a key head
        dict(name="attend_window_layer", op="attend", shape=6, requests=48, n_lo=1, n_hi=7, len_lo=300, len_hi=32768,
             q_heads=24, kv_heads=8, width=64, block=16, window=2048),
        # the masks of one user's eight drafts
        dict(name="masks_one_user", op="masks", shape=7, requests=1, n_lo=8, n_hi=8, words=1),
        # the masks of wide trees for a large batch
        dict(name="masks_wide_trees", op="masks", shape=8, requests=1024, n_lo=1, n_hi=200, words=4),
        # one step's block tables and slots for eight running requests
        dict(name="plan_small_batch", op="plan", shape=9, requests=8, new_hi=8, prompt_share=0.0, prompt_hi=8,
             release_share=0.0, len_hi=4000, block=16, scarce=False),
        # a large server's step: most requests append accepted tokens, some bring a prompt, some end
        dict(name="plan_large_server", op="plan", shape=10, requests=4096, new_hi=8, prompt_share=0.02,
             prompt_hi=1500, release_share=0.03, len_hi=8000, block=16, scarce=False),
        # the accepted drafts of 64 requests, gathered from the drafted rows into their slots
        dict(name="write_accepted", op="write", shape=11, tokens=211, rows=512, kv_heads=8, width=128, block=16,
             blocks=512, gather=True),
        # a prompt of 16384 tokens written row by row
        dict(name="write_prompt", op="write", shape=12, tokens=16384, rows=16384, kv_heads=8, width=128, block=64,
             blocks=512, gather=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "masks", "plan", "write"])
    shape = rng.randrange(1 << 30)
    if op == "attend":
        q_heads, kv_heads, width = rng.choice([(64, 8, 128), (32, 4, 128), (40, 8, 128), (16, 16, 128), (24, 8, 64),
                                               (64, 8, 64), (8, 1, 64)])
        n_hi = _log(rng, 1, 64)
        # no more than the listed cases read from the cache or compute
        room = 190000 * 1024 // (kv_heads * width)
        len_hi = min(_log(rng, 16, 131072), room)
        most = min(64, room // len_hi, int(1.7e11 / (4.0 * q_heads * width * len_hi * n_hi)))
        return dict(op=op, shape=shape, requests=_log(rng, 1, max(1, most)), n_lo=rng.randint(1, n_hi), n_hi=n_hi,
                    len_lo=rng.randint(0, len_hi), len_hi=len_hi, q_heads=q_heads, kv_heads=kv_heads, width=width,
                    block=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, 2048, 333]))
    if op == "masks":
        n_hi = _log(rng, 1, 200)
        return dict(op=op, shape=shape, requests=_log(rng, 1, 1024), n_lo=rng.randint(1, n_hi), n_hi=n_hi,
                    words=(n_hi + 63) // 64)
    if op == "plan":
        return dict(op=op, shape=shape, requests=_log(rng, 1, 4096), new_hi=rng.randint(1, 16),
                    prompt_share=rng.choice([0.0, 0.02, 0.2]), prompt_hi=_log(rng, 16, 1500),
                    release_share=rng.choice([0.0, 0.05]), len_hi=_log(rng, 16, 8000), block=rng.choice([16, 32, 64]),
                    scarce=rng.random() < 0.4)
    gather = rng.random() < 0.5
    tokens = _log(rng, 1, 16384)
    block = rng.choice([16, 32, 64, 128])
    return dict(op=op, shape=shape, tokens=tokens, rows=tokens + (rng.randint(0, tokens) if gather else 0),
                kv_heads=rng.choice([1, 3, 8]), width=rng.choice([64, 128]), block=block,
                blocks=tokens // block + rng.randint(1, 64), gather=gather)


def _lengths(case):
    """Cached tokens and drafted tokens of each request of an attend or masks case."""
    r = random.Random(case["shape"])
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["requests"])]
    if case["op"] == "masks":
        return [r.randint(0, 5000) for _ in n], n
    lo, hi = case["len_lo"], case["len_hi"]
    lens = [int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1 for _ in n]
    lens[0] = hi
    return lens, n


def _plan_shape(case):
    """Held tokens and new tokens (-1: the request ends) of each request, and the free blocks' share."""
    r = random.Random(case["shape"])
    lens, new = [], []
    for _ in range(case["requests"]):
        kind = r.random()
        if kind < case["prompt_share"]:
            lens.append(0)
            new.append(r.randint(1, case["prompt_hi"]))
        elif kind < case["prompt_share"] + case["release_share"]:
            lens.append(r.randint(1, case["len_hi"]))
            new.append(-1)
        else:
            lens.append(r.randint(1, case["len_hi"]))
            new.append(r.randint(0, case["new_hi"]))
    return lens, new


# ---------------------------------------------------------------------------------------------
# what the operators cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "attend":
        lens, n = _lengths(case)
        d, hq, hk, w = case["width"], case["q_heads"], case["kv_heads"], case["window"]
        seen = [min(x, w - 1) if w else x for x in lens]
        t = sum(n)
        blocks = sum(-(-x // case["block"]) for x in seen)
        byts = 2 * 2 * hk * d * (sum(seen) + t) + 2 * 2 * hq * d * t + 4 * hq * t + 8 * t + 4 * t + 4 * blocks
        # a drafted token sees its ancestors and itself: at least half of a chain's triangle is not there to skip
        pairs = sum(a * s + a for a, s in zip(n, seen))
        return {"bytes": byts, "flops": 4 * d * hq * pairs}
    if case["op"] == "masks":
        _, n = _lengths(case)
        return {"bytes": sum(n) * (4 + 4 + 8 * case["words"]) + 8 * len(n), "flops": 0}
    if case["op"] == "plan":
        lens, new = _plan_shape(case)
        bs = case["block"]
        need = sum(max(0, -(-(a + max(b, 0)) // bs) - -(-a // bs)) for a, b in zip(lens, new) if b >= 0)
        freed = sum(-(-a // bs) for a, b in zip(lens, new) if b < 0)
        # per request three numbers in and three out; per new block one read and one write; per token one slot
        return {"bytes": 24 * len(lens) + 8 * (need + freed) + 4 * sum(max(b, 0) for b in new), "flops": 0}
    row = 2 * case["kv_heads"] * case["width"]
    return {"bytes": 2 * 2 * row * case["tokens"] + (8 if case["gather"] else 4) * case["tokens"], "flops": 0}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _parents(rs, n, offsets):
    """Random trees: a node continues the node before it (half of the time) or hangs off an earlier one or the prefix."""
    i = np.concatenate([np.arange(x) for x in n]) if len(n) else np.zeros(0, int)
    up = (rs.random_sample(i.size) * (i + 1)).astype(np.int64) - 1
    return np.where(rs.random_sample(i.size) < 0.5, i - 1, up).astype(np.int32)


def _tree_masks_host(parents, n, words):
    mask = np.zeros((len(parents), words), np.uint64)
    depth = np.zeros(len(parents), np.int32)
    at = 0
    for x in n:
        bits, dep = [], []
        for i in range(x):
            p = int(parents[at + i])
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            dep.append(dep[p] + 1 if p >= 0 else 0)
            for w in range(words):
                mask[at + i, w] = np.uint64(bits[-1] >> (64 * w) & (1 << 64) - 1)
        depth[at:at + x] = dep
        at += x
    return mask.view(np.int64), depth


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    s = {"case": case}

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    if case["op"] in ("attend", "masks"):
        lens, n = _lengths(case)
        offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        t = int(offsets[-1])
        parents = _parents(rs, n, offsets)
        s |= {"lens": dev(np.array(lens, np.int32)), "token_offsets": dev(offsets), "tokens": t, "n_max": max(n)}
    if case["op"] == "masks":
        s["parents"] = dev(parents)
        return s
    if case["op"] == "attend":
        hq, hk, d, bs = case["q_heads"], case["kv_heads"], case["width"], case["block"]
        held = [-(-x // bs) for x in lens]
        blocks, wide = sum(held) + 3, max(1, max(held))
        order, at = rs.permutation(blocks).astype(np.int32), 0
        table = np.zeros((len(lens), wide), np.int32)
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        words = (max(n) + 63) // 64
        mask, depth = _tree_masks_host(parents, n, words)
        pos = depth + np.repeat(np.array(lens, np.int32), n)
        # keys with channels of unequal size, as projections after a norm have them
        size = torch.empty(hk, 1, d, device="cuda").uniform_(0.5, 1.5, generator=g)
        k = (torch.randn(blocks, hk, bs, d, device="cuda", generator=g) * size).bfloat16()
        v = torch.randn(blocks, hk, bs, d, device="cuda", generator=g).bfloat16()
        # the rows of a fused projection: queries, keys and values of a token side by side
        qkv = torch.randn(t, (hq + 2 * hk) * d, device="cuda", generator=g).bfloat16()
        q, kn, vn = qkv.split([hq * d, hk * d, hk * d], dim=1)
        s |= {"k": k, "v": v, "q": q.unflatten(1, (hq, d)), "k_new": kn.unflatten(1, (hk, d)),
              "v_new": vn.unflatten(1, (hk, d)), "block_table": dev(table), "mask": dev(mask),
              "pos": dev(pos.astype(np.int32)), "scale": d ** -0.5, "len_max": max(lens)}
        return s
    if case["op"] == "plan":
        lens, new = _plan_shape(case)
        bs = case["block"]
        owned = np.array([-(-x // bs) for x in lens], np.int32)
        tokens = sum(max(x, 0) for x in new)
        after = max(1, max(-(-(a + max(b, 0)) // bs) for a, b in zip(lens, new)))
        need = sum(max(0, -(-(a + max(b, 0)) // bs) - -(-a // bs)) for a, b in zip(lens, new) if b >= 0)
        free = need // 2 if case["scarce"] else need + 64
        size = int(owned.sum()) + free + 8
        order = rs.permutation(size).astype(np.int32)
        table = np.full((len(lens), after), -1, np.int32)
        filled = np.arange(after)[None, :] < owned[:, None]
        table[filled] = order[:int(owned.sum())]
        head = int(rs.randint(size))
        ring = np.full(size, -1, np.int32)
        ring[(head + np.arange(free)) % size] = order[size - free:]
        s |= {"lens": dev(np.array(lens, np.int32)), "new": dev(np.array(new, np.int32)), "owned": dev(owned),
              "block_table": dev(table), "ring": dev(ring), "ring_state": dev(np.array([head, free], np.int32)),
              "tokens": max(1, tokens)}
        return s
    hk, d, bs, t = case["kv_heads"], case["width"], case["block"], case["tokens"]
    kv = torch.randn(case["rows"], 2 * hk * d, device="cuda", generator=g).bfloat16()
    kn, vn = kv.split([hk * d, hk * d], dim=1)
    slots = rs.permutation(case["blocks"] * bs)[:t].astype(np.int32) if case["gather"] else \
        (rs.permutation(case["blocks"])[:, None] * bs + np.arange(bs)).reshape(-1)[:t].astype(np.int32)
    if t > 8:
        slots[rs.randint(t)] = -1  # a token whose request had no room
    s |= {"k": torch.randn(case["blocks"], hk, bs, d, device="cuda", generator=g).bfloat16(),
          "v": torch.randn(case["blocks"], hk, bs, d, device="cuda", generator=g).bfloat16(),
          "k_new": kn.unflatten(1, (hk, d)), "v_new": vn.unflatten(1, (hk, d)), "slots": dev(slots),
          "src": dev(np.sort(rs.permutation(case["rows"])[:t]).astype(np.int32)) if case["gather"] else None}
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _plain_attend(s):
    case = s["case"]
    hq, hk, d, bs, w = case["q_heads"], case["kv_heads"], case["width"], case["block"], case["window"]
    lens, off = s["lens"].long(), s["token_offsets"].long()
    n, b, grp = s["n_max"], lens.numel(), hq // hk
    dev = lens.device
    # rows of a request, padded to the longest
    i = torch.arange(n, device=dev)
    live = i < (off[1:] - off[:-1])[:, None]
    row = torch.where(live, off[:-1, None] + i, 0)
    pos = s["pos"].long()[row]
    q = s["q"][row].float().unflatten(2, (hk, grp)).permute(0, 2, 1, 3, 4).reshape(b, hk, n * grp, d)
    # the part of the prefix that a window leaves, padded to the longest
    span = min(s["len_max"], w - 1) if w else s["len_max"]
    first = (lens - span).clamp(min=0)
    p = first[:, None] + torch.arange(span, device=dev)
    held = p < lens[:, None]
    p = torch.where(held, p, 0)
    blk = torch.gather(s["block_table"].long(), 1, p // bs)

    def keys(cache, fresh):
        c = cache[blk, :, p % bs].float().masked_fill(~held[:, :, None, None], 0.0)
        f = fresh[row].float().masked_fill(~live[:, :, None, None], 0.0)
        return torch.cat([c, f], dim=1).transpose(1, 2)

    see_prefix = held[:, None, :] & live[:, :, None]
    word = s["mask"][row]
    see_draft = (torch.gather(word, 2, (i // 64).expand(b, n, n)) >> (i % 64) & 1).bool()
    see_draft = see_draft & live[:, :, None] & live[:, None, :]
    if w:
        see_prefix = see_prefix & (pos[:, :, None] - p[:, None, :] < w)
        see_draft = see_draft & (pos[:, :, None] - pos[:, None, :] < w)
    see = torch.cat([see_prefix, see_draft], dim=2)
    see = see[:, None, :, None, :].expand(b, hk, n, grp, span + n).reshape(b, hk, n * grp, span + n)
    x = (torch.matmul(q, keys(s["k"], s["k_new"]).transpose(2, 3)) * s["scale"]).masked_fill(~see, -math.inf)
    top = x.amax(dim=3, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(dim=3, keepdim=True)
    o = torch.matmul(e, keys(s["v"], s["v_new"])) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top)[..., 0]
    o = o.unflatten(2, (n, grp)).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d)
    lse = lse.unflatten(2, (n, grp)).permute(0, 2, 1, 3).reshape(b, n, hq)
    return {"out": o[live].bfloat16(), "lse": lse[live]}


def _own_attend(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:  # what a serving loop holds from step to step
        case = s["case"]
        cache = lm.kv_cache_of(s["k"], s["v"])
        dims = lm.attn_dims_of(n_requests=case["requests"], n_tokens=s["tokens"], max_request_tokens=s["n_max"],
                               q_heads=case["q_heads"], max_blocks=s["block_table"].shape[1],
                               mask_words=s["mask"].shape[1], window=case["window"], scale=s["scale"])
        q = s["q"]
        s["kept"] = (dims, cache, torch.empty(q.shape, dtype=q.dtype, device=q.device),
                     torch.empty(q.shape[:2], dtype=torch.float32, device=q.device),
                     torch.empty(lm.lmoe_tree_attention_workspace_bytes(dims, cache), dtype=torch.uint8,
                                 device=q.device))
    dims, cache, out, lse, ws = s["kept"]
    lm.lmoe_tree_attention(dims, cache, s["q"], s["k_new"], s["v_new"], s["token_offsets"], s["lens"],
                           s["block_table"], s["mask"], s["pos"], out, lse, ws)
    return {"out": out, "lse": lse}


def _plain_masks(s):
    off = s["token_offsets"].long()
    n, words = s["n_max"], s["case"]["words"]
    i = torch.arange(n, device=off.device)
    live = i < (off[1:] - off[:-1])[:, None]
    up = torch.where(live, s["parents"].long()[torch.where(live, off[:-1, None] + i, 0)], -1)
    # reflexive closure of the parent relation, by squaring
    a = torch.eye(n, device=off.device) + (up[:, :, None] == i).float()
    for _ in range(max(1, n - 1).bit_length()):
        a = (torch.matmul(a, a) > 0).float()
    bits = torch.nn.functional.pad((a > 0).long(), (0, 64 * words - n)).unflatten(2, (words, 64))
    mask = (bits << torch.arange(64, device=off.device)).sum(dim=3)
    pos = s["lens"][:, None] + (a.sum(dim=2) - 1).int()
    return {"mask": mask[live], "pos": pos[live]}


def _own_masks(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:
        dev = s["lens"].device
        s["kept"] = (torch.empty(s["tokens"], s["case"]["words"], dtype=torch.int64, device=dev),
                     torch.empty(s["tokens"], dtype=torch.int32, device=dev))
    mask, pos = s["kept"]
    lm.lmoe_tree_masks(s["token_offsets"], s["parents"], s["lens"], mask, pos)
    return {"mask": mask, "pos": pos}


def _plain_plan(s):
    bs, cap = s["case"]["block"], s["tokens"]
    lens, new, owned = s["lens"].long(), s["new"].long(), s["owned"].long()
    table, ring = s["block_table"], s["ring"]
    wide, size = table.shape[1], ring.numel()
    head, count = s["ring_state"].long().unbind()
    add = new.clamp(min=0)
    end = add.cumsum(0)
    start = end - add
    after = (lens + add + bs - 1) // bs
    fits = (new >= 0) & (after <= wide) & (end <= cap)
    need = torch.where(fits, (after - owned).clamp(min=0), 0)
    taken = need.cumsum(0)
    served = fits & ((need == 0) | (taken <= count))
    need, before = torch.where(served, need, 0), taken - need
    ends = new < 0
    freed = torch.where(ends, owned, 0)
    push = freed.cumsum(0) - freed
    j = torch.arange(wide, device=lens.device)
    # blocks of ended requests go to the ring's tail, new ones come from its head
    back = (j < freed[:, None]).nonzero(as_tuple=True)
    ring[(head + count + push[back[0]] + back[1]) % size] = table[back]
    grow = ((j >= owned[:, None]) & (j < (owned + need)[:, None])).nonzero(as_tuple=True)
    table[grow] = ring[(head + before[grow[0]] + grow[1] - owned[grow[0]]) % size]
    t = torch.arange(cap, device=lens.device)
    b = torch.searchsorted(end, t, right=True).clamp(max=lens.numel() - 1)
    p = (lens[b] + t - start[b]).clamp(min=0)
    slot = table.long()[b, (p // bs).clamp(max=wide - 1)] * bs + p % bs
    slot = torch.where(served[b] & (t < end[b]), slot, -1)
    got = need.sum()
    return {"block_table": table, "ring": ring, "slots": slot.int(),
            "token_offsets": torch.cat([start[:1], end]).int(),
            "lens": torch.where(ends, 0, torch.where(served, lens + add, lens)).int(),
            "owned": torch.where(ends, 0, owned + need).int(),
            "ring_state": torch.stack([(head + got) % size, count - got + freed.sum()]).int()}


def _own_plan(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:
        b, dev = s["lens"].numel(), s["lens"].device
        s["kept"] = {k: torch.empty(m, dtype=torch.int32, device=dev) for k, m in
                     (("lens", b), ("owned", b), ("ring_state", 2), ("token_offsets", b + 1), ("slots", s["tokens"]))}
    o = s["kept"]
    lm.lmoe_kv_plan(s["case"]["block"], s["lens"], s["new"], s["owned"], s["block_table"], s["ring"], s["ring_state"],
                    o["lens"], o["owned"], o["ring_state"], o["token_offsets"], o["slots"])
    return {"block_table": s["block_table"], "ring": s["ring"], **o}


def _plain_write(s):
    bs = s["case"]["block"]
    keep = (s["slots"] >= 0).nonzero(as_tuple=True)[0]
    slot = s["slots"].long()[keep]
    src = s["src"].long()[keep] if s["src"] is not None else keep
    s["k"][slot // bs, :, slot % bs] = s["k_new"][src]
    s["v"][slot // bs, :, slot % bs] = s["v_new"][src]
    return {"k": s["k"], "v": s["v"]}


def _own_write(s):
    import latent_moe_layer_fp32_gb300 as lm

    if "kept" not in s:
        s["kept"] = lm.kv_cache_of(s["k"], s["v"])
    lm.lmoe_kv_write(s["kept"], s["k_new"], s["v_new"], s["src"], s["slots"])
    return {"k": s["k"], "v": s["v"]}


_PLAIN = {"attend": _plain_attend, "masks": _plain_masks, "plan": _plain_plan, "write": _plain_write}
_OWN = {"attend": _own_attend, "masks": _own_masks, "plan": _own_plan, "write": _own_write}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, request by request
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("masks", "plan"):
        return None  # whole numbers
    s = prepare(case, seed)
    bs = case["block"]
    if case["op"] == "write":
        k, v = s["k"].double(), s["v"].double()
        slots = s["slots"].tolist()
        src = s["src"].tolist() if case["gather"] else list(range(len(slots)))
        pairs = [(a, b) for a, b in zip(slots, src) if a >= 0]
        for x in range(bs):  # slot by slot of a block
            at = [(a // bs, b) for a, b in pairs if a % bs == x]
            if at:
                to, of = (torch.tensor(z, device="cuda") for z in zip(*at))
                k[to, :, x] = s["k_new"].double()[of]
                v[to, :, x] = s["v_new"].double()[of]
        return {"k": k, "v": v}
    lens, n = _lengths(case)
    hq, hk, w = case["q_heads"], case["kv_heads"], case["window"]
    outs, lses, at = [], [], 0
    flat_k, flat_v = (c.transpose(1, 2).reshape(-1, hk, case["width"]) for c in (s["k"], s["v"]))
    for b, (ln, m) in enumerate(zip(lens, n)):
        lo = max(0, ln - w + 1) if w else 0
        t = torch.arange(lo, ln, device="cuda")
        rows = s["block_table"][b].long()[t // bs] * bs + t % bs
        k = torch.cat([flat_k[rows], s["k_new"][at:at + m]]).double()
        v = torch.cat([flat_v[rows], s["v_new"][at:at + m]]).double()
        at_pos = s["pos"][at:at + m].long()
        key_pos = torch.cat([t, at_pos])
        bits = s["mask"][at:at + m].cpu().numpy().view(np.uint64)
        tree = torch.tensor([[int(bits[i, j // 64]) >> (j % 64) & 1 for j in range(m)] for i in range(m)],
                            dtype=torch.bool, device="cuda")
        see = torch.cat([torch.ones(m, ln - lo, dtype=torch.bool, device="cuda"), tree], dim=1)
        if w:
            see &= at_pos[:, None] - key_pos[None, :] < w
        for h in range(hq):
            x = (s["q"][at:at + m, h].double() @ k[:, h // (hq // hk)].T) * s["scale"]
            x = torch.where(see, x, torch.full_like(x, -math.inf))
            z = torch.logsumexp(x, dim=1)
            outs.append(torch.exp(x - z[:, None]) @ v[:, h // (hq // hk)])
            lses.append(z)
        at += m
    out = [torch.stack(outs[i * hq:(i + 1) * hq], dim=1) for i in range(len(n))]
    lse = [torch.stack(lses[i * hq:(i + 1) * hq], dim=1) for i in range(len(n))]
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
