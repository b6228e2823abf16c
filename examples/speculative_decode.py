"""Speculative decoding with trees of drafts over a paged key/value cache.

    python examples/speculative_decode.py [--layers 2] [--requests 6] [--tokens 48] [--block-size 16]

A small model with random weights (attention with rotary positions, then the latent
mixture-of-experts sandwich block, a few layers of both) continues several prompts.  Each step
runs what a server runs around a verify step:

    lmoe_tree_masks       the drafter's trees -> masks and positions
    per layer
      lmoe_tree_attention   the drafted rows over the cached tokens and their own ancestors
      lmoe_block_forward    the mixture-of-experts block
    (the longest path of each tree that the model agrees with is accepted)
    lmoe_kv_plan          the accepted counts -> blocks, lengths and slots
    lmoe_kv_write         per layer, the accepted rows -> the cache

A prompt enters by the same calls, as chains of up to 256 rows; a request that ends gives its
blocks back and another takes its place.  The result is checked against decoding one token a step.

The linear layers around the library's calls (projections, embedding, output) are plain matrix
products; the drafter is a table: the output matrix is the embedding in another order, so the
token that the residual stream alone would give is known in advance.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import latent_moe_layer_fp32_gb300 as lm  # noqa: E402
import synth  # noqa: E402

VOCAB, HEADS, KV_HEADS, HEAD_DIM = 512, 8, 2, 64
CHUNK = 256  # rows of a prompt in one call


def _device(a):
    if a is None:
        return None
    t = torch.from_numpy(a.view("int16") if a.dtype == "uint16" else a)
    return t.cuda().view(torch.bfloat16) if a.dtype == "uint16" else t.cuda()


class Model:
    """Weights; its forward pass over ragged rows is `Server.rows`."""

    def __init__(self, layers, seed=0):
        self.d = synth.CONFIGS["tiny"]
        g = torch.Generator().manual_seed(seed)
        width = (HEADS + 2 * KV_HEADS) * HEAD_DIM

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()

        h = self.d.H
        self.embed = normal(VOCAB, h, std=0.25)  # small: the layers overrule the table now and then
        self.follows = torch.randperm(VOCAB, generator=g)  # the token that the embedding alone leads to
        head = torch.empty_like(self.embed)
        head[self.follows.cuda()] = self.embed
        self.head = head
        self.layers = []
        for i in range(layers):
            w = {k: _device(v) for k, v in synth.make_weights(self.d, seed=seed + i).items()}
            nw = {k: _device(v) for k, v in synth.make_block_norms(self.d, seed=seed + i).items()}
            self.layers.append({
                "qkv": normal(h, width, std=h ** -0.5), "out": normal(HEADS * HEAD_DIM, h, std=h ** -0.5),
                "moe": lm.weights_of(w), "norms": lm.norms_of(nw, self.d.eps), "keep": (w, nw)})


def _rms(x, eps):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)).to(torch.bfloat16)


def _rotate(x, pos):
    """Rotary positions of rows [T, heads, HEAD_DIM]."""
    half = HEAD_DIM // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    a = pos.float()[:, None] * freq
    c, s = a.cos()[:, None], a.sin()[:, None]
    lo, hi = x[..., :half].float(), x[..., half:].float()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1).to(torch.bfloat16)


class Server:
    """A paged cache of every layer, and places for requests that live in it."""

    def __init__(self, model, requests, blocks, block_size, max_blocks):
        self.m, self.b, self.bs = model, requests, block_size
        dev = dict(device="cuda", dtype=torch.int32)
        shape = (blocks, KV_HEADS, block_size, HEAD_DIM)
        self.kv = [(torch.zeros(shape, device="cuda", dtype=torch.bfloat16),
                    torch.zeros(shape, device="cuda", dtype=torch.bfloat16)) for _ in model.layers]
        self.cache = [lm.kv_cache_of(k, v) for k, v in self.kv]
        self.table = torch.zeros((requests, max_blocks), **dev)
        self.ring = torch.arange(blocks, **dev)
        # two sets of lengths, block counts and ring states: a plan reads one and writes the other
        self.lens = [torch.zeros(requests, **dev), torch.zeros(requests, **dev)]
        self.owned = [torch.zeros(requests, **dev), torch.zeros(requests, **dev)]
        self.state = [torch.tensor([0, blocks], **dev), torch.zeros(2, **dev)]
        self.ws = torch.empty(0, dtype=torch.uint8, device="cuda")

    def _workspace(self, n):
        if self.ws.numel() < n:
            self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        return self.ws

    def rows(self, tokens, offsets, parents):
        """Logits of the drafted rows, and each layer's new keys and values (not in the cache yet)."""
        t, d = len(tokens), self.m.d
        n_max = max(b - a for a, b in zip(offsets, offsets[1:]))
        words = (n_max + 63) // 64
        dev = dict(device="cuda", dtype=torch.int32)
        off = torch.tensor(offsets, **dev)
        mask = torch.empty((t, words), device="cuda", dtype=torch.int64)
        pos = torch.empty(t, **dev)
        ws = self._workspace(256)
        lm.lmoe_tree_masks(off, torch.tensor(parents, **dev), self.lens[0], mask, pos, ws)
        assert lm.lmoe_status_check(ws) == 0
        attn = lm.attn_dims_of(self.b, t, n_max, HEADS, self.table.shape[1], words, HEAD_DIM ** -0.5)
        moe = lm.dims_of(t, d.H, d.L, d.I, d.E, d.k, d.eps)
        ws = self._workspace(max(lm.lmoe_block_workspace_bytes(moe),
                                 lm.lmoe_tree_attention_workspace_bytes(attn, self.cache[0])))
        x = self.m.embed[torch.tensor(tokens, device="cuda")]
        o = torch.empty((t, HEADS, HEAD_DIM), device="cuda", dtype=torch.bfloat16)
        new = []
        for cache, w in zip(self.cache, self.m.layers):
            qkv = (_rms(x, d.eps) @ w["qkv"]).view(t, HEADS + 2 * KV_HEADS, HEAD_DIM)
            qk = _rotate(qkv[:, :HEADS + KV_HEADS], pos)
            k, v = qk[:, HEADS:], qkv[:, HEADS + KV_HEADS:]  # slices: rows lie apart
            lm.lmoe_tree_attention(attn, cache, qk[:, :HEADS], k, v, off, self.lens[0], self.table, mask, pos, o,
                                   None, ws)
            assert lm.lmoe_status_check(ws) == 0
            x = x + o.view(t, -1) @ w["out"]
            lm.lmoe_block_forward(moe, w["moe"], w["norms"], x, x, ws)
            assert lm.lmoe_status_check(ws) == 0
            new.append((k, v))
        return _rms(x, d.eps).float() @ self.m.head.float().T, new

    def commit(self, counts, new=None, src=()):
        """counts[b] rows of request b (those of src, in request order) enter the cache; -1 ends the request."""
        dev = dict(device="cuda", dtype=torch.int32)
        n = max(1, sum(max(c, 0) for c in counts))
        slots = torch.empty(n, **dev)
        off = torch.empty(self.b + 1, **dev)
        lm.lmoe_kv_plan(self.bs, self.lens[0], torch.tensor(counts, **dev), self.owned[0], self.table, self.ring,
                        self.state[0], self.lens[1], self.owned[1], self.state[1], off, slots)
        served = [int(b) - int(a) == c or c < 0 for a, b, c in
                  zip(self.lens[0].tolist(), self.lens[1].tolist(), counts)]
        if not all(served):
            raise RuntimeError("out of cache blocks")
        for pair in (self.lens, self.owned, self.state):
            pair.reverse()
        if src:
            at = torch.tensor(src, **dev)
            for cache, (k, v) in zip(self.cache, new):
                ws = self._workspace(256)
                lm.lmoe_kv_write(cache, k, v, at, slots, ws)
                assert lm.lmoe_status_check(ws) == 0

    def prompt(self, place, tokens):
        """A prompt into the cache, all but its last token, in chains of up to CHUNK rows."""
        for a in range(0, len(tokens) - 1, CHUNK):
            part = tokens[a:min(a + CHUNK, len(tokens) - 1)]
            offsets = [0 if b <= place else len(part) for b in range(self.b + 1)]
            _, new = self.rows(part, offsets, list(range(-1, len(part) - 1)))
            self.commit([len(part) if b == place else 0 for b in range(self.b)], new, list(range(len(part))))


def draft(model, last, depth, g):
    """A tree over the last accepted token: the table's chain, with a random sibling beside each of its nodes
    (now and then before it).  Tokens and parents; the root's parent is the cached prefix."""
    tokens, parents, at = [last], [-1], 0
    for _ in range(depth):
        chain = int(model.follows[tokens[at]])
        other = int(torch.randint(VOCAB, (1,), generator=g))
        pair = [chain, other] if torch.rand(1, generator=g) < 0.7 else [other, chain]
        here = len(tokens)
        tokens += pair
        parents += [at, at]
        at = here + pair.index(chain)
    return tokens, parents


def accept(tokens, parents, choice):
    """The path from the root along the model's own choices: its rows and the token after it."""
    path, at = [0], 0
    while True:
        nxt = next((i for i in range(at + 1, len(tokens)) if parents[i] == at and tokens[i] == choice[at]), None)
        if nxt is None:
            return path, choice[at]
        path.append(nxt)
        at = nxt


def generate(model, prompts, tokens, places=4, block_size=16, depth=4, seed=1):
    """Continues each prompt by `tokens` tokens, `places` requests at a time, depth drafted levels a step (0: one
    token a step).  Returns the continuations and the number of steps."""
    longest = max(len(p) for p in prompts) + tokens + depth + 1
    max_blocks = -(-longest // block_size)
    srv = Server(model, places, places * max_blocks, block_size, max_blocks)
    g = torch.Generator().manual_seed(seed)
    waiting, live, out, steps = list(range(len(prompts))), [None] * places, [[] for _ in prompts], 0
    last = [0] * len(prompts)
    while True:
        for b in range(places):
            if live[b] is None and waiting:
                live[b] = waiting.pop(0)
                srv.prompt(b, prompts[live[b]])
                last[live[b]] = prompts[live[b]][-1]
        if not any(r is not None for r in live):
            return out, steps
        toks, parents, offsets = [], [], [0]
        for b in range(places):
            if live[b] is not None:
                t, p = draft(model, last[live[b]], depth, g)
                toks, parents = toks + t, parents + p
            offsets.append(len(toks))
        logits, new = srv.rows(toks, offsets, parents)
        choice = logits.argmax(-1).tolist()
        steps += 1
        counts, src = [0] * places, []
        for b in range(places):
            if live[b] is None:
                continue
            a, e = offsets[b], offsets[b + 1]
            path, nxt = accept(toks[a:e], parents[a:e], choice[a:e])
            counts[b] = len(path)
            src += [a + i for i in path]
            out[live[b]] += [toks[a + i] for i in path[1:]] + [nxt]
            last[live[b]] = nxt
        srv.commit(counts, new, src)
        ended = [r is not None and len(out[r]) >= tokens for r in live]
        if any(ended):
            srv.commit([-1 if e else 0 for e in ended])
            for b in range(places):
                if ended[b]:
                    out[live[b]] = out[live[b]][:tokens]
                    live[b] = None


def margins(model, prompts, outs, block_size=16):
    """How far each generated token's logit lies below the best one when the model decodes one token a step,
    with the generated tokens as its input (0: its own choice)."""
    n = len(prompts)
    longest = max(len(p) + len(o) for p, o in zip(prompts, outs))
    srv = Server(model, n, n * -(-longest // block_size), block_size, -(-longest // block_size))
    for b, p in enumerate(prompts):
        srv.prompt(b, p)
    gaps, feed = [], [p[-1] for p in prompts]
    for i in range(len(outs[0])):
        logits, new = srv.rows(feed, list(range(n + 1)), [-1] * n)
        srv.commit([1] * n, new, list(range(n)))
        feed = [o[i] for o in outs]
        gaps += (logits.max(-1).values - logits[torch.arange(n), feed]).tolist()
    return gaps, float(logits.std())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--block-size", type=int, default=16)
    a = ap.parse_args()
    lm.build()
    model = Model(a.layers)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(VOCAB, (1 + 97 * i,), generator=g).tolist() for i in range(a.requests)]
    outs, steps = generate(model, prompts, a.tokens, block_size=a.block_size)
    plain, plain_steps = generate(model, prompts, a.tokens, block_size=a.block_size, depth=0)
    gaps, spread = margins(model, prompts, outs, a.block_size)
    same = sum(x == y for o, p in zip(outs, plain) for x, y in zip(o, p))
    print(f"{a.requests} requests x {a.tokens} tokens: {steps} verify steps, {plain_steps} steps of one token each; "
          f"{same} of {a.requests * a.tokens} tokens equal")
    print(f"largest gap to the one-token decoder's best logit: {max(gaps):.3f} (logits' spread {spread:.1f})")


if __name__ == "__main__":
    main()
