"""Decoding over an 8-bit paged key/value cache.

    python examples/decode_fp8.py [--layers 2] [--requests 4] [--tokens 48] [--block-size 16]

A small model with random weights (attention with normed heads and rotary positions, then the latent
mixture-of-experts sandwich block) continues several prompts, one token a step for all of them.  Each step runs what a
server runs around a decode step:

    lmoe_kv_plan                 one more token a request -> blocks, lengths and slots
    per layer
      lmoe_qk_norm_rope            the projection's queries and keys, in place
      lmoe_kv_write_fp8            the new keys and values into the cache
      lmoe_decode_attention_fp8    the queries over all that their requests hold
      lmoe_block_forward           the mixture-of-experts block

A prompt enters in chunks of up to 256 rows: lmoe_kv_read_fp8 brings what is cached of it back as bf16 for
lmoe_tree_attention, whose rows then go into the 8-bit cache by lmoe_kv_write_fp8.
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
    def __init__(self, layers, seed=0):
        self.d = synth.CONFIGS["tiny"]
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()

        h = self.d.H
        self.embed, self.head = normal(VOCAB, h, std=1.0), normal(VOCAB, h, std=h ** -0.5)
        self.freq = (10000.0 ** (-torch.arange(HEAD_DIM // 2) / (HEAD_DIM // 2))).float().cuda()
        self.layers = []
        for i in range(layers):
            w = {k: _device(v) for k, v in synth.make_weights(self.d, seed=seed + i).items()}
            nw = {k: _device(v) for k, v in synth.make_block_norms(self.d, seed=seed + i).items()}
            self.layers.append({
                "qkv": normal(h, (HEADS + 2 * KV_HEADS) * HEAD_DIM, std=h ** -0.5),
                "out": normal(HEADS * HEAD_DIM, h, std=h ** -0.5), "q_gain": 1 + normal(HEAD_DIM, std=0.1),
                "k_gain": 1 + normal(HEAD_DIM, std=0.1), "moe": lm.weights_of(w), "norms": lm.norms_of(nw, self.d.eps),
                "keep": (w, nw)})


def _rms(x, eps):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)).to(torch.bfloat16)


class Server:
    """An 8-bit paged cache of every layer, and one place for each request."""

    def __init__(self, model, requests, block_size, max_blocks):
        self.m, self.b, self.bs = model, requests, block_size
        blocks, i32 = requests * max_blocks, dict(device="cuda", dtype=torch.int32)
        shape = (blocks, KV_HEADS, block_size, HEAD_DIM)
        self.keep = [[torch.zeros(s, device="cuda", dtype=torch.uint8) for s in (shape, shape, shape[:3], shape[:3])]
                     for _ in model.layers]
        self.cache = [lm.kv_cache_fp8_of(*x) for x in self.keep]
        self.table = torch.zeros((requests, max_blocks), **i32)
        self.ring = torch.arange(blocks, **i32)
        self.lens = [torch.zeros(requests, **i32), torch.zeros(requests, **i32)]
        self.owned = [torch.zeros(requests, **i32), torch.zeros(requests, **i32)]
        self.state = [torch.tensor([0, blocks], **i32), torch.zeros(2, **i32)]
        # one request's prefix in bf16, block by block in order
        self.bf16 = [torch.zeros((max_blocks, KV_HEADS, block_size, HEAD_DIM), device="cuda", dtype=torch.bfloat16)
                     for _ in range(2)]
        self.prefix = lm.kv_cache_of(*self.bf16)
        self.ws = torch.empty(0, dtype=torch.uint8, device="cuda")

    def workspace(self, n):
        if self.ws.numel() < n:
            self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        return self.ws

    def plan(self, counts):
        i32 = dict(device="cuda", dtype=torch.int32)
        slots, off = torch.empty(max(1, sum(counts)), **i32), torch.empty(self.b + 1, **i32)
        lm.lmoe_kv_plan(self.bs, self.lens[0], torch.tensor(counts, **i32), self.owned[0], self.table, self.ring,
                        self.state[0], self.lens[1], self.owned[1], self.state[1], off, slots)
        for pair in (self.lens, self.owned, self.state):
            pair.reverse()
        if int(slots.min()) < 0:
            raise RuntimeError("out of cache blocks")
        return slots

    def heads(self, w, x, pos):
        """A layer's queries, keys and values of rows x: slices of one projection, normed and turned in place."""
        t = x.shape[0]
        qkv = (_rms(x, self.m.d.eps) @ w["qkv"]).view(t, HEADS + 2 * KV_HEADS, HEAD_DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        lm.lmoe_qk_norm_rope(lm.rope_dims_of(t, HEADS, KV_HEADS, HEAD_DIM), q, k, w["q_gain"], w["k_gain"], pos,
                             self.m.freq, None, q, k)
        return q, k, v

    def block(self, w, x, o):
        d, t = self.m.d, x.shape[0]
        x = x + o.view(t, -1) @ w["out"]
        moe = lm.dims_of(t, d.H, d.L, d.I, d.E, d.k, d.eps)
        ws = self.workspace(lm.lmoe_block_workspace_bytes(moe))
        lm.lmoe_block_forward(moe, w["moe"], w["norms"], x, x, ws)
        assert lm.lmoe_status_check(ws) == 0
        return x

    def logits(self, x):
        return _rms(x, self.m.d.eps).float() @ self.m.head.float().T

    def step(self, tokens):
        """One token a request -> the logits of the next ones."""
        pos = self.lens[0].clone()
        slots = self.plan([1] * self.b)
        dims = lm.decode_dims_of(self.b, HEADS, self.table.shape[1], HEAD_DIM ** -0.5)
        x = self.m.embed[torch.tensor(tokens, device="cuda")]
        o = torch.empty((self.b, HEADS, HEAD_DIM), device="cuda", dtype=torch.bfloat16)
        for cache, w in zip(self.cache, self.m.layers):
            q, k, v = self.heads(w, x, pos)
            lm.lmoe_kv_write_fp8(cache, k, v, None, slots)
            ws = self.workspace(lm.lmoe_decode_attention_fp8_workspace_bytes(dims, cache))
            lm.lmoe_decode_attention_fp8(dims, cache, q, self.lens[0], self.table, o, None, ws)
            assert lm.lmoe_status_check(ws) == 0
            x = self.block(w, x, o)
        return self.logits(x)

    def prompt(self, place, tokens):
        """A prompt, all but its last token, into one request's place."""
        i32 = dict(device="cuda", dtype=torch.int32)
        blocks = torch.arange(self.table.shape[1], **i32)[None]  # of the bf16 prefix
        for at in range(0, len(tokens) - 1, CHUNK):
            part = tokens[at:min(at + CHUNK, len(tokens) - 1)]
            n = len(part)
            slots = self.plan([n if b == place else 0 for b in range(self.b)])
            pos = torch.arange(at, at + n, **i32)
            dims = lm.attn_dims_of(1, n, n, HEADS, self.table.shape[1], (n + 63) // 64, HEAD_DIM ** -0.5)
            x = self.m.embed[torch.tensor(part, device="cuda")]
            o = torch.empty((n, HEADS, HEAD_DIM), device="cuda", dtype=torch.bfloat16)
            rows = [torch.empty((at, KV_HEADS, HEAD_DIM), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
            for cache, w in zip(self.cache, self.m.layers):
                q, k, v = self.heads(w, x, pos)
                if at:
                    lm.lmoe_kv_read_fp8(cache, torch.tensor([0, at], **i32), None, self.table[place:place + 1], *rows)
                    lm.lmoe_kv_write(self.prefix, *rows, None, torch.arange(at, **i32))
                ws = self.workspace(lm.lmoe_tree_attention_workspace_bytes(dims, self.prefix))
                lm.lmoe_tree_attention(dims, self.prefix, q, k, v, torch.tensor([0, n], **i32), torch.tensor([at], **i32),
                                       blocks, None, None, o, None, ws)
                assert lm.lmoe_status_check(ws) == 0
                lm.lmoe_kv_write_fp8(cache, k, v, None, slots)
                x = self.block(w, x, o)


def generate(model, prompts, tokens, block_size=16):
    """Continues each prompt by `tokens` tokens; the continuations and the last step's logits."""
    longest = max(len(p) for p in prompts) + tokens
    srv = Server(model, len(prompts), block_size, -(-longest // block_size))
    for b, p in enumerate(prompts):
        srv.prompt(b, p)
    out, last = [[] for _ in prompts], [p[-1] for p in prompts]
    for _ in range(tokens):
        logits = srv.step(last)
        last = logits.argmax(-1).tolist()
        for o, t in zip(out, last):
            o.append(t)
    return out, logits


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--block-size", type=int, default=16)
    a = ap.parse_args()
    lm.build()
    model = Model(a.layers)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(VOCAB, (1 + 131 * i,), generator=g).tolist() for i in range(a.requests)]
    outs, _ = generate(model, prompts, a.tokens, block_size=a.block_size)
    for p, o in zip(prompts, outs):
        print(f"prompt of {len(p)} tokens -> {o[:8]} ...")
    elements = 2 * KV_HEADS * HEAD_DIM
    print(f"a cached token takes {elements + 2 * KV_HEADS} bytes a layer ({2 * elements} in bf16)")


if __name__ == "__main__":
    main()
