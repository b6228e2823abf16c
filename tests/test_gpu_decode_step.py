"""The calls of a decode step together, as a serving loop uses them: lmoe_kv_plan, lmoe_qk_norm_rope in place on the
projection's rows, lmoe_kv_write_fp8, lmoe_decode_attention_fp8 - step by step and as a replayed graph - and
lmoe_kv_read_fp8 into a bf16 cache for lmoe_tree_attention.  Bounds as in test_gpu_decode_fp8.py and
test_gpu_tree_attention.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import latent_moe_layer_fp32_gb300 as lm
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lm.load()
    return lm


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class Loop:
    """A layer's attention for B requests; the projection's rows are given."""

    def __init__(self, lm, B, hq, hk, d, bs, max_blocks, window=0, order="head", seed=0):
        self.lm, self.B, self.hq, self.hk, self.d, self.bs, self.window = lm, B, hq, hk, d, bs, window
        i32 = dict(device="cuda", dtype=torch.int32)
        blocks = B * max_blocks
        shape = (blocks, hk, bs, d) if order == "head" else (blocks, bs, hk, d)
        self.kv = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.kv = [x if order == "head" else x.transpose(1, 2) for x in self.kv]
        self.sc = [torch.full((blocks, hk, bs), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.cache = lm.kv_cache_fp8_of(*self.kv, *self.sc)
        self.table = torch.zeros((B, max_blocks), **i32)
        g = torch.Generator().manual_seed(seed)
        self.ring = torch.randperm(blocks, generator=g).to(**i32)
        self.state = [torch.zeros(B, **i32), torch.zeros(B, **i32), torch.tensor([0, blocks], **i32)]  # lens, owned, ring
        self.next = [torch.empty_like(x) for x in self.state]
        self.new = torch.ones(B, **i32)
        self.off, self.slots = torch.empty(B + 1, **i32), torch.empty(B, **i32)
        self.gain = [(1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2)]
        self.freq = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda()
        self.rope = lm.rope_dims_of(B, hq, hk, d)
        self.dims = lm.decode_dims_of(B, hq, max_blocks, d ** -0.5, window=window)
        self.qkv = torch.zeros(B, (hq + 2 * hk) * d, dtype=torch.bfloat16, device="cuda")
        self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in self.qkv.split([hq * d, hk * d, hk * d], dim=1))
        self.out = torch.empty(B, hq, d, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty(B, hq, device="cuda")
        self.ws = torch.empty(lm.lmoe_decode_attention_fp8_workspace_bytes(self.dims, self.cache), dtype=torch.uint8,
                              device="cuda")

    def step(self):
        """One token for every request, from the projection's rows in self.qkv."""
        lm, (lens, owned, ring), nx = self.lm, self.state, self.next
        lm.lmoe_kv_plan(self.bs, lens, self.new, owned, self.table, self.ring, ring, nx[0], nx[1], nx[2], self.off,
                        self.slots)
        lm.lmoe_qk_norm_rope(self.rope, self.q, self.k, *self.gain, lens, self.freq, None, self.q, self.k)
        lm.lmoe_kv_write_fp8(self.cache, self.k, self.v, None, self.slots)
        lm.lmoe_decode_attention_fp8(self.dims, self.cache, self.q, nx[0], self.table, self.out, self.lse, self.ws)
        for a, b in zip(self.state, nx):
            a.copy_(b)


def bound(q, keys, vals, scales, scale):
    """Reference output of one head's rows and its bound."""
    s = scale * (q @ keys.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    p /= p.sum(axis=1, keepdims=True)
    ref, mass = p @ vals, p @ np.abs(vals)
    S = (scale * (np.abs(q) @ np.abs(keys).T)).max(axis=1)[:, None]
    e = (q.shape[1] + 16) * 2.0**-23 * S + 2.0**-20
    low = (p * scales).max(axis=1)[:, None] * (np.abs(vals) / scales[:, None]).sum(axis=0)
    tol = 2.0**-8 * np.abs(ref) + (2.0**-11 + 2.0**-17 + 2.0**-23 * S + (len(keys) / 16 + 40) * 2.0**-23 + 2 * e) * mass
    return ref, (tol + 2.0**-39 * low + 2.0**-133) * (1 + 2.0**-6)


@pytest.mark.parametrize("graph", [False, True], ids=["calls", "graph"])
@pytest.mark.parametrize("hq,hk,d,bs,window,order", [(8, 2, 64, 16, 0, "head"), (10, 2, 128, 16, 9, "slot"),
                                                     (16, 1, 128, 32, 0, "head")])
def test_steps(lm, hq, hk, d, bs, window, order, graph):
    B, steps = 5, 40
    loop = Loop(lm, B, hq, hk, d, bs, 4, window, order, seed=hq)
    g = torch.Generator(device="cuda").manual_seed(1)
    start = [x.clone() for x in (*loop.state, loop.table, loop.ring)]
    if graph:
        loop.step()  # (warms up; its state is put back)
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            loop.step()
        for a, b in zip((*loop.state, loop.table, loop.ring), start):
            a.copy_(b)
        for x in loop.sc:
            x.fill_(255)
    K, V, VS = np.zeros((B, steps, hk, d)), np.zeros((B, steps, hk, d)), np.zeros((B, steps, hk))
    for i in range(steps):
        rows = torch.randn(loop.qkv.shape, device="cuda", generator=g).bfloat16()
        loop.qkv.copy_(rows)
        captured.replay() if graph else loop.step()
        assert lm.lmoe_status_check(loop.ws) == 0
        q0, k0, _ = rows.split([hq * d, hk * d, hk * d], dim=1)
        pos = np.full((1, B), i)
        q, k = host(loop.q), host(loop.k)
        for got, x, gain in ((q, q0, loop.gain[0]), (k, k0, loop.gain[1])):
            y, pair = fp8_ref.norm_rope(host(x).reshape(B, -1, d), host(gain), pos, loop.freq.cpu().numpy(), None, d,
                                        False, True, 1e-6)
            assert (np.abs(got - y) <= 2.0**-8 * np.abs(y) + (2.0**-21 + (d + 16) * 2.0**-24) * 1.01 * pair).all()
        K[:, i] = fp8_ref.values(*fp8_ref.quantise(k))
        codes, sc = fp8_ref.quantise(host(loop.v))
        V[:, i], VS[:, i] = fp8_ref.values(codes, sc), fp8_ref.scale_values(sc)
        out, lo = host(loop.out), max(0, i + 1 - window) if window else 0
        G = hq // hk
        for b in range(B):
            for h in range(hk):
                of = slice(h * G, (h + 1) * G)
                ref, tol = bound(q[b, of], K[b, lo:i + 1, h], V[b, lo:i + 1, h], VS[b, lo:i + 1, h], d ** -0.5)
                assert (np.abs(out[b, of] - ref) <= tol).all(), (i, b, h)
    assert loop.state[0].tolist() == [steps] * B
    # the rows back, exactly
    off = torch.arange(B + 1, dtype=torch.int32, device="cuda") * steps
    rows = [torch.empty(B * steps, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lm.lmoe_kv_read_fp8(loop.cache, off, None, loop.table, *rows)
    assert np.array_equal(host(rows[0]).reshape(K.shape), K) and np.array_equal(host(rows[1]).reshape(V.shape), V)
    # ... into a bf16 cache, over which the next drafts are verified: one draft sees what the decode step sees and itself
    bf16 = [torch.zeros(loop.kv[0].shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p = torch.arange(steps, device="cuda")
    slots = (loop.table[:, p // bs] * bs + p % bs).flatten().int()
    cache = lm.kv_cache_of(*bf16)
    lm.lmoe_kv_write(cache, *rows, None, slots)
    dims = lm.attn_dims_of(B, B, 1, hq, loop.table.shape[1], 1, d ** -0.5)
    fresh = torch.randn(B, hq + 2 * hk, d, device="cuda", generator=g).bfloat16()
    out = torch.empty(B, hq, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lm.lmoe_tree_attention_workspace_bytes(dims, cache), dtype=torch.uint8, device="cuda")
    lm.lmoe_tree_attention(dims, cache, fresh[:, :hq], fresh[:, hq:hq + hk], fresh[:, hq + hk:],
                           torch.arange(B + 1, dtype=torch.int32, device="cuda"), loop.state[0], loop.table, None, None, out,
                           None, ws)
    assert lm.lmoe_status_check(ws) == 0
    f = host(fresh)
    for b in range(B):
        for h in range(hk):
            keys = np.concatenate([K[b, :, h], f[b, hq + h][None]])
            vals = np.concatenate([V[b, :, h], f[b, hq + hk + h][None]])
            of = slice(h * G, (h + 1) * G)
            ref, tol = bound(f[b, of], keys, vals, np.ones(len(keys)), d ** -0.5)
            mass = np.abs(vals).max(axis=0)  # P is bf16 there: 2^-8 of sum p |v| more
            assert (np.abs(host(out)[b, of] - ref) <= tol + 2.0**-8 * mass).all(), (b, h)


def test_a_request_that_finds_no_block_keeps_its_answers(lm):
    """The plan serves no request past the free blocks: its slot is -1, nothing is written, its length stays."""
    loop = Loop(lm, 2, 4, 2, 64, 16, 2, seed=3)
    loop.state[2].copy_(torch.tensor([0, 1], dtype=torch.int32))  # one block for both
    loop.qkv.copy_(torch.randn(loop.qkv.shape, device="cuda").bfloat16())
    v = host(loop.v)
    loop.step()
    assert lm.lmoe_status_check(loop.ws) == 0
    assert loop.state[0].tolist() == [1, 0] and loop.slots.tolist()[1] == -1
    want = fp8_ref.values(*fp8_ref.quantise(v[0]))  # one position: the value itself
    assert np.abs(host(loop.out)[0].reshape(2, 2, 64) - want[:, None]).max() <= 2.0**-10 * np.abs(want).max()
    assert not loop.out[1].any() and torch.isneginf(loop.lse[1]).all()


def test_another_device_is_refused(lm, monkeypatch):
    loop = Loop(lm, 2, 4, 2, 64, 16, 2)
    i32 = dict(device="cuda", dtype=torch.int32)
    off, rows = torch.zeros(3, **i32), torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    calls = (lambda: lm.lmoe_qk_norm_rope(loop.rope, loop.q, loop.k, None, None, loop.state[0], loop.freq, None, loop.q, loop.k),
             lambda: lm.lmoe_kv_write_fp8(loop.cache, loop.k, loop.v, None, loop.slots),
             lambda: lm.lmoe_kv_read_fp8(loop.cache, off, None, loop.table, rows, rows.clone()),
             lambda: lm.lmoe_decode_attention_fp8(loop.dims, loop.cache, loop.q, loop.state[0], loop.table, loop.out, loop.lse,
                                                  loop.ws))
    here = torch.cuda.current_device()
    monkeypatch.setattr(lm, "_device", lambda: here + 1)  # as if another device were the current one
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
