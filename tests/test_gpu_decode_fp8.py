"""Attention of one token a request over the 8-bit paged cache against plain 64-bit loops.

Bounds, from the arithmetic of include/lmoe.h and the kernel (A = sum_j p_j |v_j|; S = max_j scale sum_d |q_d k_jd|):
  scores   queries and codes are exact in f16, their products in fp32; head_dim additions of at most 2^-23
           relative each, the scales and the change of base: |ds| <= (head_dim + 8) 2^-23 S + 2^-22 |s|;
           exponentials 2^-21; so p is off by at most e = (head_dim + 16) 2^-23 S + 2^-20 relative
  out      p times its value's scale stands as f16 with an exponent of its own: the sum of the score and that
           exponent (up to 2^7 + |s|, |s| <= S) rounds in fp32, 2^-17 + 2^-23 S; rounding to f16 2^-11 A, or, below
           2^-28 of the row's largest p * scale, 2^-39 of that for each code; fp32 sums over n keys (n / 16 + 40) 2^-23 A;
           the result's own rounding to bf16 2^-8 |out|
  lse      e + 2^-19 (1 + |lse|)
"""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Inputs of one call: a paged cache with shuffled blocks, queries as a slice of a projection.  Slots that no
    request sees hold NaN codes and NaN scales."""

    def __init__(self, lens, hq=8, hk=2, d=128, bs=16, window=0, order="head", seed=0, qscale=1.0, scale=None,
                 k_exp=(0, 0), v_exp=(0, 0), spare=3, pad=0, zero_rows=0.0):
        rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        self.hq, self.hk, self.d, self.bs, self.window = hq, hk, d, bs, window
        B = len(lens)
        held = -(-np.maximum(self.lens, 0) // bs)
        self.blocks = int(held.sum()) + spare
        ids = rng.permutation(self.blocks).astype(np.int32)
        self.table = np.full((B, max(1, int(held.max()))), self.blocks - 1, np.int32)
        shape = (self.blocks, hk, bs)
        codes = [rng.integers(0, 256, (*shape, d)).astype(np.uint8) for _ in range(2)]
        for i, c in enumerate(codes):
            c[(c & 127) == 127] = 0
            # most codes of ordinary size, as the codes of normal rows are
            c[:] = np.where(rng.random(c.shape) < 0.9, (c & 0x8F) | 0x60, c)
        sc = [rng.integers(127 - 8 + lo, 127 - 8 + hi + 1, shape).astype(np.uint8) for lo, hi in (k_exp, v_exp)]
        if zero_rows:
            zero = rng.random(shape) < zero_rows
            codes[1][zero], sc[1][zero] = 0, 0
        seen = np.zeros(shape, bool)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = ids[at:at + h]
            at += h
            n = int(self.lens[b])
            p = np.arange(max(0, n - window) if window else 0, max(0, n))
            seen[self.table[b][p // bs], :, p % bs] = True
        for c, s in zip(codes, sc):
            c[~seen], s[~seen] = 0x7F, 255
        self.codes, self.sc = codes, sc
        full = (self.blocks, hk, bs, d + pad) if order == "head" else (self.blocks, bs, hk, d + pad)
        self.k, self.v = (torch.full(full, 0x7F, dtype=torch.uint8, device="cuda")[..., :d] for _ in range(2))
        if order != "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.k.copy_(dev(codes[0]))
        self.v.copy_(dev(codes[1]))
        self.ks, self.vs = dev(sc[0]), dev(sc[1])
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = (torch.randn(B, hq * d + 24, device="cuda", generator=g) * qscale).bfloat16()
        self.q = w[:, 8:8 + hq * d].unflatten(1, (hq, d))
        self.scale = float(scale if scale is not None else d ** -0.5)

    def args(self, lm, **kw):
        cache = lm.kv_cache_fp8_of(self.k, self.v, self.ks, self.vs)
        a = dict(n_requests=len(self.lens), q_heads=self.hq, max_blocks=self.table.shape[1], scale=self.scale,
                 window=self.window)
        dims = lm.decode_dims_of(**(a | kw))
        ws = torch.full((lm.lmoe_decode_attention_fp8_workspace_bytes(dims, cache),), 255, dtype=torch.uint8,
                        device="cuda")
        self.kept = (dev(self.lens), dev(self.table), ws)
        return dims, cache, self.q, *self.kept[:2]

    def run(self, lm, want=0, lse=True, stream=None, **kw):
        args = self.args(lm, **kw)
        out = torch.full(self.q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full(self.q.shape[:2], 9.0, device="cuda") if lse else None
        lm.lmoe_decode_attention_fp8(*args, out, ls, self.kept[2], stream=stream)
        assert lm.lmoe_status_check(self.kept[2], stream) == want
        return out, ls

    def ref(self):
        k, v = (fp8_ref.values(c, s) for c, s in zip(self.codes, self.sc))
        q = self.q.float().cpu().numpy().astype(np.float64)
        return fp8_ref.decode(q, k, v, None, self.lens, self.table, self.window, self.scale,
                              fp8_ref.scale_values(self.sc[1]))

    def check(self, lm, got=None, **kw):
        out, ls = got or self.run(lm, **kw)
        with np.errstate(invalid="ignore"):
            ref, lse, mass, dot, low = self.ref()
        got = out.float().cpu().numpy().astype(np.float64)
        S = dot[..., None]
        e = (self.d + 16) * 2.0**-23 * S + 2.0**-20
        n = np.minimum(self.lens, self.window) if self.window else self.lens
        sums = (np.maximum(n, 0) / 16 + 40)[:, None, None] * 2.0**-23
        tol = 2.0**-8 * np.abs(ref) + (2.0**-11 + 2.0**-17 + 2.0**-23 * S + sums + 2 * e) * mass + 2.0**-39 * low + 2.0**-133
        tol *= 1 + 2.0**-6  # what is of second order
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
        empty = np.isneginf(lse)
        assert (got[empty] == 0).all()
        if ls is not None:
            gl = ls.cpu().numpy().astype(np.float64)
            assert np.array_equal(np.isneginf(gl), empty)
            with np.errstate(invalid="ignore"):
                bad = ~(np.abs(gl - lse) <= e[..., 0] + 2.0**-19 * (1 + np.abs(lse))) & ~empty
            assert not bad.any(), (np.argwhere(bad)[:5], gl[bad][:5], lse[bad][:5])
        return out, ls


LENGTHS = [[0], [1], [15], [16], [17], [31], [32], [33], [255], [256], [257], [1000], [5001], [0, 1, 130, 0, 513, 0]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENGTHS, ids=["-".join(map(str, x)) for x in LENGTHS])
def test_lengths(lm, lens, d):
    Case(lens, d=d, seed=len(lens) + lens[0]).check(lm)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 8), (6, 2), (21, 7), (40, 8), (64, 8), (9, 1), (32, 2), (17, 1),
                                   (46, 2), (128, 1), (20, 4)])
def test_heads(lm, hq, hk, d):
    Case([300, 77, 1], hq=hq, hk=hk, d=d, seed=hq).check(lm)


@pytest.mark.parametrize("order,pad", [("head", 0), ("slot", 0), ("head", 16), ("slot", 48)])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_layouts(lm, bs, order, pad):
    for d in (64, 128):
        Case([3 * bs, 5 * bs - 1, 17, 2 * bs + 1], d=d, bs=bs, order=order, pad=pad, seed=bs + d).check(lm)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 1000, 4096, 2**31 - 1])
def test_windows(lm, window):
    for d in (64, 128):
        Case([1, 31, 32, 64, 1000, 1031, 2500], d=d, hq=6, hk=2, window=window, seed=window % 97).check(lm)


@pytest.mark.parametrize("lens,hq,hk,d", [([70000], 8, 1, 128), ([33333], 16, 1, 64), ([40, 20000, 3, 9000], 16, 2, 128),
                                          ([20] * 700, 5, 1, 64), ([1, 40, 0] * 300, 4, 2, 128),
                                          (list(range(400)), 8, 1, 128)],
                         ids=["one", "one_16", "long_and_short", "many_short", "many_empty", "ragged"])
def test_splits(lm, lens, hq, hk, d):
    Case(lens, hq=hq, hk=hk, d=d, bs=32, seed=3).check(lm)


def test_most_requests(lm):
    lens = np.random.default_rng(0).integers(0, 3, 8192)
    Case(lens.tolist(), hq=2, hk=1, d=64, seed=8).check(lm)


@pytest.mark.parametrize("qscale,scale", [(2.0**-100, 2.0**97), (2.0**60, 2.0**-63), (8.0, None), (30.0, None),
                                          (1e-30, None), (0.0, None)])
def test_score_sizes(lm, qscale, scale):
    for d in (64, 128):
        Case([400, 33], d=d, qscale=qscale, scale=scale, seed=4).check(lm)


@pytest.mark.parametrize("k_exp,v_exp,zero", [((-3, 3), (-3, 3), 0.0), ((0, 0), (-60, 60), 0.2), ((0, 0), (-110, -100), 0.1),
                                              ((-100, -90), (100, 105), 0.0), ((0, 0), (0, 0), 1.0), ((0, 0), (-2, 2), 0.5)])
def test_scales_of_any_size(lm, k_exp, v_exp, zero):
    """Values whose scales differ by up to 2^120 within a row, and rows of zeros (whose scale byte is 0)."""
    for d in (64, 128):
        Case([700, 31, 1], d=d, k_exp=k_exp, v_exp=v_exp, zero_rows=zero, seed=6).check(lm)


@pytest.mark.parametrize("size", [1e3, 1e5, 1e9, 1e30])
def test_far_scores(lm, size):
    """However large the scores are, a row with one position in sight gets that position's value, and one whose first
    position's score lies far above the others gets the first's."""
    for d in (64, 128):
        c = Case([1, 40, 300], hq=8, hk=2, d=d, window=1, v_exp=(-9, 9), seed=7, qscale=size)
        out, _ = c.run(lm)
        v = fp8_ref.values(c.codes[1], c.sc[1])
        c2 = Case([200], hq=8, hk=2, d=d, v_exp=(-9, 9), seed=8)
        c2.codes[0][np.isin(c2.sc[0], 255, invert=True)] = 0
        c2.codes[0][c2.table[0][0], :, 0] = 0x38  # ones; the other keys are zero
        c2.sc[0][c2.table[0][0], :, 0] = 127
        c2.k.copy_(dev(c2.codes[0]))
        c2.ks.copy_(dev(c2.sc[0]))
        c2.q.fill_(size)
        out2, _ = c2.run(lm)
        want2 = fp8_ref.values(c2.codes[1], c2.sc[1])[c2.table[0][0], :, 0]
        pairs = [(out2[0], want2)]
        for b, n in enumerate((1, 40, 300)):
            pairs.append((out[b], v[c.table[b][(n - 1) // c.bs], :, (n - 1) % c.bs]))
        for got, want in pairs:
            got = got.float().cpu().numpy().astype(np.float64).reshape(2, 4, d)
            # exact products and a power of two: only the quotient by the sum, 1, is off
            assert np.abs(got - want[:, None]).max() <= 2.0**-8 * np.abs(want).max()
            assert (np.abs(got - want[:, None]) <= 2.0**-8 * np.abs(want[:, None])).all()


def test_a_key_that_holds_all_with_small_values(lm):
    # the largest score has the smallest values: they must come through at full precision
    c = Case([64], hq=1, hk=1, d=128, seed=9)
    c.codes[0][:] = np.where(np.isin(c.sc[0], 255)[..., None], c.codes[0], 0)
    blk = c.table[0][1]
    c.codes[0][blk, 0, 3] = 0x38  # ones
    c.sc[0][blk, 0, 3] = 127
    c.q.fill_(40.0)  # score 40 * 128 / sqrt(128) = 452 for it, 0 for the others
    c.sc[1][blk, 0, 3] -= 60
    c.k.copy_(dev(c.codes[0]))
    c.ks.copy_(dev(c.sc[0]))
    c.vs.copy_(dev(c.sc[1]))
    c.check(lm)


def test_nan_rows_reach_only_who_sees_them(lm):
    c = Case([40, 40], hq=8, hk=2, d=128, seed=10)
    c.ks[int(c.table[0, 1]), 1, 5] = 255   # request 0, kv head 1
    c.vs[int(c.table[1, 2]), 0, 1] = 255   # request 1, kv head 0
    out, ls = c.run(lm)
    nan = torch.isnan(out.float()).all(dim=2).cpu().numpy()
    assert np.array_equal(nan, [[False] * 4 + [True] * 4, [True] * 4 + [False] * 4])
    assert np.array_equal(nan, torch.isnan(out.float()).any(dim=2).cpu().numpy())
    assert torch.isnan(ls[0, 4:]).all() and torch.isfinite(ls[0, :4]).all() and torch.isfinite(ls[1]).all()


def test_without_lse_and_twice_the_same(lm):
    c = Case([5000, 17, 900], hq=16, hk=2, seed=11)
    a, ls = c.check(lm)
    b, _ = c.run(lm, lse=False)
    again, ls2 = c.run(lm)
    assert torch.equal(a, b) and torch.equal(a, again) and torch.equal(ls, ls2)


def test_reports_what_is_out_of_range(lm):
    c = Case([40, 50, 60], hq=4, hk=2, seed=12)
    ref, _ = c.run(lm)
    # lengths below 0 and past the table: those rows stay as they were, the others are right
    c.lens[1] = -1
    out, ls = c.run(lm, want=-5)
    assert (out[1] == 9).all() and (ls[1] == 9).all() and torch.equal(out[::2], ref[::2])
    c.lens[1] = c.table.shape[1] * c.bs + 1
    out, ls = c.run(lm, want=-5)
    assert (out[1] == 9).all() and (ls[1] == 9).all() and torch.equal(out[::2], ref[::2])
    c.lens[1] = 2**31 - 1
    out, _ = c.run(lm, want=-5)
    assert (out[1] == 9).all() and torch.equal(out[::2], ref[::2])
    # blocks outside the cache
    c.lens[1] = 50
    for block in (-1, c.blocks, 2**31 - 1, -2**31):
        old, c.table[1, 2] = c.table[1, 2], block
        out, _ = c.run(lm, want=-5)
        assert torch.equal(out[::2], ref[::2])
        c.table[1, 2] = old
    # a block number that no position in sight needs is not looked at
    c.table[0, 3:] = -7
    out, _ = c.run(lm)
    assert torch.equal(out, ref)


def test_a_full_table(lm):
    # the last page ends with the table's row, and the last tile inside it
    for bs in (16, 32, 64):
        Case([5 * bs, 3 * bs], bs=bs, seed=bs).check(lm)


def test_offsets_past_32_bits(lm):
    # the last blocks of a cache of more than 2^32 bytes a tensor
    blocks, hk, bs, d = 68000, 8, 64, 128
    k, v = (torch.empty(blocks, hk, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(blocks, hk, bs, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Case([100], hq=16, hk=hk, d=d, bs=bs, seed=13, spare=0)
    n = c.blocks
    for big, small in ((k, c.k), (v, c.v), (ks, c.ks), (vs, c.vs)):
        big[-n:] = small
    c.table += blocks - n
    c.k, c.v, c.ks, c.vs = k, v, ks, vs
    got = c.run(lm)
    c.table -= blocks - n
    c.check(lm, got=got)


def test_streams_and_graphs(lm):
    a, b = Case([900, 5, 2000], hq=16, hk=2, seed=14), Case([3000, 64], hq=8, hk=2, d=64, seed=15)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = a.run(lm)
    s.synchronize()
    a.check(lm, got=got)
    # two calls that share a workspace, one behind the other in a graph, replayed with other inputs
    args = [x.args(lm) for x in (a, b)]
    ws = max((x.kept[2] for x in (a, b)), key=lambda t: t.numel())
    outs = [(torch.zeros_like(x.q.contiguous()), torch.zeros(x.q.shape[:2], device="cuda")) for x in (a, b)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for x, o in zip(args, outs):
            lm.lmoe_decode_attention_fp8(*x, *o, ws)
    for turn in range(3):
        for x, o in zip((a, b), outs):
            x.q.copy_(torch.randn(x.q.shape, device="cuda").bfloat16())
            for y in o:
                y.fill_(7.0)
        if turn == 2:  # other lengths
            a.lens[:] = [0, 4, 1999]
            a.kept[0].copy_(dev(a.lens))
        g.replay()
        assert lm.lmoe_status_check(ws) == 0
        for x, o in zip((a, b), outs):
            x.check(lm, got=o)


def test_binding_refuses(lm):
    c = Case([40], hq=4, hk=2)
    dims, cache, q, lens, table = c.args(lm)
    out, ws = torch.empty_like(q.contiguous()), c.kept[2]
    with pytest.raises(lm.LmoeError) as e:
        lm.lmoe_decode_attention_fp8(dims, cache, q, lens, table, out, None, ws[:256])
    assert e.value.code == -6
    with pytest.raises(TypeError):
        lm.lmoe_decode_attention_fp8(dims, cache, q.float(), lens, table, out, None, ws)
    with pytest.raises(TypeError):
        lm.lmoe_decode_attention_fp8(dims, cache, q, lens.long(), table, out, None, ws)
    with pytest.raises(ValueError):
        lm.lmoe_decode_attention_fp8(dims, cache, q, lens, table, out[:, :2], None, ws)
    with pytest.raises(ValueError):
        lm.kv_cache_fp8_of(c.k, c.v, c.ks, c.vs[:-1])
    with pytest.raises(TypeError):
        lm.kv_cache_fp8_of(c.k.float(), c.v.float(), c.ks, c.vs)
