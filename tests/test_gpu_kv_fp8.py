"""Writes to and reads from the 8-bit cache against plain loops: codes, scales and values have one right answer, so
everything has to be equal."""
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


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def status_ws():
    return torch.full((256,), 255, dtype=torch.uint8, device="cuda")


def caches(blocks, hk, bs, d, order="head", fill=3):
    shape = (blocks, hk, bs, d) if order == "head" else (blocks, bs, hk, d)
    c = [torch.full(shape, fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    c = c if order == "head" else [x.transpose(1, 2) for x in c]
    return (*c, *(torch.full((blocks, hk, bs), fill, dtype=torch.uint8, device="cuda") for _ in range(2)))


@pytest.mark.parametrize("order", ["head", "slot"])
@pytest.mark.parametrize("n,hk,bs,d,gather,pad", [(1, 8, 16, 128, False, 0), (3, 1, 16, 64, True, 8),
                                                  (211, 3, 32, 64, True, 64), (100, 8, 64, 128, False, 1040),
                                                  (77, 5, 256, 128, True, 0), (259, 2, 128, 64, False, 24),
                                                  (1025, 1, 16, 64, True, 0)])
def test_write(lm, n, hk, bs, d, gather, pad, order):
    g = torch.Generator(device="cuda").manual_seed(n)
    rng = np.random.default_rng(n)
    blocks, rows = n // bs + 4, n + (n // 2 if gather else 0)
    wide = torch.randn(rows, 2 * hk * d + pad, device="cuda", generator=g)
    wide = (wide * torch.exp2(30 * torch.randn(rows, 1, device="cuda", generator=g))).bfloat16()
    kn, vn = (wide[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in range(2))
    slots = rng.permutation(blocks * bs)[:n].astype(np.int32)
    if n > 2:
        slots[rng.integers(n)] = -1
        slots[rng.integers(n)] = -5
    src = rng.integers(0, rows, n).astype(np.int32) if gather else np.arange(n, dtype=np.int32)
    cache = caches(blocks, hk, bs, d, order)
    expect = [x.clone().contiguous().cpu().numpy() for x in cache]
    for i, new in enumerate((kn, vn)):
        codes, scale = fp8_ref.quantise(host(new)[src])
        at = slots >= 0
        expect[i][slots[at] // bs, :, slots[at] % bs] = codes[at]
        expect[2 + i][slots[at] // bs, :, slots[at] % bs] = scale[at]
    ws = status_ws()
    lm.lmoe_kv_write_fp8(lm.kv_cache_fp8_of(*cache), kn, vn, dev(src) if gather else None, dev(slots), ws)
    assert lm.lmoe_status_check(ws) == 0
    for got, want in zip(cache, expect):
        assert np.array_equal(got.cpu().numpy(), want)


def test_write_every_size_of_value(lm):
    """Rows whose largest magnitude is each power of two's first, 448-like and next value, subnormals, zeros of both
    signs, ties between codes, infinities and NaN."""
    bits = np.arange(1 << 15, dtype=np.uint16)  # every magnitude
    hk, d, bs = 4, 64, 16
    rng = np.random.default_rng(1)
    rows = []
    for top in list(range(0, 0x7F80, 37)) + [0x7F7F, 0x7F80, 0x7F81, 0x7FC0, 1, 2, 0x43E0, 0x43E1, 0x43DF, 0x0080, 0x007F]:
        row = rng.integers(max(0, top - (12 << 7)), top + 1, d).astype(np.uint16)
        row[rng.integers(d)] = top
        row[rng.integers(d)] = 0
        rows.append(row | (rng.integers(0, 2, d).astype(np.uint16) << 15))
    # all magnitudes within a factor of 2^15 below 448: every tie there is
    near = bits[(bits >= 0x43E0 - (18 << 7)) & (bits < 0x43E0)]
    for i in range(0, len(near), d - 1):
        part = near[i:i + d - 1]
        rows.append(np.concatenate([part, np.zeros(d - 1 - len(part), np.uint16), [0x43E0]]).astype(np.uint16))
    while len(rows) % hk:
        rows.append(np.zeros(d, np.uint16))
    x = np.stack(rows).reshape(-1, hk, d)
    n = len(x)
    t = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    cache = caches(-(-n // bs), hk, bs, d)
    lm.lmoe_kv_write_fp8(lm.kv_cache_fp8_of(*cache), t, t.flip(0).contiguous(), None, dev(np.arange(n, dtype=np.int32)))
    with np.errstate(invalid="ignore"):
        codes, scale = fp8_ref.quantise(host(t))
    for i, turn in ((0, slice(None)), (1, slice(None, None, -1))):
        got = cache[i].transpose(1, 2).reshape(-1, hk, d)[:n].cpu().numpy()
        gs = cache[2 + i].transpose(1, 2).reshape(-1, hk)[:n].cpu().numpy()
        assert np.array_equal(gs, scale[turn])
        assert np.array_equal(got, codes[turn])


def test_write_passes_over_what_is_out_of_range(lm):
    cache = caches(2, 1, 16, 64, fill=0)
    kn = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    src = dev(np.array([0, 1, 4, -1, 2], np.int32))
    slots = dev(np.array([3, 32, 4, 5, 6], np.int32))
    ws = status_ws()
    lm.lmoe_kv_write_fp8(lm.kv_cache_fp8_of(*cache), kn, kn, src, slots, ws)
    assert lm.lmoe_status_check(ws) == -5
    lm.lmoe_kv_write_fp8(lm.kv_cache_fp8_of(*cache), kn, kn, src, slots)
    for c in cache[:2]:
        assert c[:, 0, :, 0].flatten().nonzero().flatten().tolist() == [3, 6]
    for c in cache[2:]:
        assert c.flatten().nonzero().flatten().tolist() == [3, 6]


class Read:
    def __init__(self, lens, firsts, hk=2, d=64, bs=16, order="head", pad=0, seed=0, gap=0):
        rng = np.random.default_rng(seed)
        self.hk, self.d, self.bs = hk, d, bs
        top = [a + b for a, b in zip(lens, firsts or [0] * len(lens))]
        held = [-(-x // bs) for x in top]
        self.blocks = sum(held) + 2
        ids = rng.permutation(self.blocks).astype(np.int32)
        self.table = np.full((len(lens), max(1, max(held))), -3, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = ids[at:at + h]
            at += h
        self.off = (gap + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
        self.first = None if firsts is None else np.array(firsts, np.int32)
        self.n = int(self.off[-1]) + gap
        self.cache = caches(self.blocks, hk, bs, d, order)
        for c in self.cache[:2]:
            c.copy_(dev(rng.integers(0, 256, (self.blocks, hk, bs, d)).astype(np.uint8)))
        for c in self.cache[2:]:
            c.copy_(dev(rng.integers(0, 256, (self.blocks, hk, bs)).astype(np.uint8)))
        wide = torch.full((max(1, self.n), 2 * hk * d + pad), 9.0, dtype=torch.bfloat16, device="cuda")
        self.out = [wide[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in range(2)]

    def run(self, lm, want=0):
        ws = status_ws()
        self.kept = (dev(self.off), None if self.first is None else dev(self.first), dev(self.table))
        lm.lmoe_kv_read_fp8(lm.kv_cache_fp8_of(*self.cache), *self.kept, *self.out, ws)
        assert lm.lmoe_status_check(ws) == want

    def expect(self, skip=()):
        res = []
        for c, s in zip(self.cache[:2], self.cache[2:]):
            with np.errstate(over="ignore"):
                val = torch.from_numpy(fp8_ref.values(c.cpu().numpy(), s.cpu().numpy())).float().bfloat16()
            e = torch.full((max(1, self.n), self.hk, self.d), 9.0).bfloat16()
            for b in range(len(self.off) - 1):
                f = 0 if self.first is None else int(self.first[b])
                for t in range(self.off[b], self.off[b + 1]):
                    p = f + t - self.off[b]
                    if (b, p // self.bs) not in skip:
                        e[t] = val[self.table[b, p // self.bs], :, p % self.bs]
            res.append(e)
        return res

    def check(self, lm, want=0, skip=()):
        self.run(lm, want)
        for got, e in zip(self.out, self.expect(skip)):
            got = got.cpu()
            nan = torch.isnan(e)
            assert torch.equal(torch.isnan(got), nan)
            assert torch.equal(got.masked_fill(nan, 0), e.masked_fill(nan, 0))


@pytest.mark.parametrize("order", ["head", "slot"])
@pytest.mark.parametrize("lens,firsts,hk,d,bs,pad,gap", [
    ([1], None, 1, 64, 16, 0, 0), ([0, 5, 0, 0, 40], None, 8, 128, 16, 64, 0), ([33, 1, 64], [5, 100, 0], 3, 64, 32, 8, 7),
    ([300], [12], 8, 128, 64, 0, 3), ([7] * 300, None, 1, 128, 16, 0, 0), ([100, 0, 257], [0, 0, 255], 5, 64, 256, 16, 1),
    ([3], [500], 256, 64, 128, 0, 0)])
def test_read(lm, lens, firsts, hk, d, bs, pad, gap, order):
    Read(lens, firsts, hk, d, bs, order, pad, seed=len(lens) + hk, gap=gap).check(lm)


def test_read_most_requests(lm):
    Read((np.arange(8192) % 3).tolist(), None, hk=1, d=64, seed=5).check(lm)


def test_read_reports_what_is_out_of_range(lm):
    r = Read([20, 40, 20], None, seed=6)
    r.table[1, 1] = r.blocks
    r.check(lm, want=-5, skip={(1, 1)})
    r = Read([20, 40, 20], None, seed=6)
    r.table[1, 1] = -1
    r.check(lm, want=-5, skip={(1, 1)})
    # positions below 0 and past the table
    r = Read([20, 40, 20], [0, 0, 0], seed=6)
    r.first[0], r.first[2] = -4, 2**31 - 8
    before = [o.clone() for o in r.out]
    r.run(lm, want=-5)
    for o, b in zip(r.out, before):
        assert torch.equal(o[:4], b[:4]) and torch.equal(o[60:], b[60:])
    # offsets that pass the rows or descend: nothing is written out of range, and it is reported
    r = Read([20, 40, 20], None, seed=6)
    r.off[3] = 81
    before = [o.clone() for o in r.out]
    r.run(lm, want=-5)
    for o, b in zip(r.out, before):
        assert torch.equal(o[60:], b[60:]) and not torch.equal(o[:60], b[:60])
    # ... also where no row shows it
    r = Read([20, 40, 20], None, seed=6)
    r.off[3] = 50
    before = [o.clone() for o in r.out]
    r.run(lm, want=-5)
    for o, b in zip(r.out, before):
        assert torch.equal(o[60:], b[60:]) and not torch.equal(o[:20], b[:20])
    r = Read([20, 40, 20], None, seed=6)
    r.off[0] = -3
    before = [o.clone() for o in r.out]
    r.run(lm, want=-5)
    for o, b in zip(r.out, before):
        assert torch.equal(o[:20], b[:20])


def test_what_was_written_reads_back(lm):
    """Values of four significant bits within 2^14 of their row's largest come back as they were."""
    hk, d, bs, n = 3, 128, 32, 150
    rng = np.random.default_rng(7)
    m = rng.integers(8, 16, (n, hk, d)) * np.exp2(rng.integers(-12, 1, (n, hk, d))) * rng.choice([-1, 1], (n, hk, d))
    x = torch.from_numpy(m * np.exp2(rng.integers(-60, 60, (n, hk, 1)))).bfloat16().cuda()
    cache = caches(8, hk, bs, d)
    c = lm.kv_cache_fp8_of(*cache)
    table = rng.permutation(8)[:5].astype(np.int32)
    p = np.arange(n)
    slots = dev((table[p // bs] * bs + p % bs).astype(np.int32))
    lm.lmoe_kv_write_fp8(c, x, -x, None, slots)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    lm.lmoe_kv_read_fp8(c, dev(np.array([0, n], np.int32)), None, dev(table[None]), ko, vo)
    assert torch.equal(ko, x) and torch.equal(vo, -x)
    # ... and, read and written again, gives the same codes
    again = caches(8, hk, bs, d)
    lm.lmoe_kv_write_fp8(lm.kv_cache_fp8_of(*again), ko, vo, None, slots)
    assert all(torch.equal(a, b) for a, b in zip(cache, again))


def test_offsets_past_32_bits(lm):
    blocks, hk, bs, d = 68000, 8, 64, 128
    cache = [torch.empty(blocks, hk, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.empty(blocks, hk, bs, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for c in cache:
        c[-1].zero_()
    x = torch.randn(2, hk, d, device="cuda").bfloat16()
    c = lm.kv_cache_fp8_of(*cache)
    lm.lmoe_kv_write_fp8(c, x, -x, None, dev(np.array([blocks * bs - 1, (blocks - 1) * bs], np.int32)))
    codes, scale = fp8_ref.quantise(host(x))
    assert np.array_equal(cache[0][-1][:, [-1, 0]].cpu().numpy(), codes.transpose(1, 0, 2))
    assert np.array_equal(cache[3][-1][:, [-1, 0]].cpu().numpy(), scale.T)
    assert int(cache[0][-1][:, 1:-1].sum()) == 0 and int(cache[2][-1][:, 1:-1].sum()) == 0
    ko, vo = (torch.zeros(bs, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lm.lmoe_kv_read_fp8(c, dev(np.array([0, bs], np.int32)), None, dev(np.array([[blocks - 1]], np.int32)), ko, vo)
    want = torch.from_numpy(fp8_ref.values(codes, scale)).bfloat16().cuda()
    assert torch.equal(ko[[-1, 0]], want) and torch.equal(vo[[-1, 0]], -want) and not ko[1:-1].any()


def test_streams_and_graphs(lm):
    hk, d, bs, n = 2, 64, 16, 50
    cache = caches(4, hk, bs, d)
    c = lm.kv_cache_fp8_of(*cache)
    x = torch.randn(n, hk, d, device="cuda").bfloat16()
    slots, table = dev(np.arange(n, dtype=np.int32)), dev(np.arange(4, dtype=np.int32)[None])
    off = dev(np.array([0, n], np.int32))
    ko, vo = torch.empty_like(x), torch.empty_like(x)

    def step():
        lm.lmoe_kv_write_fp8(c, x, x, None, slots)
        lm.lmoe_kv_read_fp8(c, off, None, table, ko, vo)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        x.copy_(torch.randn(n, hk, d, device="cuda").bfloat16())
        g.replay()
        torch.cuda.synchronize()
        want = torch.from_numpy(fp8_ref.values(*fp8_ref.quantise(host(x)))).bfloat16().cuda()
        assert torch.equal(ko, want) and torch.equal(vo, want)
