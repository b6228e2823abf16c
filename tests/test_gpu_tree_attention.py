"""Tree attention over the paged cache against plain 64-bit loops.

Bounds, from the arithmetic that include/lmoe.h states (u = 2^-9, half of bf16's
unit roundoff: the result's own rounding may take all of 2 u, so where a few keys
hold a row's weight P has to be finer than one bf16; A = sum_j p_j |v_j|;
S = max_j scale sum_d |q_d k_jd|):
  scores   products are exact in fp32, head_dim additions of at most 2^-23
           relative each (truncating accumulators), the scale and the change
           of base: |ds| <= (head_dim + 8) 2^-23 S + 2^-22 |s|; exponentials
           2^-21; so p is off by at most e = (head_dim + 16) 2^-23 S + 2^-20
           relative, before and after the division
  out      p rounded to bf16: u A; the result rounded to bf16: u |out| <= u A;
           fp32 sums over the keys: 2^-14 A;  in all (2 u + 2^-12 + 4 e) A,
           with a subnormal's worth of absolute slack
  lse      e + 2^-19 (1 + |lse|)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_ref

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
    """Inputs of one call: a paged cache with shuffled blocks, drafts as slices of one projection."""

    def __init__(self, lens, ns, hq=8, hk=2, d=64, bs=16, window=0, mask="tree", pos=True, order="head", seed=0,
                 qscale=1.0, spare=3, scale=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.ns = np.array(lens, np.int32), np.array(ns, np.int32)
        self.hq, self.hk, self.d, self.bs, self.window = hq, hk, d, bs, window
        self.off = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        T = max(1, int(self.off[-1]))
        held = -(-self.lens // bs)
        self.blocks = int(held.sum()) + spare
        ids = rng.permutation(self.blocks).astype(np.int32)
        self.table = np.full((len(lens), max(1, int(held.max()))), self.blocks - 1, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = ids[at:at + h]
            at += h
        shape = (self.blocks, hk, bs, d) if order == "head" else (self.blocks, bs, hk, d)
        self.k, self.v = (torch.randn(shape, device="cuda", generator=g).bfloat16() for _ in range(2))
        if order != "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        w = torch.randn(T, (hq + 2 * hk) * d + 16, device="cuda", generator=g)
        w[:, :hq * d] *= qscale
        w = w.bfloat16()
        self.q = w[:, :hq * d].unflatten(1, (hq, d))
        self.kn = w[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        self.vn = w[:, (hq + hk) * d:(hq + 2 * hk) * d].unflatten(1, (hk, d))
        self.words = max(1, (int(self.ns.max()) + 63) // 64)
        self.mask = self.pos = None
        par = np.concatenate([[int(rng.integers(-1, i)) if i else -1 for i in range(n)] for n in ns] or [[]])
        m, p = kv_ref.tree_masks(self.off, par.astype(int), self.lens, self.words)
        if mask == "tree":
            self.mask = m
        elif mask == "any":  # arbitrary bits, rows without their own among them
            self.mask = rng.integers(0, 1 << 63, (T, self.words)).astype(np.uint64) * 2 + 1
            self.mask &= rng.integers(0, 1 << 63, (T, self.words)).astype(np.uint64)
        elif mask == "none":
            self.mask = np.zeros((T, self.words), np.uint64)
        if pos:
            self.pos = p
        if not len(par):  # no drafts at all: one row that belongs to no request
            self.mask, self.pos = np.zeros((1, 1), np.uint64), np.zeros(1, np.int32)
        self.scale = float(scale if scale is not None else d ** -0.5)

    def dims(self, lm, **kw):
        a = dict(n_requests=len(self.lens), n_tokens=self.q.shape[0], max_request_tokens=max(1, int(self.ns.max())),
                 q_heads=self.hq, max_blocks=self.table.shape[1], mask_words=self.words, window=self.window,
                 scale=self.scale)
        return lm.attn_dims_of(**(a | kw))

    def run(self, lm, want=0, ws=None, stream=None, lse=True, **kw):
        cache, dims = lm.kv_cache_of(self.k, self.v), self.dims(lm, **kw)
        out = torch.full(self.q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full(self.q.shape[:2], 9.0, device="cuda") if lse else None
        if ws is None:
            ws = torch.full((lm.lmoe_tree_attention_workspace_bytes(dims, cache),), 255, dtype=torch.uint8,
                            device="cuda")
        # the caller's arrays on the device, kept until the status has been read
        self.kept = (dev(self.off), dev(self.lens), dev(self.table),
                     None if self.mask is None else dev(self.mask.view(np.int64)),
                     None if self.pos is None else dev(self.pos))
        off, lens, table, mask, pos = self.kept
        lm.lmoe_tree_attention(dims, cache, self.q, self.kn, self.vn, off, lens, table, mask, pos, out, ls, ws,
                               stream=stream)
        assert lm.lmoe_status_check(ws, stream) == want
        return out, ls

    def ref(self):
        f = [x.float().cpu().numpy().astype(np.float64) for x in (self.q, self.kn, self.vn, self.k, self.v)]
        return kv_ref.attention(*f, self.off, self.lens, self.table, self.mask, self.pos, self.window, self.scale)

    def check(self, lm, **kw):
        out, ls = self.run(lm, **kw)
        with np.errstate(invalid="ignore"):
            ref, lse, mass, dot = self.ref()
        n = int(self.off[-1])
        got = out.float().cpu().numpy().astype(np.float64)[:n]
        ref, lse, mass, dot = ref[:n], lse[:n], mass[:n], dot[:n]
        e = (self.d + 16) * 2.0**-23 * dot + 2.0**-20
        tol = (2.0**-8 + 2.0**-12 + 4 * e[..., None]) * mass + 2.0**-133
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
        empty = np.isneginf(lse)
        assert (got[empty] == 0).all()
        if ls is not None:
            gl = ls.cpu().numpy().astype(np.float64)[:n]
            assert np.array_equal(np.isneginf(gl), empty)
            with np.errstate(invalid="ignore"):
                bad = ~(np.abs(gl - lse) <= e + 2.0**-19 * (1 + np.abs(lse))) & ~empty
            assert not bad.any(), (np.argwhere(bad)[:5], gl[bad][:5], lse[bad][:5])
        return out


LENGTHS = [[0], [1], [15], [16], [17], [127], [128], [129], [255], [256], [257], [1000], [3001], [0, 1, 130, 513]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENGTHS, ids=["-".join(map(str, x)) for x in LENGTHS])
def test_prefix_lengths(lm, lens, d):
    Case(lens, [3] * len(lens), d=d, seed=len(lens) + lens[0]).check(lm)
    Case(lens, [1] * len(lens), d=d, seed=1, mask=None, pos=False).check(lm)


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (3, 1), (8, 8), (24, 8), (40, 8), (7, 1), (64, 8), (128, 1)])
@pytest.mark.parametrize("n", [1, 5])
def test_head_layouts(lm, hq, hk, n):
    Case([77, 300], [n, n], hq=hq, hk=hk, d=128, seed=hq).check(lm)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 192, 200, 255, 256])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (8, 1, 128)])
def test_tree_sizes(lm, n, hq, hk, d):
    Case([150, 0], [n, max(0, n - 3)], hq=hq, hk=hk, d=d, seed=n).check(lm)


@pytest.mark.parametrize("rows", [31, 32, 33, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 70])
def test_rows_at_the_kernels_bounds(lm, rows, d, window):
    """One query head a key head: a request's rows are its drafts.  Long, short and empty prefixes, ends in tiles."""
    Case([700, 129, 0, 63], [rows, max(1, rows - 31), rows // 2, 1], hq=2, hk=2, d=d, window=window, seed=rows).check(lm)


@pytest.mark.parametrize("order", ["head", "slot"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_block_sizes_and_orders(lm, bs, order, d):
    Case([bs - 1, 2 * bs, 5 * bs + 3, 700], [4, 1, 3, 8], d=d, bs=bs, order=order, seed=bs).check(lm)


@pytest.mark.parametrize("window", [1, 2, 5, 16, 100, 128, 129, 333, 5000])
@pytest.mark.parametrize("pos,mask", [(True, "tree"), (False, None), (False, "any")])
def test_windows(lm, window, pos, mask):
    Case([0, 3, 127, 128, 400, 1111], [5, 9, 3, 8, 20, 33], window=window, pos=pos, mask=mask, seed=window).check(lm)


def test_positions_below_the_prefix_count_as_its_end(lm):
    c = Case([200, 40], [6, 6], window=30, seed=2)
    c.pos = c.pos - np.int32(100)
    c.check(lm)


@pytest.mark.parametrize("far", [3, 1000, 2**31 - 1])
def test_positions_past_any_tree_count_as_its_deepest_place(lm, far):
    c = Case([200, 40, 3], [6, 6, 9], window=30, seed=2)
    c.pos[::3] = np.minimum(c.pos[::3].astype(np.int64) + far, 2**31 - 1).astype(np.int32)
    c.check(lm)


@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 200])
def test_windows_as_wide_as_there_can_be(lm, window):
    Case([300, 0, 128], [5, 3, 70], window=window, seed=61).check(lm)


@pytest.mark.parametrize("mask", ["any", "none"])
def test_masks_that_leave_rows_empty(lm, mask):
    # no prefix and no visible draft: zeros and an lse of -infinity, next to rows that do see something
    Case([0, 0, 5, 0], [7, 1, 3, 130], mask=mask, seed=3).check(lm)
    Case([0, 40], [9, 9], mask=mask, window=4, seed=4).check(lm)


def test_requests_without_drafts(lm):
    Case([10, 500, 0, 70], [0, 3, 0, 0], seed=5).check(lm)
    Case([10, 20], [0, 0], seed=5).check(lm)


@pytest.mark.parametrize("qscale", [0.0, 1e-30, 40.0, 1e4, 1e30])
def test_score_ranges(lm, qscale):
    # from all-equal scores to a softmax that is one key, in tiles far apart
    Case([900, 130], [5, 2], qscale=qscale, d=128, seed=7).check(lm)


def one_hot_case(power, order, ties, d, n=3, length=700, heads=4, seed=67):
    """Scores that are whole numbers up to 255 times 2^power, exact in fp32 (one product of two powers of two and a
    small integer each, the rest zero), so that a row's softmax is the mean of the keys that tie for the largest
    (or, for queries of the other sign, the smallest) number.  `order`: where the numbers rise, along the keys of the
    prefix and then of the drafts; `ties`: how many keys share the first place."""
    c = Case([length], [n], hq=heads, hk=1, d=d, seed=seed, mask="none", scale=2.0**-4)
    c.mask |= np.uint64(1)  # every row sees the prefix and draft 0
    rng = np.random.default_rng(seed)
    total = length + 1
    num = np.sort(rng.integers(20, 230, total))
    num = {"rising": num, "falling": num[::-1], "mixed": rng.permutation(num)}[order].copy()
    first, last = rng.permutation(total)[:ties], rng.permutation(total)[:ties]
    num[first] = 255
    num[np.setdiff1d(last, first)[:ties]] = 1
    last = np.flatnonzero(num == 1)
    v = rng.integers(1, 100, (total, d)) * rng.choice([-1, 1], (total, d))
    # |score| = num * 2^power, split over q, k and the scale of 2^-4
    hi = power // 2 + 4
    q = torch.zeros(n, heads, d)
    q[:, :, 5] = 2.0**hi
    q[:, 1::2, 5] = -2.0**hi
    k = torch.zeros(total, d)
    k[:, 5] = torch.from_numpy(num.astype(np.float32)) * 2.0**(power - hi + 4)
    c.q.copy_(q)
    c.kn.zero_()
    c.vn.zero_()
    at = torch.arange(length, device="cuda")
    blk = dev(c.table[0]).long()[at // c.bs]
    c.k[blk, 0, at % c.bs] = k[:length].bfloat16().cuda()
    c.v[blk, 0, at % c.bs] = torch.from_numpy(v[:length].astype(np.float32)).bfloat16().cuda()
    c.kn[0, 0] = k[length].bfloat16().cuda()
    c.vn[0, 0] = torch.from_numpy(v[length].astype(np.float32)).bfloat16().cuda()
    out, lse = np.zeros((n, heads, d)), np.zeros((n, heads))
    for h in range(heads):
        win = last if h % 2 else first
        out[:, h] = v[win].mean(axis=0)
        lse[:, h] = (-1 if h % 2 else 255) * 2.0**power + np.log(len(win))
    return c, out, lse


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("power,ties,d", [(8, 1, 64), (14, 2, 128), (15, 1, 64), (16, 4, 64), (17, 1, 128), (20, 3, 64),
                                          (40, 2, 128), (80, 1, 64), (110, 4, 64)])
def test_the_largest_score_takes_all(lm, power, ties, d, order):
    """Scores of 2^8 to 2^118 whose largest stand at least 2^power above the rest (a factor of 1.1: far more than
    fp32's rounding of them).  The weights are exact, so out is the mean of the winners' values with the roundings of
    1 / ties (2 units of 2^-23), the product with it (2^-24) and bf16 (2^-8 with its neighbourhood); lse has the
    roundings of scale * log2(e), the product with it, ln(2), the product with that, and a sum: 2^-21 |lse| + 2^-19."""
    c, out, lse = one_hot_case(power, order, ties, d)
    got, ls = c.run(lm)
    got, ls = got.float().cpu().numpy().astype(np.float64), ls.cpu().numpy().astype(np.float64)
    assert (np.abs(got - out) <= (2.0**-8 + 2.0**-20) * np.abs(out) + 2.0**-20).all(), np.abs(got - out).max()
    assert (np.abs(ls - lse) <= 2.0**-21 * np.abs(lse) + 2.0**-19).all()


@pytest.mark.parametrize("d,group,n", [(64, 1, 1), (128, 1, 2), (128, 16, 3), (64, 40, 2), (128, 16, 10)])
def test_probabilities_that_round_badly(lm, d, group, n):
    """Keys of one weight that lies just above halfway between two bf16 numbers and is rounded down, all with the same
    value, behind a first tile of heavier keys: every probability's rounding (2^-8 of it at most) goes the same way.
    With the result's own rounding (2^-8) the bound is (2^-7 + 2^-12 + 4 e) A, where A is what they weigh.  Enough
    requests that a CTA works through whole ones (a cut starts anew, with a second bf16 part of its probabilities)."""
    B, hk, bs = 40, 8, 64
    c = Case([640] * B, [n] * B, hq=hk * group, hk=hk, d=d, bs=bs, mask="none", seed=71, scale=1.0, spare=0)
    parts, rest = [], np.log(0.5 + 2.0**-9) - 1e-5
    for _ in range(3):
        parts.append(float(torch.tensor(rest).bfloat16()))
        rest -= parts[-1]
    c.q.zero_()
    c.q[:, :, :3] = 1.0
    c.k.zero_()
    c.v.zero_()
    late = dev(c.table)[:, 128 // bs:].long().flatten()
    c.k[late, :, :, :3] = torch.tensor(parts).bfloat16().cuda()
    c.v[late] = (1 + torch.arange(d) / 128.0).bfloat16().cuda()
    out, _ = c.run(lm)
    got = out.float().cpu().numpy().astype(np.float64)
    w = np.exp(sum(parts))
    share = 512 * w / (128 + 512 * w)
    ref = share * (1 + np.arange(d) / 128.0)  # = A: the values are positive
    e = (d + 16) * 2.0**-23 * 1.0 + 2.0**-20  # (products of 1 and the parts: below 1 in all)
    off = np.abs(got - ref) / ref
    assert (off <= 2.0**-7 + 2.0**-12 + 4 * e).all(), off.max()


def test_rising_and_falling_maxima(lm):
    # the running maximum moves in every tile (rising), or only in the first (falling)
    for sign in (1.0, -1.0):
        c = Case([1500], [4], d=64, hk=1, hq=4, seed=8)
        ramp = torch.linspace(-30 * sign, 30 * sign, 1500, device="cuda")
        at = torch.arange(1500, device="cuda")
        blk = dev(c.table[0]).long()[at // 16]
        c.q.copy_(torch.full_like(c.q, 1.0))
        c.k[blk, 0, at % 16] = (ramp[:, None] / 8).expand(1500, 64).bfloat16()
        c.check(lm)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("d", [64, 128])
def test_poison_in_unseen_places(lm, poison, window, d):
    """Stale slots, foreign blocks, cached keys behind the window, other requests' drafts and
    unseen drafts of the own request hold NaN or infinities; the reference skips them."""
    lens, ns = [37, 300, 0, 128], [6, 3, 5, 9]
    c = Case(lens, ns, window=window, seed=11, d=d)
    used = torch.zeros(c.blocks, c.bs, dtype=torch.bool)
    for b, ln in enumerate(lens):
        lo = max(0, ln - window + 1) if window else 0
        for p in range(lo, ln):
            used[c.table[b, p // c.bs], p % c.bs] = True
    hide = (~used).cuda()[:, None, :, None]
    c.k.masked_fill_(hide, poison)
    c.v.masked_fill_(hide, poison)
    # one branch of each tree is poisoned: its rows see it, the others must not
    for b, n in enumerate(ns):
        c.kn[int(c.off[b]) + n - 1] = poison
        c.vn[int(c.off[b]) + n - 1, :, 3] = poison
    out, ls = c.run(lm)
    with np.errstate(invalid="ignore"):
        ref, lse, mass, dot = c.ref()
    sick = np.zeros(len(ref), bool)
    for b, n in enumerate(ns):
        for i in range(n):
            bits = int(c.mask[c.off[b] + i, 0])
            sick[c.off[b] + i] = bits >> (n - 1) & 1
    assert sick.sum() >= len(ns) and not sick.all()
    got = out.float().cpu().numpy().astype(np.float64)
    e = (c.d + 16) * 2.0**-23 * dot + 2.0**-20
    tol = (2.0**-8 + 2.0**-12 + 4 * e[..., None]) * mass + 2.0**-133
    assert (np.abs(got - ref) <= tol)[~sick].all()
    assert np.isfinite(ls.cpu().numpy()[~sick]).all()


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["draft", "window"])
def test_poisoned_values_reach_only_the_rows_that_see_them(lm, poison, where):
    """A value of a draft (or of a cached position inside some rows' window) that is not finite
    makes that element of the rows that see it not finite, and of no other row."""
    c = Case([300], [8], hq=16, hk=2, d=128, window=40 if where == "window" else 0, seed=13)
    c.mask = np.array([[(1 << i) | 1] for i in range(8)], np.uint64)  # eight leaves of one root
    c.pos = np.array([300, 301, 302, 303, 304, 305, 306, 307], np.int32)
    if where == "draft":
        c.vn[5, 1, 77] = poison
        sees = np.arange(8) == 5
    else:
        p = 300 - 40 + 4  # in sight of positions up to 303
        c.v[int(c.table[0, p // 16]), 1, p % 16, 77] = poison
        sees = np.arange(8) <= 3
    out, ls = c.run(lm)
    got = out.float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref, lse, mass, dot = c.ref()
    hit = np.zeros(got.shape, bool)
    hit[sees, 8:, 77] = True
    assert not np.isfinite(got[hit]).any()
    assert np.array_equal(np.isnan(got[hit]), np.isnan(ref[hit]))
    e = (c.d + 16) * 2.0**-23 * dot + 2.0**-20
    with np.errstate(invalid="ignore"):
        ok = np.abs(got - ref) <= (2.0**-8 + 2.0**-12 + 4 * e[..., None]) * mass + 2.0**-133
    assert ok[~hit].all()
    assert np.isfinite(ls.cpu().numpy()).all()


def test_many_requests_and_repeatability(lm):
    rng = np.random.default_rng(17)
    c = Case(rng.integers(0, 700, 60), rng.integers(0, 12, 60), hq=16, hk=4, seed=17)
    a = c.check(lm)
    b, _ = c.run(lm)
    assert torch.equal(a, b)
    # the order of the requests does not matter to the bits of a one-request call... only to its split:
    # a second call without an lse gives the same output
    d, _ = c.run(lm, lse=False)
    assert torch.equal(a, d)


@pytest.mark.parametrize("n,d", [(8, 128), (8, 64), (30, 128), (30, 64)])
def test_many_tiles_in_a_row(lm, n, d):
    # long enough that every part of the split walks many tiles and several heads; the same bits each time
    c = Case([20000, 311], [n, 3], hq=64, hk=8, d=d, bs=32, seed=31)
    ref = c.check(lm)
    for _ in range(10):
        assert torch.equal(c.run(lm)[0], ref)


@pytest.mark.parametrize("d", [64, 128])
def test_segments_of_one_and_two_row_tiles_in_a_row(lm, d):
    # more than 128 rows a key head: at a segment's end both groups, or one of them, fetch the next one's queries
    # if its record is there by then, and else later: the same bits either way
    rng = np.random.default_rng(41)
    c = Case(rng.integers(0, 900, 24), rng.integers(9, 48, 24), hq=16, hk=2, d=d, seed=41)
    ref = c.check(lm)
    for _ in range(20):
        assert torch.equal(c.run(lm)[0], ref)


def test_offsets_past_32_bits(lm):
    c = Case([200], [4], hq=16, hk=8, d=128, bs=64, seed=19)
    blocks = 36000  # more than 2^31 elements and 2^32 bytes per tensor
    big = [torch.empty(blocks, 8, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    new = np.array([[blocks - 1, blocks - 7, 3, blocks - 2]], np.int32)
    for x, y in zip(big, (c.k, c.v)):
        for o, n in zip(c.table[0], new[0]):
            x[int(n)] = y[int(o)]
    ref = c.check(lm)
    c.k, c.v, c.table = big[0], big[1], new
    out, _ = c.run(lm)
    assert torch.equal(out, ref)


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("n,window,below", [(9, 40, 3), (60, 40, 3), (200, 150, 20), (60, 40, 61), (200, 300, 100),
                                            (3, 1, 1)])
def test_positions_past_31_bits(lm, n, window, below, flat):
    """The drafts of a request whose cached positions end just below 2^31: where they stand in a chain passes 31
    bits, what they see does not (flat: alternatives for one place, so no position does).  The same bits as for a
    short request with the same last pages."""
    c = Case([512 - below], [n], bs=256, window=window, mask=None, pos=False, seed=59, hk=1, hq=2, spare=1)
    if flat:
        c.mask = np.zeros((n, c.words), np.uint64)
        for i in range(n):
            c.mask[i, i // 64] = np.uint64(1 << i % 64)
        c.pos = np.full(n, 512 - below, np.int32)
    ref = c.check(lm)
    last = c.table[0, :2].copy()
    c.table = np.full((1, 1 << 23), c.blocks - 1, np.int32)
    c.table[0, -2:] = last
    c.lens = np.array([2**31 - below], np.int32)
    if flat:
        c.pos = np.full(n, 2**31 - below, np.int32)
    out, _ = c.run(lm)
    assert torch.equal(out, ref)


def test_another_stream_and_a_graph(lm):
    c = Case([500, 90], [8, 3], hq=16, hk=2, d=128, seed=23)
    ref = c.check(lm)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, _ = c.run(lm, stream=s)
    assert torch.equal(out, ref)
    cache, dims = lm.kv_cache_of(c.k, c.v), c.dims(lm)
    ws = torch.empty(lm.lmoe_tree_attention_workspace_bytes(dims, cache), dtype=torch.uint8, device="cuda")
    args = [dev(x) for x in (c.off, c.lens, c.table, c.mask.view(np.int64), c.pos)]
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lm.lmoe_tree_attention(dims, cache, c.q, c.kn, c.vn, *args, out, None, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    # the graph reads lengths and tables on the device: a replay with other lengths is another step
    args[1].copy_(torch.tensor([333, 17], dtype=torch.int32))
    c.lens = np.array([333, 17], np.int32)
    args[4].sub_(dev(np.repeat(np.array([500 - 333, 90 - 17], np.int32), [8, 3])))
    g.replay()
    c.pos = c.pos - np.repeat(np.array([500 - 333, 90 - 17], np.int32), [8, 3])
    assert torch.equal(c.check(lm), out)


def test_copy_descriptors_of_another_cache_are_not_used(lm):
    # a descriptor whose fields changed after its maps were made, and one without maps
    c = Case([300, 90], [8, 3], hq=16, hk=2, d=128, seed=37)
    ref = c.check(lm)
    made = lm.kv_cache_of

    def stale(k, v):
        cache = made(torch.zeros_like(k), torch.zeros_like(v))
        cache.k, cache.v = k.data_ptr(), v.data_ptr()
        return cache

    def bare(k, v):
        cache = made(k, v)
        cache.maps = None
        return cache

    class Lm:
        def __getattr__(self, name):
            return getattr(lm, name)

    for of in (stale, bare):
        other = Lm()
        other.kv_cache_of = of
        assert torch.equal(c.run(other)[0], ref)


def test_waits_as_long_as_a_long_request(lm):
    """A key head for each SM and a hundred million positions (four pages by turns): every CTA works through one
    segment of 780,000 tiles, well over a second, in which its cleaning warp waits for the last one.  That is no
    wait that ran out.  (Its status is looked at; 64-bit loops over as many keys would take minutes.)"""
    heads = torch.cuda.get_device_properties(0).multi_processor_count
    c = Case([4 * 256], [17], hq=8 * heads, hk=heads, d=128, bs=256, seed=53, spare=0)
    c.table = np.tile(c.table[:, :4], (1, 97657))
    c.lens = np.array([c.table.shape[1] * 256], np.int32)
    assert c.lens[0] // 128 > 780000
    out, ls = c.run(lm)
    assert torch.isfinite(out.float()).all() and torch.isfinite(ls).all()


def test_device_checks(lm):
    # a bad request is reported and skipped, the others are computed
    c = Case([40, 50, 60], [3, 3, 3], seed=29)
    ref, _ = c.run(lm)
    for field, value in (("lens", -1), ("lens", c.table.shape[1] * c.bs + 1), ("lens", 2**31 - 1)):
        good = getattr(c, field).copy()
        getattr(c, field)[1] = value
        out, _ = c.run(lm, want=-5)
        assert torch.equal(out[:3], ref[:3]) and torch.equal(out[6:], ref[6:]) and (out[3:6] == 9.0).all()
        setattr(c, field, good)
    for off in ([0, 3, 2, 9], [0, 3, 20, 9], [-1, 3, 6, 9], [0, 3, 6, 10]):
        good, c.off = c.off, np.array(off, np.int32)
        c.run(lm, want=-5)
        c.off = good
    out, _ = c.run(lm, want=-5, max_request_tokens=2)
    assert (out == 9.0).all()
    for bad in (-1, c.blocks, 2**31 - 1, -2**31):
        good = c.table.copy()
        c.table[1, 0] = bad
        out, _ = c.run(lm, want=-5)
        assert torch.equal(out[:3], ref[:3]) and torch.equal(out[6:], ref[6:])
        c.table = good
    assert torch.equal(c.run(lm)[0], ref)
