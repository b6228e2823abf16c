"""Tree masks, block plans and slot writes against plain loops: whole numbers and
copies, so everything has to be equal."""
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


def status_ws():
    return torch.full((256,), 255, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------------------------
# masks
# ---------------------------------------------------------------------------------------------

def trees(rng, ns, kind):
    par = []
    for n in ns:
        for i in range(n):
            par.append({"chain": i - 1, "flat": -1, "star": 0 if i else -1,
                        "random": int(rng.integers(-1, i)) if i else -1}[kind])
    return np.array(par, np.int32)


@pytest.mark.parametrize("kind", ["chain", "flat", "star", "random"])
@pytest.mark.parametrize("ns,words", [([1], 1), ([8], 1), ([64, 1, 0, 63], 1), ([65, 128, 2], 2), ([129, 3], 3),
                                      ([256, 255, 0, 193], 4), ([5] * 300, 1)],
                         ids=["one", "eight", "full_word", "two_words", "three_words", "four_words", "many"])
def test_tree_masks(lm, ns, words, kind):
    rng = np.random.default_rng(len(ns) + words)
    off = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    par = trees(rng, ns, kind)
    lens = rng.integers(0, 1 << 30, len(ns)).astype(np.int32)
    for ln in (lens, None):
        em, ep = kv_ref.tree_masks(off, par, ln, words)
        mask = torch.full((len(par), words), -1, dtype=torch.int64, device="cuda")
        pos = torch.full((len(par),), -7, dtype=torch.int32, device="cuda")
        ws = status_ws()
        lm.lmoe_tree_masks(dev(off), dev(par), None if ln is None else dev(ln), mask, pos, ws)
        assert lm.lmoe_status_check(ws) == 0
        assert np.array_equal(mask.cpu().numpy().view(np.uint64), em)
        assert np.array_equal(pos.cpu().numpy(), ep)


def test_tree_masks_reports_bad_trees(lm):
    def call(off, par, words=1):
        mask = torch.full((len(par), words), -1, dtype=torch.int64, device="cuda")
        pos = torch.full((len(par),), -7, dtype=torch.int32, device="cuda")
        ws = status_ws()
        lm.lmoe_tree_masks(dev(np.array(off, np.int32)), dev(np.array(par, np.int32)), None, mask, pos, ws)
        return lm.lmoe_status_check(ws), mask.cpu().numpy()[:, 0], pos.cpu().numpy()

    # a parent that is the row itself, a later row or below -1 counts as -1
    for bad in (1, 2, 9, -2, 1 << 30):
        rc, mask, pos = call([0, 3], [-1, bad, 0])
        assert rc == -5 and mask.tolist() == [1, 2, 5] and pos.tolist() == [0, 0, 1]
    # a request wider than the mask: empty masks
    rc, mask, pos = call([0, 65, 66], [-1] * 66)
    assert rc == -5 and mask.tolist() == [0] * 65 + [1] and pos.tolist() == [0] * 66
    # offsets that descend or pass the rows: that request is left alone
    rc, mask, _ = call([0, 2, 1, 4], [-1] * 3)
    assert rc == -5 and mask.tolist() == [1, 2, -1]


# ---------------------------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------------------------

def plan_case(rng, B, bs, max_blocks, free, new, lens=None, slack=0, short_slots=0):
    lens = rng.integers(0, max_blocks * bs // 2 + 1, B).astype(np.int32) if lens is None else np.array(lens, np.int32)
    new = np.array(new, np.int32)
    owned = (-(-lens // bs) + rng.integers(0, slack + 1, B)).astype(np.int32)
    owned = np.minimum(owned, max_blocks).astype(np.int32)
    size = int(owned.sum()) + free + 5
    ids = rng.permutation(size).astype(np.int32)
    table = np.full((B, max_blocks), -9, np.int32)
    at = 0
    for b in range(B):
        table[b, :owned[b]] = ids[at:at + owned[b]]
        at += owned[b]
    head = int(rng.integers(size))
    ring = np.full(size, -3, np.int32)
    for i in range(free):
        ring[(head + i) % size] = ids[at + i]
    n_slots = max(1, int(np.maximum(new, 0).sum()) - short_slots)
    return bs, max_blocks, n_slots, lens, new, owned, table, ring, np.array([head, free], np.int32)


def run_plan(lm, bs, max_blocks, n_slots, lens, new, owned, table, ring, state, off=0):
    B = len(lens)
    t, r = dev(table), dev(ring)
    o = {k: torch.full((n,), -77, dtype=torch.int32, device="cuda") for k, n in
         (("lens", B), ("owned", B), ("state", 2), ("offsets", B + 1), ("slots", n_slots))}
    args = [dev(np.concatenate([np.full(off, -5, np.int32), x]))[off:] for x in (lens, new, owned)]
    st = dev(state)
    for _ in range(2):  # the same inputs again give the same outputs
        lm.lmoe_kv_plan(bs, *args, t, r, st, o["lens"], o["owned"], o["state"], o["offsets"], o["slots"])
        got = {k: v.cpu().numpy() for k, v in o.items()} | {"block_table": t.cpu().numpy(), "ring": r.cpu().numpy()}
    return got


def check_plan(lm, case):
    exp, got = kv_ref.plan(*case), run_plan(lm, *case)
    for k in exp:
        assert np.array_equal(got[k], exp[k]), k


@pytest.mark.parametrize("B,bs,max_blocks", [(1, 16, 4), (7, 16, 9), (33, 64, 5), (1000, 32, 20), (1025, 16, 8),
                                             (4097, 16, 3), (8192, 16, 2), (5, 1, 40), (9, 48, 7)])
def test_plan_random(lm, B, bs, max_blocks):
    rng = np.random.default_rng(B + bs)
    new = rng.integers(-1, 2 * bs + 2, B)
    check_plan(lm, plan_case(rng, B, bs, max_blocks, free=2 * B + 8, new=new, slack=1))
    # too few free blocks: the requests that fit in order are served
    check_plan(lm, plan_case(rng, B, bs, max_blocks, free=max(1, B // 2), new=new, slack=1))
    # too few slots: the last requests wait
    check_plan(lm, plan_case(rng, B, bs, max_blocks, free=2 * B + 8, new=new, short_slots=bs + 3))


@pytest.mark.parametrize("B", [1026, 1027, 1028, 2050, 4095, 4096, 5003, 8191])
def test_plan_any_alignment(lm, B):
    """Arrays that start between 16-byte boundaries, and request counts that fill no whole four."""
    rng = np.random.default_rng(B)
    case = plan_case(rng, B, 16, 4, free=B, new=rng.integers(-1, 20, B), slack=1)
    exp = kv_ref.plan(*case)
    for off in (0, 1, 3):
        got = run_plan(lm, *case, off=off)
        for k in exp:
            assert np.array_equal(got[k], exp[k]), (off, k)


@pytest.mark.parametrize("new,lens,free", [([0], [0], 3), ([0], [16], 0), ([1], [16], 1), ([1], [16], 0),
                                           ([16], [0], 1), ([17], [0], 2), ([33, 1, 1], [0, 15, 16], 1),
                                           ([-1, -1], [0, 40], 0), ([-1, 40, -1, 3], [64, 0, 31, 15], 3),
                                           ([100, 1], [0, 3], 9)])
def test_plan_edges(lm, new, lens, free):
    rng = np.random.default_rng(5)
    check_plan(lm, plan_case(rng, len(new), 16, 4, free, new, lens=lens))


def test_plan_long_prompts(lm):
    rng = np.random.default_rng(8)
    check_plan(lm, plan_case(rng, 3, 16, 4096, 9000, [50000, 7, 60001], lens=[100, 5, 0]))


def test_plan_overflowing_sums(lm):
    # token counts whose sum passes 32 bits: nothing past the slots is served, the rest is
    rng = np.random.default_rng(9)
    case = list(plan_case(rng, 4, 16, 8, 20, [5, 0, 0, 0], lens=[3, 4, 5, 6]))
    case[4] = np.array([5, 2**31 - 1, 2**31 - 1, 4], np.int32)
    got = run_plan(lm, *case)
    assert got["lens"].tolist() == [8, 4, 5, 6] and got["offsets"].tolist()[:3] == [0, 5, 2**31 - 1]
    assert (got["slots"] >= 0).all()


def test_plan_lengths_past_31_bits(lm):
    # a request whose length would pass 31 bits is not served, its neighbours are; positions up to there are exact
    top, bs = 2**31 - 1, 1 << 30
    table = np.array([[0, 1, -9, -9], [1, 0, -9, -9], [1, 1, -9, -9]], np.int32)
    got = run_plan(lm, bs, 4, 16, np.array([top - 4, top - 19, top - 3], np.int32), np.array([10, 3, 3], np.int32),
                   np.array([2, 2, 2], np.int32), table, np.array([5, 6, 7, 8], np.int32), np.array([0, 4], np.int32))
    assert got["lens"].tolist() == [top - 4, top - 16, top] and got["owned"].tolist() == [2, 2, 2]
    assert got["offsets"].tolist() == [0, 10, 13, 16] and got["state"].tolist() == [0, 4]
    first = top - 19 - bs  # in the second block of its table, which is block 0; the next request's is block 1
    assert got["slots"].tolist() == [-1] * 10 + [first, first + 1, first + 2] + [top - 3, top - 2, top - 1]
    assert np.array_equal(got["block_table"], table)
    # more table than positions, more owned than held: still not served
    got = run_plan(lm, 1 << 29, 100, 16, np.array([top], np.int32), np.array([16], np.int32),
                   np.array([60], np.int32), np.zeros((1, 100), np.int32), np.array([5], np.int32),
                   np.array([0, 1], np.int32))
    assert got["lens"].tolist() == [top] and got["owned"].tolist() == [60] and got["slots"].tolist() == [-1] * 16


@pytest.mark.parametrize("block,bs,slot", [(2047, 1 << 20, 2047 << 20), (2048, 1 << 20, -1), (5000, 1 << 20, -1),
                                           (1 << 28, 16, -1), (2**31 - 1, 16, -1), (-1, 16, -1), (-2**31, 16, -1)])
def test_plan_slots_past_31_bits(lm, block, bs, slot):
    # a block number from the ring, and one from the table, whose slot is no int32 (or that is none): -1, not another slot
    for lens, table, ring in ((0, -9, block), (bs - 5, block, -9)):
        got = run_plan(lm, bs, 1, 3, np.array([lens], np.int32), np.array([3], np.int32),
                       np.array([1 if lens else 0], np.int32), np.array([[table]], np.int32),
                       np.array([ring], np.int32), np.array([0, 1], np.int32))
        at = lens if slot >= 0 else 0
        assert got["slots"].tolist() == ([slot + at, slot + at + 1, slot + at + 2] if slot >= 0 else [-1] * 3)


def test_plan_as_many_slots_as_there_can_be(lm):
    n = 2**31 - 1  # 8.6 GB
    slots = torch.zeros(n, dtype=torch.int32, device="cuda")
    lens, new, owned, state = (dev(np.array(x, np.int32)) for x in ([3, 0], [5, 2], [1, 0], [0, 2]))
    table, ring = dev(np.array([[4, -9], [-9, -9]], np.int32)), dev(np.array([7, 8], np.int32))
    o = [torch.zeros(m, dtype=torch.int32, device="cuda") for m in (2, 2, 2, 3)]
    lm.lmoe_kv_plan(16, lens, new, owned, table, ring, state, *o, slots)
    assert slots[:7].tolist() == [67, 68, 69, 70, 71, 112, 113]
    assert int(slots[7:].max()) == -1 and int(slots[7:].min()) == -1
    assert [x.tolist() for x in o] == [[8, 2], [1, 1], [1, 1], [0, 5, 7]]


# ---------------------------------------------------------------------------------------------
# writes
# ---------------------------------------------------------------------------------------------

def caches(blocks, hk, bs, d, order, fill=0.0):
    shape = (blocks, hk, bs, d) if order == "head" else (blocks, bs, hk, d)
    c = [torch.full(shape, fill, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return c if order == "head" else [x.transpose(1, 2) for x in c]


@pytest.mark.parametrize("order", ["head", "slot"])
@pytest.mark.parametrize("n,hk,bs,d,gather,pad", [(1, 8, 16, 128, False, 0), (3, 1, 16, 64, True, 8),
                                                  (211, 3, 32, 64, True, 64), (1000, 8, 64, 128, False, 1024),
                                                  (777, 5, 256, 128, True, 0), (2049, 2, 128, 64, False, 24)])
def test_write(lm, n, hk, bs, d, gather, pad, order):
    g = torch.Generator(device="cuda").manual_seed(n)
    rng = np.random.default_rng(n)
    blocks, rows = n // bs + 4, n + (n // 2 if gather else 0)
    wide = torch.randn(rows, 2 * hk * d + pad, device="cuda", generator=g).bfloat16()
    kn, vn = (wide[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in range(2))
    slots = rng.permutation(blocks * bs)[:n].astype(np.int32)
    if n > 2:
        slots[rng.integers(n)] = -1
        slots[rng.integers(n)] = -5
    src = rng.integers(0, rows, n).astype(np.int32) if gather else np.arange(n, dtype=np.int32)
    k, v = caches(blocks, hk, bs, d, order, fill=7.0)
    ek, ev = (x.clone().contiguous().float().cpu().numpy() for x in (k, v))
    hkn, hvn = kn.float().cpu().numpy(), vn.float().cpu().numpy()
    for t in range(n):
        if slots[t] >= 0:
            ek[slots[t] // bs, :, slots[t] % bs] = hkn[src[t]]
            ev[slots[t] // bs, :, slots[t] % bs] = hvn[src[t]]
    ws = status_ws()
    lm.lmoe_kv_write(lm.kv_cache_of(k, v), kn, vn, dev(src) if gather else None, dev(slots), ws)
    assert lm.lmoe_status_check(ws) == 0
    assert np.array_equal(k.float().cpu().numpy(), ek) and np.array_equal(v.float().cpu().numpy(), ev)


def test_write_passes_over_what_is_out_of_range(lm):
    k, v = caches(2, 1, 16, 64, "head")
    kn = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    src = dev(np.array([0, 1, 4, -1, 2], np.int32))
    slots = dev(np.array([3, 32, 4, 5, 6], np.int32))
    ws = status_ws()
    lm.lmoe_kv_write(lm.kv_cache_of(k, v), kn, kn, src, slots, ws)
    assert lm.lmoe_status_check(ws) == -5
    lm.lmoe_kv_write(lm.kv_cache_of(k, v), kn, kn, src, slots)  # without a workspace: passed over all the same
    for c in (k, v):
        rows = c[:, 0, :, 0].flatten().float().cpu().tolist()
        assert [i for i, x in enumerate(rows) if x] == [3, 6]


def test_write_offsets_past_32_bits(lm):
    # the last blocks of a cache of more than 2^31 elements (and 2^32 bytes) per tensor
    blocks, hk, bs, d = 36000, 8, 64, 128
    k, v = (torch.empty(blocks, hk, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[-1].zero_()
    v[-1].zero_()
    kn = torch.randn(2, hk, d, device="cuda").bfloat16()
    vn = torch.randn(2, hk, d, device="cuda").bfloat16()
    slots = dev(np.array([blocks * bs - 1, (blocks - 1) * bs], np.int32))
    lm.lmoe_kv_write(lm.kv_cache_of(k, v), kn, vn, None, slots)
    for c, n in ((k, kn), (v, vn)):
        assert torch.equal(c[-1, :, -1], n[0]) and torch.equal(c[-1, :, 0], n[1])
        assert int((c[-1, :, 1:-1] != 0).sum()) == 0


def test_calls_on_another_stream_and_in_a_graph(lm):
    B, bs = 6, 16
    rng = np.random.default_rng(3)
    case = plan_case(rng, B, bs, 12, 40, [3, 0, 17, -1, 1, 8])
    exp = kv_ref.plan(*case)
    _, _, n_slots, lens, new, owned, table, ring, state = case
    dv = [dev(x) for x in (lens, new, owned, table, ring, state)]
    o = [torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (B, B, 2, B + 1, n_slots)]
    k, v = caches(len(ring), 2, bs, 64, "head")
    kn = torch.randn(n_slots, 2, 64, device="cuda").bfloat16()
    cache = lm.kv_cache_of(k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lm.lmoe_kv_plan(bs, *dv[:3], *dv[3:], *o)
        lm.lmoe_kv_write(cache, kn, kn, None, o[4])
    s.synchronize()
    for x in o:
        x.fill_(-77)
    k.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lm.lmoe_kv_plan(bs, *dv[:3], *dv[3:], *o)
        lm.lmoe_kv_write(cache, kn, kn, None, o[4])
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(o[4].cpu().numpy(), exp["slots"])
    slots = torch.from_numpy(exp["slots"]).long()
    assert torch.equal(k[(slots // bs).cuda(), :, (slots % bs).cuda()], kn)
