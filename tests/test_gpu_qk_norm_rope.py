"""Norm and rotation of heads against a plain 64-bit computation.

Bounds: the norm (a sum of head_dim squares, a reciprocal root, two products) is within (head_dim + 16) 2^-24 relative;
the angle is the exact product to 2^-25 of a half turn, cosine and sine within 2^-22; so an element that comes from the
pair (a, b) is off by at most (2^-21 + (head_dim + 16) 2^-24) (|a| + |b|) before it is rounded to bf16 (2^-8 of itself,
or half of the smallest subnormal, 2^-134)."""
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


class Case:
    def __init__(self, T, hq, hk, d, rot=None, axes=1, axis=None, interleaved=False, norm=True, gain=True, eps=1e-6,
                 far=5000, pad=0, seed=0, size=1.0, theta=10000.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.T, self.hq, self.hk, self.d, self.rot = T, hq, hk, d, d if rot is None else rot
        self.axes, self.il, self.norm, self.eps = axes, interleaved, norm, eps
        wide = (torch.randn(T, (hq + 2 * hk) * d + pad, device="cuda", generator=g) * size).bfloat16()
        self.wide = wide
        self.q = wide[:, :hq * d].unflatten(1, (hq, d)) if hq else None
        self.k = wide[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)) if hk else None
        self.gain = [(1 + 0.3 * torch.randn(d, device="cuda", generator=g)).bfloat16() if gain else None for _ in range(2)]
        self.pos = rng.integers(-far, far, (axes, T)).astype(np.int32)
        half = self.rot // 2
        self.freq = (theta ** (-np.arange(half) / max(half, 1))).astype(np.float32)
        self.axis = axis if axis is None else np.array(axis, np.int32)

    def run(self, lm, out=None, **kw):
        a = dict(n_tokens=self.T, q_heads=self.hq, k_heads=self.hk, head_dim=self.d, rot_dim=self.rot, n_axes=self.axes,
                 interleaved=self.il, norm=self.norm, eps=self.eps)
        dims = lm.rope_dims_of(**(a | kw))
        q, k = out or [None if x is None else torch.full(x.shape, 9.0, dtype=torch.bfloat16, device="cuda")
                       for x in (self.q, self.k)]
        lm.lmoe_qk_norm_rope(dims, self.q, self.k, *self.gain, dev(self.pos), dev(self.freq),
                             None if self.axis is None else dev(self.axis), q, k)
        torch.cuda.synchronize()
        return q, k

    def ref(self):
        return [None if x is None else fp8_ref.norm_rope(host(x), None if g is None else host(g), self.pos, self.freq,
                                                         self.axis, self.rot, self.il, self.norm, self.eps)
                for x, g in zip((self.q, self.k), self.gain)]

    def check(self, lm, got=None, ref=None):
        got, ref = got or self.run(lm), ref or self.ref()
        for x, r in zip(got, ref):
            if r is None:
                continue
            y, pair = r
            tol = 2.0**-8 * np.abs(y) + (2.0**-21 + (self.d + 16) * 2.0**-24) * (1 + 2.0**-7) * pair + 2.0**-134
            err = np.abs(host(x) - y)
            assert (err <= tol).all(), (np.argwhere(err > tol)[:4], host(x)[err > tol][:4], y[err > tol][:4])
        return got


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(8, 8), (16, 8), (64, 64), (64, 32), (72, 40), (80, 80), (96, 96), (128, 128), (128, 24),
                                   (128, 0), (136, 136), (192, 64), (256, 256), (248, 200)])
def test_widths(lm, d, rot, interleaved):
    Case(5, 3, 2, d, rot, interleaved=interleaved, seed=d + rot).check(lm)
    Case(3, 2, 1, d, rot, interleaved=interleaved, norm=False, seed=d).check(lm)


@pytest.mark.parametrize("T,hq,hk,d", [(1, 64, 8, 128), (1, 1, 0, 64), (1, 0, 1, 64), (7, 5, 1, 128), (700, 1, 1, 64),
                                       (2500, 2, 0, 64), (3000, 0, 3, 80), (1300, 40, 8, 128), (900, 11, 2, 256),
                                       (2, 1024, 1024, 8), (1, 1024, 3, 128)])
def test_shapes(lm, T, hq, hk, d):
    for il in (False, True):
        Case(T, hq, hk, d, interleaved=il, seed=T).check(lm)


@pytest.mark.parametrize("axes,axis", [(1, None), (2, None), (3, [0, 1, 2] * 10 + [0, 1]), (3, [0] * 8 + [1] * 12 + [2] * 12),
                                       (4, [3] * 32), (2, [0, 1, 2, -1] * 8)], ids=str)
def test_axes(lm, axes, axis):
    # (an axis that there is not turns nothing; without a table all frequencies go by axis 0)
    for il in (False, True):
        Case(40, 4, 2, 64, axes=axes, axis=axis, interleaved=il, seed=axes).check(lm)


@pytest.mark.parametrize("far", [1, 131072, 2**24 + 1, 2**31 - 1])
def test_far_positions(lm, far):
    c = Case(300, 2, 1, 128, far=far, norm=False, seed=3, theta=500000.0)
    c.pos[0, :6] = [0, far, far - 1, -far, -far - 1 if far < 2**31 - 1 else -2**31, far // 2]
    c.check(lm)


def test_any_frequency(lm):
    c = Case(200, 2, 1, 64, far=10**6, norm=False, seed=4)
    c.freq = np.array([0.0, -0.0, 1023.9, -1.0, -0.37, 1e-30, 1e-45, 3.1415927, 6.2831855, 0.5, 2.0**-40, 100.0] + [0.01] * 20,
                      np.float32)
    c.check(lm)


@pytest.mark.parametrize("size,eps,gain", [(1e-3, 1e-6, True), (1e15, 0.0, True), (1e-15, 1e-12, False), (1.0, 1e-5, False)])
def test_norms(lm, size, eps, gain):
    Case(50, 4, 2, 128, size=size, eps=eps, gain=gain, seed=5).check(lm)


def test_rows_of_zeros(lm):
    c = Case(4, 2, 1, 64, seed=6)
    c.q[1].zero_()
    q, k = c.check(lm)
    assert not q[1].any()


def test_nan_and_infinity_stay_in_their_head(lm):
    c = Case(3, 4, 2, 64, seed=7)
    ref = c.run(lm)
    c.q[1, 2, 5] = float("nan")
    c.k[2, 0, 63] = float("inf")
    q, k = c.run(lm)
    assert torch.isnan(q[1, 2]).all()
    q[1, 2], k[2, 0] = ref[0][1, 2], ref[1][2, 0]
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_what_is_not_turned_stays_as_it_is(lm, interleaved):
    """Without a norm, elements from rot_dim on are copied: infinities, NaN and zeros of both signs too."""
    c = Case(5, 2, 1, 64, rot=24, norm=False, interleaved=interleaved, seed=12)
    c.q[:, :, 24:].copy_(torch.tensor([float("inf"), 1.0, -0.0, float("-inf"), 0.0, float("nan"), 2.0, -0.0] * 5))
    q, k = c.run(lm)
    got, want = q[:, :, 24:].contiguous(), c.q[:, :, 24:].contiguous()
    nan = torch.isnan(want)  # (any NaN for a NaN, all else to the bit)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])
    assert torch.equal(k[:, :, 24:], c.k[:, :, 24:]) and torch.isfinite(q[:, :, :24]).all()


def test_in_place_and_into_wider_rows(lm):
    for il in (False, True):
        c = Case(70, 6, 2, 128, pad=40, interleaved=il, seed=8)
        ref, want = c.ref(), c.run(lm)
        wide = torch.full((70, 10 * 128 + 8), 9.0, dtype=torch.bfloat16, device="cuda")
        out = (wide[:, 8:8 + 6 * 128].unflatten(1, (6, 128)), wide[:, 8 + 7 * 128:8 + 9 * 128].unflatten(1, (2, 128)))
        c.check(lm, c.run(lm, out=out), ref)
        assert (wide[:, :8] == 9).all() and (wide[:, 8 + 6 * 128:8 + 7 * 128] == 9).all() and (wide[:, -128:] == 9).all()
        rest = c.wide[:, 8 * 128:].clone()
        got = c.run(lm, out=(c.q, c.k))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(c.wide[:, 8 * 128:], rest)


def test_offsets_past_32_bits(lm):
    # rows that lie far apart: the last one starts past 2^32 bytes
    stride, T = 1 << 26, 40
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((T, 2, 64), (stride, 64, 1))
    c = Case(T, 2, 0, 64, seed=9)
    want, _ = c.run(lm)
    q.copy_(c.q)
    c.q = q
    got, _ = c.run(lm)
    assert torch.equal(got, want)
    got, _ = c.run(lm, out=(q, None))
    assert torch.equal(got, want)


def test_streams_and_graphs(lm):
    c = Case(33, 4, 2, 64, seed=10)
    want = c.run(lm)
    args = (lm.rope_dims_of(33, 4, 2, 64), c.q, c.k, *c.gain, dev(c.pos), dev(c.freq), None)
    out = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lm.lmoe_qk_norm_rope(*args, *out)
    s.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lm.lmoe_qk_norm_rope(*args, *out)
    c.q.copy_(torch.randn(33, 4, 64, device="cuda").bfloat16())
    g.replay()
    torch.cuda.synchronize()
    c.check(lm, out)


def test_binding_refuses(lm):
    c = Case(5, 4, 2, 64)
    q, k = (torch.empty_like(x.contiguous()) for x in (c.q, c.k))
    good = dict(dims=lm.rope_dims_of(5, 4, 2, 64), q=c.q, k=c.k, q_gain=None, k_gain=None, pos=dev(c.pos), inv_freq=dev(c.freq),
                axis=None, q_out=q, k_out=k)
    lm.lmoe_qk_norm_rope(**good)
    for bad, kind in ((dict(q=c.q.float()), TypeError), (dict(q=c.q[:4]), ValueError), (dict(k=c.q), ValueError),
                      (dict(pos=dev(c.pos)[:, :4]), ValueError), (dict(pos=dev(c.pos).long()), TypeError),
                      (dict(inv_freq=dev(c.freq)[:31]), ValueError), (dict(axis=dev(c.pos)[0]), ValueError),
                      (dict(q_gain=dev(c.freq)), TypeError), (dict(pos=None), lm.LmoeError), (dict(k_out=c.q[:, :2]), lm.LmoeError),
                      (dict(dims=lm.rope_dims_of(5, 4, 2, 64, rot_dim=20)), lm.LmoeError)):
        with pytest.raises(kind):
            lm.lmoe_qk_norm_rope(**(good | bad))
