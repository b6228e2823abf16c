"""Angles near 0, whose sine is all that an element gets: pairs (0, b) turn into (-b sin t, b cos t).

A position's step is cut off at 2^-64 turns, so the angle of position p is off by at most |p| 2^-64 turns, and by 2^-24
of itself (of half a turn, for angles above 1) from its rounding to fp32; the sine by 2^-22 of itself, a product by
2^-23: together 2^-21 of the element, 2^-22 |b| for angles above 1 and 2 pi |p| 2^-64 |b|, besides the element's
rounding to bf16, 2^-8 (2^-134 below the normal ones)."""
from __future__ import annotations

import numpy as np
import pytest

import fp8_ref
from test_gpu_qk_norm_rope import Case, host, lm  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (80, 64)])
def test_sines_of_small_angles(lm, d, rot, interleaved):  # noqa: F811
    c = Case(24, 3, 1, d, rot, norm=False, interleaved=interleaved, seed=d)
    half = rot // 2
    c.freq = np.float32(2.0) ** -np.linspace(0, 45, half).astype(np.float32)
    c.freq[1::3] *= -1
    c.pos[0] = [0, 1, -1, 2, 3, -5, 7, 11, 100, -1000, 4095, 65537] * 2
    first = slice(0, rot, 2) if interleaved else slice(0, half)
    for x in (c.q, c.k):
        x[:, :, first] = 0
    got = c.run(lm)
    for x, out in zip((c.q, c.k), got):
        y, _ = fp8_ref.norm_rope(host(x), None, c.pos, c.freq, None, rot, interleaved, False, 0.0)
        t = c.pos[0].astype(float)[:, None] * c.freq.astype(float)
        b = host(x)[:, :, slice(1, rot, 2) if interleaved else slice(half, rot)]
        near, t = np.abs(t[:, None]) <= 1, t[:, None]
        want, y1 = np.where(near, -b * np.sin(t), y[:, :, first]), host(out)[:, :, first]
        tol = 2.0**-8 * np.abs(want) * (1 + 2.0**-12) + 2.0**-134
        tol += (~near * 2.0**-22 + 2 * np.pi * np.abs(c.pos[0][:, None, None].astype(float)) * 2.0**-64) * np.abs(b)
        tol += 2.0**-21 * np.abs(want)
        bad = np.abs(y1 - want) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], y1[bad][:5], want[bad][:5])
    assert not got[0][0].float()[:, first].any() and (host(got[0])[1, :, first] != 0).all()
