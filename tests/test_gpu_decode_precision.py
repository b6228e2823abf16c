"""How finely probabilities enter the product with the values, where scores are known exactly.

Queries of -1, 0 and 1, keys of 0, 1 and 2 of both signs and a power of two as scale make every score a sum of a few
whole numbers, which no order of addition changes.  So what is off is (relative to a probability; s: its score to base 2,
e: its value's exponent, |e| <= 10):
  the score's product with log2(e), less the base, plus e, plus the shift, each rounded in fp32 to 2^-24 of itself:
  4 (|s| + 16 + |e|) 2^-24; 2 ulp of the exponential; two parts of 11 bits 2^-22 (or 2^-39 of the row's largest p 2^e a
  code, which is below 2^-20 of the sum's terms here)
and relative to A = sum_j p_j |v_j| the fp32 sums of two products for 16 keys, (n / 8 + 40) 2^-23.  One part of 11 bits is off by 2^-11, which shows
where the values cancel: most elements of few keys are within 2^-4 of A.
"""
from __future__ import annotations

import numpy as np
import pytest

from test_gpu_decode_fp8 import Case, dev, lm  # noqa: F401

pytestmark = pytest.mark.gpu


def exact_scores(lens, hq, hk, d, seed, **kw):
    c = Case(lens, hq=hq, hk=hk, d=d, scale=1 / 16, v_exp=(-2, 2), seed=seed, **kw)
    rng = np.random.default_rng(seed)
    seen = c.sc[0] != 255
    c.codes[0][seen] = rng.choice(np.array([0, 0x38, 0xB8, 0x40, 0xC0], np.uint8), c.codes[0][seen].shape)
    c.sc[0][seen] = 127
    c.k.copy_(dev(c.codes[0]))
    c.ks.copy_(dev(c.sc[0]))
    c.q.copy_(dev(rng.integers(-1, 2, tuple(c.q.shape)).astype(np.float32)))
    return c


def off(c, got):
    """Of each element: how far it is off, and by how much it may be."""
    with np.errstate(invalid="ignore"):
        ref, lse, mass, _, low = c.ref()
    n = np.minimum(c.lens, c.window) if c.window else c.lens
    s = 1.45 * (c.d * 2 * c.scale)  # the largest score to base 2 that there can be
    p = 4 * (s + 26) * 2.0**-24 + 2.0**-22 + 2.0**-22
    tol = 2.0**-8 * np.abs(ref) + (p + (n[:, None, None] / 8 + 40) * 2.0**-23) * mass + 2.0**-39 * low
    return np.abs(got - ref), tol * (1 + 2.0**-6)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(4, 4), (20, 4), (32, 4), (64, 4), (40, 2)])
def test_values_that_cancel(lm, hq, hk, d):  # noqa: F811
    lens = [2, 3, 4, 5, 7, 12, 33, 40, 64, 200, 1000]
    c = exact_scores(lens, hq, hk, d, seed=hq + d)
    out, _ = c.run(lm)
    err, tol = off(c, out.float().cpu().numpy().astype(np.float64))
    assert (err <= tol).all(), (np.argwhere(err > tol)[:5], (err / tol).max())
