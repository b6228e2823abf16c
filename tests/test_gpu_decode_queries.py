"""Queries whose elements are of very different size, beside keys that leave the largest one out.

A row of queries is f16 times a power of two that brings its largest magnitude Q to 2^14 to 2^15: an element of 2^-31 Q
or more is exact, a smaller one off by at most half of a subnormal's step, 2^-25 / 2^14 Q = 2^-39 Q.  So a score is off
by up to ds = scale 2^-39 Q sum_d |k_d| more than otherwise, lse by ds, and a probability by exp(2 ds) - 1 of itself."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref
from test_gpu_decode_fp8 import Case, dev, lm  # noqa: F401

pytestmark = pytest.mark.gpu


def case(d):
    c = Case([300, 40, 7], hq=24, hk=2, d=d, seed=d)
    c.codes[0][c.sc[0] != 255, 5] = 0
    c.k.copy_(dev(c.codes[0]))
    c.q.copy_((1 + c.q.abs() % 1).copysign(c.q))  # of 1 to 2
    c.q[:, :, 5] = 0
    return c


@pytest.mark.parametrize("d", [64, 128])
def test_exact_down_to_2_to_the_minus_31(lm, d):  # noqa: F811
    c = case(d)
    want, lse = c.check(lm)
    for t in (1, 14, 25, 30, 31):
        c.q[:, ::2, 5] = 2.0**t
        out, ls = c.run(lm)
        assert torch.equal(out, want) and torch.equal(ls, lse), t


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [32, 33, 34, 37, 45, 100])
def test_below_that_to_multiples(lm, d, t):  # noqa: F811
    c = case(d)
    c.q[:, :, 5] = 2.0**t
    out, ls = c.run(lm)
    with np.errstate(invalid="ignore"):
        ref, lse, mass, dot, low = c.ref()
    k = np.abs(fp8_ref.values(c.codes[0], c.sc[0])).sum(axis=-1)
    ds = min(c.scale * 2.0**-39 * 2.0**t * np.nanmax(k), 300.0)
    e = (d + 16) * 2.0**-23 * dot + 2.0**-20
    assert (np.abs(ls.double().cpu().numpy() - lse) <= e + ds + 2.0**-19 * (1 + np.abs(lse))).all()
    more = 2.0**-17 + 2.0**-23 * dot[..., None] + (300 / 8 + 40) * 2.0**-23 + 2 * e[..., None] + np.expm1(2 * ds)
    tol = (2.0**-8 * np.abs(ref) + more * mass + 2.0**-39 * low) * (1 + 2.0**-6)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert torch.isfinite(out.float()).all()
