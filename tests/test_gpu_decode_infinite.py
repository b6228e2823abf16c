"""Rows some of whose scores leave fp32's range: minus infinity counts as none, wherever it stands; plus infinity makes
the row NaN."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_ref
from test_gpu_decode_fp8 import Case, dev, lm  # noqa: F401

pytestmark = pytest.mark.gpu

FAR, NEAR = 127 + 30, 127 - 94  # scale bytes of keys of ones: with queries of 1e30 scores of 2^130 and of some -400 to -570


def case(d, first, requests=64, n=600, hk=8):
    """Requests of n positions, of which every other run of 64 has far keys; even query heads are 1e30, odd ones 1.
    There are several tiles for each warp, so that many begin a request with far keys and go on to near ones."""
    c = Case([n] * requests, hq=2 * hk, hk=hk, d=d, v_exp=(-2, 2), seed=d)
    c.far = (np.arange(n) // 64 + first) % 2 == 0
    c.codes[0][:], c.sc[0][:] = 0xB8, NEAR
    blk, at = c.table[:, np.arange(n) // c.bs], np.arange(n) % c.bs
    c.at = (blk, at)
    c.sc[0][blk[:, c.far], :, at[c.far]] = FAR
    c.q.fill_(1.0)
    c.q[:, ::2] = 1e30
    return c


def put(c):
    c.k.copy_(dev(c.codes[0]))
    c.ks.copy_(dev(c.sc[0]))


@pytest.mark.parametrize("first", [0, 1], ids=["far_first", "near_first"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity_count_as_none(lm, d, first):  # noqa: F811
    c = case(d, first)
    put(c)
    out, ls = c.run(lm)
    v = fp8_ref.values(c.codes[1], c.sc[1])
    blk, at = c.at
    v = v[blk[:, ~c.far], :, at[~c.far]]  # [B, near, heads, d]
    n = v.shape[1]
    want = np.repeat(v.mean(axis=1), 2, axis=1)
    # equal scores: the sums alone are off, and the result's rounding
    tol = 2.0**-8 * np.abs(want) + ((n / 8 + 40) * 2.0**-23 + 2.0**-20) * np.repeat(np.abs(v).mean(axis=1), 2, axis=1)
    assert (np.abs(out.float().cpu().numpy() - want) <= tol).all()
    q = c.q[0, :, 0].double().cpu().numpy()
    lse = np.log(n) - q * d * c.scale * 2.0 ** (NEAR - 127)
    assert (lse[::2] < -126 * np.log(2)).all()  # powers of them, less no base, are zeros
    assert (np.abs(ls.double().cpu().numpy() - lse) <= 2.0**-19 * (1 + np.abs(lse))).all()


@pytest.mark.parametrize("d", [64, 128])
def test_no_other_scores(lm, d):  # noqa: F811
    c = case(d, 0)
    c.sc[0][:] = FAR
    put(c)
    out, ls = c.run(lm)
    assert not out[:, ::2].any() and torch.isneginf(ls[:, ::2]).all()
    assert torch.isfinite(out.float()).all() and torch.isfinite(ls[:, 1::2]).all()


@pytest.mark.parametrize("p", [0, 70, 599])
@pytest.mark.parametrize("d", [64, 128])
def test_plus_infinity_makes_its_row_nan(lm, d, p):  # noqa: F811
    c = case(d, 0)
    b = np.arange(0, 64, 3)
    c.codes[0][c.table[b, p // c.bs], :, p % c.bs] = 0x38  # 1 in place of -1
    c.sc[0][c.table[b, p // c.bs], :, p % c.bs] = FAR
    put(c)
    out, ls = c.run(lm)
    want = torch.zeros(64, 16, dtype=torch.bool)
    want[b, ::2] = True
    assert torch.equal(torch.isnan(out.float()).all(dim=2).cpu(), want)
    assert torch.equal(torch.isnan(out.float()).any(dim=2).cpu(), want) and torch.equal(torch.isnan(ls).cpu(), want)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_nan_values_leave_lse(lm, d):  # noqa: F811
    """The first keys' values are NaN and their scores far below the others: lse is that of the scores."""
    c = case(d, 0, requests=4)
    c.sc[0][:] = NEAR  # some -400 to -570 everywhere
    c.sc[1][c.table[1, :4], :, :] = 255
    put(c)
    c.vs.copy_(dev(c.sc[1]))
    out, ls = c.run(lm)
    assert torch.isnan(out[1].float()).all() and torch.isfinite(out[[0, 2, 3]].float()).all()
    assert torch.equal(ls[1], ls[0]) and (ls[:, ::2] < -126 * np.log(2)).all() and torch.isfinite(ls).all()
