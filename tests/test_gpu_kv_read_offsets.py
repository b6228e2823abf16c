"""Rows read back where the offsets are not ascending or pass the rows: what is written is right, and all else is left."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_kv_fp8 import Read, lm  # noqa: F401

pytestmark = pytest.mark.gpu


def rows(r):
    """What position p of request b reads as, K and V, of every request's own table."""
    b, n = r.table.shape[0], r.table.shape[1] * r.bs
    off, r.off = r.off, np.arange(b + 1, dtype=np.int32) * n
    size, r.n, table, r.table = r.n, b * n, r.table, np.maximum(r.table, 0)
    e = [x.reshape(b, n, r.hk, r.d) for x in r.expect()]
    r.off, r.n, r.table = off, size, table
    return e


def same(got, want):
    nan = torch.isnan(want)
    return torch.equal(torch.isnan(got), nan) and torch.equal(got.masked_fill(nan, 0), want.masked_fill(nan, 0))


@pytest.mark.parametrize("off,fine", [
    ([0, 20, 60, 50], {0: (0, 20), 1: (20, 50)}),  # descends: rows from the last offset on are outside all requests
    ([0, 20, 60, 81], {0: (0, 20), 1: (20, 60)}),  # the last request passes the rows
    ([-3, 20, 60, 80], {1: (20, 60), 2: (60, 80)}),
    ([5, 20, 60, 80], {0: (5, 20), 1: (20, 60), 2: (60, 80)}),
], ids=["descends", "passes", "below_0", "starts_later"])
def test_the_other_requests_rows(lm, off, fine):  # noqa: F811
    r = Read([20, 40, 20], None, seed=6)
    want = rows(r)
    r.off[:] = off
    r.run(lm, want=0 if off[0] == 5 else -5)
    for got, w in zip(r.out, want):
        got, e = got.cpu(), torch.full((80, r.hk, r.d), 9.0).bfloat16()
        for b, (lo, hi) in fine.items():
            e[lo:hi] = w[b, lo - off[b]:hi - off[b]]
        assert same(got, e)


@pytest.mark.parametrize("seed", range(6))
def test_any_offsets(lm, seed):  # noqa: F811
    rng = np.random.default_rng(seed)
    r = Read([64] * 6, None, hk=1, seed=seed)
    want = rows(r)
    off = rng.integers(0, 64, 7)
    if seed % 2 == 0:
        off[0], off[6] = 2, 62
    r.off[:] = off
    r.run(lm, want=-5 if (np.diff(off) < 0).any() else 0)
    for got, w in zip(r.out, want):
        got, kept = got.cpu(), torch.full((1, r.hk, r.d), 9.0).bfloat16()
        for t in range(r.n):
            if off[0] <= t < off[6]:
                assert any(same(got[t], w[b, t - off[b]]) for b in range(6) if off[b] <= t < off[b + 1]), t
            else:
                assert same(got[t:t + 1], kept), t
