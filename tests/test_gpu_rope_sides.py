"""A side without heads needs nothing, and nothing of it is looked at."""
from __future__ import annotations

import pytest
import torch

from test_gpu_qk_norm_rope import Case, lm  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hk", [(3, 0), (0, 3)])
def test_a_gain_of_no_heads_may_be_anywhere(lm, hq, hk, interleaved):  # noqa: F811
    c = Case(9, hq, hk, 128, interleaved=interleaved, seed=hq)
    want = c.check(lm)
    # (the other side's would have to be 8-byte aligned)
    c.gain[hq > 0] = torch.full((129,), float("nan"), dtype=torch.bfloat16, device="cuda")[1:]
    assert c.gain[hq > 0].data_ptr() % 8 == 2
    got = c.run(lm)
    assert all(torch.equal(x, y) for x, y in zip(got, want) if x is not None)
    # ... and without a norm neither is
    c.norm = False
    c.gain[hq == 0] = None
    c.check(lm)
