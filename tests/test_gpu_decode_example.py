"""The decode example end to end: plan, heads, 8-bit cache, attention and the mixture-of-experts block together."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_fp8.py")
    spec = importlib.util.spec_from_file_location("decode_fp8", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.lm.load()
    return mod


@pytest.mark.parametrize("block_size", [16, 64])
def test_runs(ex, block_size):
    model = ex.Model(2)
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(ex.VOCAB, (n,), generator=g).tolist() for n in (1, 17, 64, 300, 600)]
    outs, logits = ex.generate(model, prompts, 20, block_size=block_size)
    assert [len(o) for o in outs] == [20] * len(prompts)
    assert all(0 <= t < ex.VOCAB for o in outs for t in o) and torch.isfinite(logits).all()
    again, same = ex.generate(model, prompts, 20, block_size=block_size)
    assert again == outs and torch.equal(same, logits)
