"""The speculative-decoding example end to end: trees, paged cache, block planning and writes together."""
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
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.lm.load()
    return mod


@pytest.mark.parametrize("block_size,depth", [(16, 4), (32, 2), (64, 7)])
def test_verified_tokens_are_the_decoder_s_own(ex, block_size, depth):
    """Every generated token is the one-token decoder's best, but for rounding: the two passes round activations
    at 2^-8 per layer and op, so a choice may be off where two logits lie within a few per cent of the logits'
    spread.  A router whose 4th and 5th expert lie that close may also pick another one (their gap is 0.25 on
    average, the rounding moves it by 0.01: 4% of the rows and layers, few of them rows with a close choice), so
    one token in twenty may be off by more."""
    model = ex.Model(2)
    g = torch.Generator().manual_seed(5)
    # six requests over four places (places are given back and taken again), prompts of one token to two chunks
    prompts = [torch.randint(ex.VOCAB, (n,), generator=g).tolist() for n in (1, 17, 64, 33, 300, 5)]
    outs, steps = ex.generate(model, prompts, 24, block_size=block_size, depth=depth)
    assert [len(o) for o in outs] == [24] * len(prompts)
    gaps, spread = ex.margins(model, prompts, outs, block_size)
    off = sum(x > 0.05 * spread for x in gaps)
    assert off <= len(gaps) // 20, (off, max(gaps), spread)
    _, plain_steps = ex.generate(model, prompts, 24, block_size=block_size, depth=0)
    assert steps < 0.8 * plain_steps
