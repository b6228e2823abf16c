"""What a warp of the attention kernel decides on is one answer for all its lanes.

A barrier's phase may complete between two lanes' probes of it.  Where a probe's answer leads
to warp-wide steps (a __syncwarp, a warp-aligned load from tensor memory, an arrival of one lane
for all), lanes that got different answers would part there: some would wait for the others, or
signal data that is not there yet.  No run shows that reliably, so the source is read instead."""
from __future__ import annotations

import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "latent_moe_layer_fp32_gb300", "csrc",
                   "tree_attn.cu")


def probes(name):
    """Each call of a barrier probe with what stands before it."""
    text = open(SRC).read()
    return [text[max(0, m.start() - 40):m.start()] for m in re.finditer(rf"\b{name}\(", text)]


def test_one_shot_probes_are_voted_on():
    asked = probes("mbar_test_wait")
    assert asked
    for before in asked:
        assert before.endswith("__all_sync(0xffffffffu, "), before


def test_a_warp_leaves_a_loop_only_by_a_vote():
    # a wait may run out for one lane and not for another: no loop ends on one lane's answer
    code = re.sub(r"//[^\n]*", "", open(SRC).read())
    code = code[code.index("tree_attn_kernel(const"):code.index("tree_attn_merge_kernel(const")]
    ways_out = [x for x in code.splitlines() if re.search(r"\b(break|return false);", x)
                and re.search(r"\bok\b|\bfailed\b|_wait|gave_up|ready\(|copy\(", x)]
    assert len(ways_out) >= 6
    for x in ways_out:
        # `copy` ends with a vote of its own; the other two test an `ok` that has been voted on
        assert re.search(r"__all_sync\(0xffffffffu|bar_wait_warp\(|gave_up\(\)|copy\(|if \(!ok\) break;|!ok \|\| n == 0", x), x
    assert re.search(r"if \(ok\) ok = seg_wait\(seg\);\s*ok = __all_sync\(0xffffffffu, ok\);", code)
