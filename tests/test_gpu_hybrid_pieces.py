"""The hybrid example with its prompts served in pieces and with rotary positions: it runs, and its tokens are those of the
same tokens served as one prompt.

As where the tokens come one at a time, the two differ by what the cache holds: e4m3 keys and values, half a step of
2^-4 of a value; the pieces' tokens are among those that see the rounded ones, whose outputs a KDA layer's state carries
further.  The residual stream's norm does not shrink, so 2^-4 per attention layer bounds the relative difference, and
twice that any one row's, whose part of the rounding may be above the mean.  A turn keeps a vector's length.
"""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("layers, piece, rotary", [("a", 16, False), ("a", 0, True), ("akak", 33, True), ("kkka", 130, True), ("kk", 50, False)])
def test_pieces_agree_with_whole_prompts(layers, piece, rotary):
    import hybrid_serving
    got, want = hybrid_serving.demo(layers, prompts=(37, 5, 130), steps=3, drafts=4, piece=piece, rotary=rotary)
    err = float((got.float() - want.float()).norm() / want.float().norm())
    assert err <= 2.0 ** -4 * max(1, layers.count("a")), err
    row = (got.float() - want.float()).norm(dim=-1) / want.float().norm(dim=-1)
    assert float(row.max()) <= 2.0 ** -3 * max(1, layers.count("a")), row
