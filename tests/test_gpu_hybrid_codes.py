"""What the hybrid example leaves in its caches: a prompt's keys and values take the same codes whole and in pieces."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


def served(rotary, lens, piece):
    import hybrid_serving
    s = hybrid_serving.HybridStack("a", seed=4, rotary=rotary)
    s.start(lens)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = [torch.randn(n, 512, generator=g, device="cuda").bfloat16() for n in lens]
    if piece == 0:
        s.prompt(torch.cat(x), lens)
    for at in range(0, max(lens) if piece else 0, piece or 1):
        part = [y[at:at + piece] for y in x]
        s.more(torch.cat(part), [len(y) for y in part])
    return s


@pytest.mark.parametrize("rotary", [False, True])
def test_codes_of_whole_prompts_and_of_pieces(rotary):
    """Pieces of whole pages, so that no page's scale grows between them (rounded keys would be rounded again)."""
    lens = [300, 64, 129]
    whole = served(rotary, lens, 0)
    for piece in (64, 128):
        pieces = served(rotary, lens, piece)
        assert torch.equal(whole.lengths, pieces.lengths)
        for a, b in zip(whole.memory[0], pieces.memory[0]):
            assert torch.equal(a.float(), b.float())


def test_a_step_in_which_no_sequence_brings_a_token():
    import hybrid_serving
    s = hybrid_serving.HybridStack("ka", rotary=True)
    s.start([70, 70])
    x = torch.randn(9, 512, device="cuda").bfloat16()
    s.more(x, [5, 4])
    before = [[y.clone() for y in m] if isinstance(m, tuple) else [m.clone()] for m in s.memory]
    assert s.more(x[:0], [0, 0]).shape == (0, 512) and s.lengths.tolist() == [5, 4]
    for m, was in zip(s.memory, before):
        assert all(torch.equal(y.float(), z.float()) for y, z in zip(m if isinstance(m, tuple) else [m], was))
