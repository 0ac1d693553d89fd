"""What the hybrid example refuses, on the host: its kernels are replaced by their shapes."""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))


def stack(monkeypatch, layers):
    import hybrid_serving as H
    monkeypatch.setattr(H.kda, "kda_attention_prefill", lambda q, k, v, **kw: torch.zeros_like(q))
    monkeypatch.setattr(H.kda, "kda_cache_append", lambda *a, **kw: None)
    monkeypatch.setattr(H.kda, "kda_forward", lambda q, k, v, z, A, beta, final_state=None, **kw: (torch.zeros_like(v), final_state))
    s = H.HybridStack(layers, width=16, heads=2, kv_heads=1, device="cpu")
    s.start([40, 40])
    return s


def test_a_second_prompt_is_refused_where_a_layer_would_not_see_the_first(monkeypatch):
    """The attention layers' prompts see the tokens that they bring alone: they begin a sequence."""
    s = stack(monkeypatch, "ka")
    x = torch.zeros(7, 16, dtype=torch.bfloat16)
    s.prompt(x, [3, 4])
    with pytest.raises(ValueError):
        s.prompt(x, [3, 4])
    assert s.lengths.tolist() == [3, 4]  # and nothing has changed
    s.start([40, 40])
    s.prompt(x, [3, 4])


def test_kda_layers_alone_continue(monkeypatch):
    s = stack(monkeypatch, "kk")
    x = torch.zeros(7, 16, dtype=torch.bfloat16)
    s.prompt(x, [3, 4])
    s.prompt(x, [4, 3])
    assert s.lengths.tolist() == [7, 7]


def test_pages_that_a_sequence_does_not_own_are_not_in_its_row(monkeypatch):
    """A sequence that outgrows its capacity must not write into another's pages: those entries are no page at all."""
    s = stack(monkeypatch, "a")
    s.start([200, 10, 64, 65])
    assert s.table.tolist() == [[0, 1, 2, 3], [4, -1, -1, -1], [5, -1, -1, -1], [6, 7, -1, -1]]
