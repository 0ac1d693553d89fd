"""Pieces of the hybrid example's prompts on the host: its kernels are replaced by their shapes."""
import torch

from test_hybrid_example_host import stack


def test_a_step_in_which_no_sequence_brings_a_token(monkeypatch):
    s = stack(monkeypatch, "ka")
    import hybrid_serving as H
    monkeypatch.setattr(H.kda, "kda_attention_extend", lambda q, *a, **kw: torch.zeros_like(q))
    x = torch.zeros(7, 16, dtype=torch.bfloat16)
    assert s.more(x, [3, 4]).shape == (7, 16)
    assert s.more(x[:0], [0, 0]).shape == (0, 16) and s.lengths.tolist() == [3, 4]
    assert s.more(x[:2], [2, 0]).shape == (2, 16) and s.lengths.tolist() == [5, 4]
