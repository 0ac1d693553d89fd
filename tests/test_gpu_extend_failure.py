"""Waits of kda_attention_extend that give up, driven by KDA_DEBUG_HANDOFF_TRIES without any GPU fault: the call ends, its
check word tells, and the next call is right.

A unit of at most 128 rows leaves the second half of the softmax without tiles; it follows the others' tiles at a barrier
whose waits give up, too.
"""
import pytest
import torch

from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_attention import offsets
from test_gpu_extend import DEV, IO, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,new", [([50000], [1]), ([9000, 300, 70], [300, 300, 1]), ([40000, 2000], [20, 2000])],
                         ids=["token", "chunks", "both"])
def test_waits_that_give_up_show(monkeypatch, lens, new, io):
    q, cache, table, lengths = case(lens, new, 8, 2, 128, 64, torch.float8_e4m3fn, io, seed=17)
    cu = offsets(new)
    need = B.kda_attention_extend_workspace_bytes(B.KdaAttention(len(lens), sum(new), 8, 2, 128, B._IO[io], 1.0, 0, 0, 0))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    call = lambda: B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=cu, workspace=ws)  # noqa: E731
    clean = call()
    assert B.kda_workspace_status(ws) == B.KDA_OK
    for tries in ("0", "1", "3"):
        monkeypatch.setenv("KDA_DEBUG_HANDOFF_TRIES", tries)
        out = call()
        status = B.kda_workspace_status(ws)
        monkeypatch.delenv("KDA_DEBUG_HANDOFF_TRIES")
        assert status == B.KDA_ERR_TIMEOUT if tries == "0" else status in (B.KDA_OK, B.KDA_ERR_TIMEOUT)
        assert status != B.KDA_OK or torch.equal(out, clean)
        print(f"tries {tries}: status {status}")
        assert torch.equal(call(), clean)
        assert B.kda_workspace_status(ws) == B.KDA_OK
