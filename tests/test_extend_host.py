"""What kda_attention_extend refuses on the host, before any launch (no GPU: the fake addresses are never
dereferenced)."""
import ctypes

import pytest
import torch

from linear_attention_recurrence_kda_gb300 import binding as B
from test_abi_host import L, _addr  # noqa: F401  (fixture)
from test_attention_host import BAD, BAD_Q, attention, cache
from test_stream_allocations import Side, refused, watched  # noqa: F401  (fixture)


def extend(L, p, c, ws=_addr(30, 1 << 25), wsb=1 << 30, **over):
    ptr = {n: _addr(i) for i, n in enumerate(("q", "cu", "lengths", "out"))}
    ptr["cu"] = None
    ptr.update(over)
    return L.kda_attention_extend(ptr["q"], ptr["cu"], ptr["lengths"], ctypes.byref(c) if c else None, ptr["out"],
                                  ctypes.byref(p) if p else None, ws, ctypes.c_size_t(wsb), None)


@pytest.mark.parametrize("bad,status", BAD + BAD_Q)
def test_bad_descriptors(L, bad, status):  # noqa: F811
    p = attention(**bad)
    assert extend(L, p, cache()) == status
    assert (B.kda_attention_extend_workspace_bytes(p) == 0) == ("q_stride" not in bad or bad["q_stride"] < 0)


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), B.KDA_ERR_INVALID_ARG), (dict(v_scale=None), B.KDA_ERR_INVALID_ARG),
    (dict(block_table=None), B.KDA_ERR_INVALID_ARG), (dict(k=_addr(20) + 8), B.KDA_ERR_INVALID_ARG),
    (dict(num_pages=0), B.KDA_ERR_INVALID_ARG), (dict(page_tokens=24), B.KDA_ERR_UNSUPPORTED),
    (dict(dtype=2), B.KDA_ERR_INVALID_ARG), (dict(max_pages=1 << 28), B.KDA_ERR_UNSUPPORTED)])
def test_bad_caches(L, bad, status):  # noqa: F811
    assert extend(L, attention(), cache(**bad)) == status


def test_pointers_overlap_and_workspace(L):  # noqa: F811
    p, c = attention(), cache()
    assert extend(L, None, c) == extend(L, p, None) == extend(L, attention(num_seqs=3), c) == B.KDA_ERR_INVALID_ARG
    for name in ("q", "lengths", "out"):
        assert extend(L, p, c, **{name: None}) == B.KDA_ERR_INVALID_ARG
    for name in ("q", "out"):
        assert extend(L, p, c, **{name: _addr(9) + 8}) == B.KDA_ERR_INVALID_ARG
    for name in ("cu", "lengths"):
        assert extend(L, p, c, **{name: _addr(9) + 2}) == B.KDA_ERR_INVALID_ARG
        assert extend(L, p, c, **{name: _addr(3) + 16}) == B.KDA_ERR_INVALID_ARG  # inside the output
        assert extend(L, p, c, **{name: _addr(30, 1 << 25) + 64}) == B.KDA_ERR_INVALID_ARG  # inside the workspace
    assert extend(L, p, c, out=_addr(0)) == extend(L, p, c, out=_addr(22)) == B.KDA_ERR_INVALID_ARG
    need = B.kda_attention_extend_workspace_bytes(p)
    assert need > 0
    assert extend(L, p, c, ws=None) == extend(L, p, c, ws=_addr(30) + 128) == extend(L, p, c, wsb=need - 1) == B.KDA_ERR_WORKSPACE
    for inside in (0, 20, 24):
        assert extend(L, p, c, ws=_addr(inside)) == B.KDA_ERR_INVALID_ARG


def test_binding_refuses():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q, c = t(8, 4, 64), B.kda_cache_alloc(3, 16, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        B.kda_attention_extend(q.half(), c, i32(2, 1), i32(2))
    with pytest.raises(TypeError):
        B.kda_attention_extend(q, c, i32(2, 1), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.kda_attention_extend(q, c, i32(3, 1), i32(2))
    with pytest.raises(ValueError):
        B.kda_attention_extend(q, c, i32(2, 1), i32(2), cu_seqlens=i32(2))
    with pytest.raises(ValueError):
        B.kda_attention_extend(q, c, i32(2, 1), i32(2), out=t(8, 4, 32))
    with pytest.raises(ValueError):  # channels not packed
        B.kda_attention_extend(t(8, 64, 4).transpose(1, 2), c, i32(2, 1), i32(2))


def test_allocations_on_another_stream(watched):  # noqa: F811
    where, recorded = watched
    B._extend_workspace_bytes.cache_clear()
    side = Side()
    c, i32 = B.kda_cache_alloc(3, 16, 2, 64, device="cpu"), lambda *s: torch.zeros(*s, dtype=torch.int32)
    refused(B.kda_attention_extend, torch.zeros(8, 4, 64, dtype=torch.bfloat16), c, i32(2, 1), i32(2), stream=side)
    assert where == [side] * 2 and recorded == ["current"]
    B._extend_workspace_bytes.cache_clear()
