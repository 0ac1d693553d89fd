"""Chunks over the cache at its far ends: pages whose offsets pass 32 bits, and calls in flight at once.

Tolerances as in test_gpu_extend.py."""
import pytest
import torch

from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_extend import DEV, IO, case, close, want_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
def test_pages_past_32_bits(io):
    """The call's pages lie at the end of pools of 4.5 GB each, byte offsets past 2^32."""
    lens, new = [300, 129], [70, 1]
    q, small, table, lengths = case(lens, new, 8, 4, 128, 128, torch.float8_e4m3fn, io, seed=3)
    pages, own = 69000, small.k.shape[0]
    codes = [torch.empty((pages, 4, 128, 128), dtype=small.k.dtype, device=DEV) for _ in range(2)]
    scales = [torch.ones(pages, 4, device=DEV) for _ in range(2)]
    for whole, part in zip(codes + scales, small):
        whole[pages - own:] = part
    far = torch.where(table >= 0, table + pages - own, table)
    got = B.kda_attention_extend(q, B.KvCache(*codes, *scales), far, lengths, cu_seqlens=torch.tensor([0, 70, 71], dtype=torch.int32, device=DEV))
    close(got, want_of(q, small, table, lens, new), small, max(lens))


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, give what they give one after the other, and so do two captured
    ones replayed side by side."""
    calls = [case([900, 333], [200, 40], 8, 2, 128, 64, torch.float8_e4m3fn, torch.bfloat16, seed=4),
             case([40, 2100], [40, 17], 8, 2, 64, 16, torch.int8, torch.bfloat16, seed=5)]
    cu = [torch.tensor([0, 200, 240], dtype=torch.int32, device=DEV), torch.tensor([0, 40, 57], dtype=torch.int32, device=DEV)]
    want = [B.kda_attention_extend(q, c, t, n, cu_seqlens=x) for (q, c, t, n), x in zip(calls, cu)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, ((q, c, t, n), x) in enumerate(zip(calls, cu)):
            with torch.cuda.stream(streams[i]):
                got[i].append(B.kda_attention_extend(q, c, t, n, cu_seqlens=x))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    graphs, outs = [], []
    for i, ((q, c, t, n), x) in enumerate(zip(calls, cu)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=streams[i]):
            outs.append(B.kda_attention_extend(q, c, t, n, cu_seqlens=x))
    for y in outs:
        y.zero_()
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            for _ in range(3):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], want[i]) for i in range(2))
