"""Queries turned in place on the way into the cache, as views of one projection with k and v, with k alone or with v alone:
what the call gives out of place, bit for bit, and no other row changed."""
import pytest
import torch

from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_attention import offsets, tables
from test_gpu_rotary import DEV, data

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inside", ["kv", "k", "v"])
@pytest.mark.parametrize("new", [[1] * 40, [300, 0, 77, 1]], ids=["tokens", "prompts"])
def test_in_place(new, inside, io):
    hq, hkv, d, page = 6, 2, 64, 32
    r = B.make_rotary(48, base=700.0)
    T, lens = sum(new), [n + 11 * i for i, n in enumerate(new)]
    x = data(T, hq + len(inside) * hkv + 1, d, io, 1)  # one more head that nothing reads or writes
    q, at, parts = x[:, 1:1 + hq], 1 + hq, {}
    for name in "kv":
        if name in inside:
            parts[name], at = x[:, at:at + hkv], at + hkv
        else:
            parts[name] = data(T, hkv, d, io, 2)
    table, pool = tables(lens, page, seed=4)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    call = lambda cache, **kw: B.kda_rotary_append(r, parts["k"], parts["v"], cache, table, lengths, q=q, cu_seqlens=offsets(new), **kw)  # noqa: E731
    caches = [B.kda_cache_alloc(pool, page, hkv, d) for _ in range(2)]
    keep = x.clone()
    want = call(caches[0])
    assert torch.equal(x, keep)
    got = call(caches[1], q_out=q)
    assert got is q and torch.equal(q, want)
    x[:, 1:1 + hq] = keep[:, 1:1 + hq]
    assert torch.equal(x, keep)
    for a, b in zip(*caches):
        assert torch.equal(a.float(), b.float())
