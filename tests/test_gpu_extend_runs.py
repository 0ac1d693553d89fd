"""Units whose key tiles one CTA takes in several runs (512 tiles each): joined right, whole and in pieces, with keys that
few rows see and NaN in any run.

Tolerances are those of test_gpu_extend.py for 2^16 keys, which a run does not pass, and two more roundings in fp32 a run."""
import pytest
import torch

import attention_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_attention import filled, offsets
from test_gpu_extend import DEV, IO, close

pytestmark = pytest.mark.gpu
PAGE, POOL = 128, 40


def repeated(keys, seed, hkv=2, d=64, code=torch.int8):
    """A cache of POOL pages that a sequence's table takes over and over, and the table."""
    c = filled(POOL + 1, hkv, PAGE, d, code, seed)
    table = (torch.arange(-(-keys // PAGE), dtype=torch.int32) * 7 % POOL).to(DEV)
    return c, table


def want_of(q, cache, table, keys, new):
    """Each page's keys are weighed by how often a row sees them."""
    hq, d = q.shape[1:]
    hkv = cache.k.shape[1]
    ids = table.long().cpu()
    out = torch.zeros(q.shape, dtype=torch.float64)
    kd, vd = ref.dequant(cache.k, cache.k_scale), ref.dequant(cache.v, cache.v_scale)
    for t in range(new):
        seen = keys - new + t + 1
        whole, rest = seen // PAGE, seen % PAGE
        often = torch.bincount(ids[:whole], minlength=POOL + 1).double()[:, None].repeat(1, PAGE)
        if rest:
            often[ids[whole], :rest] += 1
        often = often.reshape(-1)
        for h in range(hkv):
            rows = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            z = q[t, rows].double().cpu() @ kd[:, h].reshape(-1, d).T * d ** -0.5
            z = z.masked_fill(often == 0, -float("inf"))
            p = torch.exp(z - z.amax(1, keepdim=True)) * often
            out[t, rows] = (p / p.sum(1, keepdim=True)) @ vd[:, h].reshape(-1, d)
    return out


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
@pytest.mark.parametrize("keys,new,many", [(70_001, 150, 80), (65_700, 1, 90), (140_000, 40, 80), (13_000_123, 130, 1), (13_000_000, 1, 1)],
                         ids=["whole", "tokens", "three_runs", "pieces", "one_token_pieces"])
def test_runs(keys, new, many, io):
    """Units for every SM that one CTA holds, and few units in pieces of two runs each."""
    c, table = repeated(keys, seed=keys % 97)
    g = torch.Generator().manual_seed(1)
    hq = 4
    q = (1.5 * torch.randn(new, hq, 64, generator=g)).to(io).to(DEV)
    lengths = torch.full((many,), keys, dtype=torch.int32, device=DEV)
    cu = offsets([new] * many)
    call = lambda x: B.kda_attention_extend(q.repeat(many, 1, 1), x, table.repeat(many, 1), lengths, cu_seqlens=cu)  # noqa: E731
    out = call(c).view(many, new, hq, 64)
    assert torch.equal(out, call(c).view(many, new, hq, 64))
    want = want_of(q, c, table, keys, new)
    for n in (0, many // 3, many - 1):
        close(out[n], want, c, 1 << 16)


def test_nans_in_any_run():
    """A NaN code among values: the channel of every row that sees it, whichever run it lies in, and nothing else."""
    keys, new, many = 140_000, 150, 80
    c, table = repeated(keys, seed=3, code=torch.float8_e4m3fn)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(new, 4, 64, generator=g).bfloat16().to(DEV).repeat(many, 1, 1)
    lengths, cu = torch.full((many,), keys, dtype=torch.int32, device=DEV), offsets([new] * many)
    for at in (300, 100_000, keys - 101, keys - 1):
        t = table.clone()
        c.v[POOL], c.k[POOL] = c.v[int(t[at // PAGE])], c.k[int(t[at // PAGE])]
        c.v_scale[POOL], c.k_scale[POOL] = c.v_scale[int(t[at // PAGE])], c.k_scale[int(t[at // PAGE])]
        t[at // PAGE] = POOL  # a page of its own
        clean = B.kda_attention_extend(q, c, t.repeat(many, 1), lengths, cu_seqlens=cu).view(many, new, 4, 64)
        v = c.v.clone()
        v.view(torch.uint8)[POOL, 1, at % PAGE, 9] = 0x7F
        out = B.kda_attention_extend(q, B.KvCache(c.k, v, c.k_scale, c.v_scale), t.repeat(many, 1), lengths, cu_seqlens=cu).view(many, new, 4, 64)
        want = clean.clone()
        want[:, max(0, at - (keys - new)):, 2:, 9] = float("nan")
        same = (out == want) | (out.isnan() & want.isnan())
        assert bool(same.all()), (at, [tuple(i) for i in (~same).nonzero()[:4].tolist()])


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
def test_the_longest_table(io):
    """A sequence of 2^31 - 128 keys, as many as the largest table of its pages holds: places of its units pass 32 bits."""
    keys, new = 2 ** 31 - 128, 2
    c, table = repeated(keys, seed=5, d=32)
    assert table.numel() == 2 ** 24 - 1
    q = torch.randn(new, 4, 32, generator=torch.Generator().manual_seed(3)).to(io).to(DEV)
    ws = torch.zeros(B.kda_attention_extend_workspace_bytes(B.KdaAttention(1, new, 4, 2, 32, B._IO[io], 1.0, 0, 0, 0)), dtype=torch.uint8, device=DEV)
    out = B.kda_attention_extend(q, c, table[None], torch.tensor([keys], dtype=torch.int32, device=DEV), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_OK
    close(out, want_of(q, c, table, keys, new), c, 1 << 16)
