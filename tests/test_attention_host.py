"""What the attention entry points refuse on the host, before any launch (no GPU: the fake addresses
are never dereferenced), and the float64 forms that the GPU tests compare with."""
import ctypes

import pytest
import torch

import attention_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_abi_host import L, _addr  # noqa: F401  (fixture)


def attention(**kw):
    base = dict(num_seqs=2, total_tokens=64, num_heads=4, num_kv_heads=2, head_dim=64, io_dtype=B.KDA_BF16, scale=0.125,
                q_stride=0, k_stride=0, v_stride=0)
    base.update(kw)
    return B.KdaAttention(*[base[n] for n, _ in B.KdaAttention._fields_])


def cache(**kw):
    base = dict(k=_addr(20), v=_addr(21), k_scale=_addr(22), v_scale=_addr(23), block_table=_addr(24), num_pages=100,
                page_tokens=16, max_pages=8, dtype=B.KDA_CACHE_E4M3)
    base.update(kw)
    return B.KdaCache(*[base[n] for n, _ in B.KdaCache._fields_])


def prefill(L, p, **over):
    ptr = {n: _addr(i) for i, n in enumerate(("q", "k", "v", "cu", "out"))}
    ptr["cu"] = None
    ptr.update(over)
    return L.kda_attention_prefill(*[ptr[n] for n in ("q", "k", "v", "cu", "out")], ctypes.byref(p) if p else None, None)


def append(L, p, c, **over):
    ptr = {n: _addr(i) for i, n in enumerate(("k", "v", "cu", "lengths", "check"))}
    ptr["cu"] = None
    ptr.update(over)
    return L.kda_cache_append(ptr["k"], ptr["v"], ptr["cu"], ptr["lengths"], ctypes.byref(c) if c else None,
                              ctypes.byref(p) if p else None, ptr["check"], None)


def decode(L, p, c, ws=_addr(30, 1 << 25), wsb=1 << 26, **over):
    ptr = {n: _addr(i) for i, n in enumerate(("q", "lengths", "out"))}
    ptr.update(over)
    return L.kda_attention_decode(ptr["q"], ptr["lengths"], ctypes.byref(c) if c else None, ptr["out"],
                                  ctypes.byref(p) if p else None, ws, ctypes.c_size_t(wsb), None)


BAD = [
    (dict(num_seqs=0), B.KDA_ERR_INVALID_ARG), (dict(total_tokens=-2), B.KDA_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), B.KDA_ERR_INVALID_ARG), (dict(io_dtype=5), B.KDA_ERR_INVALID_ARG),
    (dict(head_dim=0), B.KDA_ERR_INVALID_ARG), (dict(head_dim=96), B.KDA_ERR_UNSUPPORTED),
    (dict(head_dim=256), B.KDA_ERR_UNSUPPORTED), (dict(k_stride=-128), B.KDA_ERR_INVALID_ARG),
    (dict(total_tokens=1 << 31), B.KDA_ERR_UNSUPPORTED),
]
BAD_Q = [
    (dict(num_heads=5), B.KDA_ERR_INVALID_ARG), (dict(num_heads=0), B.KDA_ERR_INVALID_ARG),
    (dict(scale=0.0), B.KDA_ERR_INVALID_ARG), (dict(scale=float("nan")), B.KDA_ERR_INVALID_ARG),
    (dict(scale=-1.0), B.KDA_ERR_INVALID_ARG), (dict(num_heads=258, num_kv_heads=2), B.KDA_ERR_UNSUPPORTED),
    (dict(q_stride=255), B.KDA_ERR_INVALID_ARG), (dict(q_stride=260), B.KDA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("bad,status", BAD + BAD_Q)
def test_bad_descriptors(L, bad, status):
    p = attention(**bad)
    assert prefill(L, p) == status
    assert decode(L, p, cache()) == status
    assert (B.kda_attention_decode_workspace_bytes(p) == 0) == ("q_stride" not in bad or bad["q_stride"] < 0)
    if (bad, status) in BAD:
        assert append(L, p, cache()) == status


def test_null_descriptors(L):
    assert prefill(L, None) == append(L, None, cache()) == decode(L, None, cache()) == B.KDA_ERR_INVALID_ARG
    assert append(L, attention(), None) == decode(L, attention(), None) == B.KDA_ERR_INVALID_ARG


def test_unequal_lengths_need_offsets(L):
    p = attention(num_seqs=3)
    assert prefill(L, p) == append(L, p, cache()) == decode(L, p, cache()) == B.KDA_ERR_INVALID_ARG
    assert decode(L, attention(num_seqs=65), cache()) == B.KDA_ERR_INVALID_ARG  # no token of some sequence


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), B.KDA_ERR_INVALID_ARG), (dict(v_scale=None), B.KDA_ERR_INVALID_ARG),
    (dict(block_table=None), B.KDA_ERR_INVALID_ARG), (dict(k=_addr(20) + 8), B.KDA_ERR_INVALID_ARG),
    (dict(k_scale=_addr(22) + 2), B.KDA_ERR_INVALID_ARG), (dict(num_pages=0), B.KDA_ERR_INVALID_ARG),
    (dict(max_pages=0), B.KDA_ERR_INVALID_ARG), (dict(page_tokens=0), B.KDA_ERR_INVALID_ARG),
    (dict(page_tokens=24), B.KDA_ERR_UNSUPPORTED), (dict(page_tokens=256), B.KDA_ERR_UNSUPPORTED),
    (dict(dtype=2), B.KDA_ERR_INVALID_ARG), (dict(max_pages=1 << 28), B.KDA_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 30), B.KDA_ERR_UNSUPPORTED)])
def test_bad_caches(L, bad, status):
    assert append(L, attention(), cache(**bad)) == status
    assert decode(L, attention(), cache(**bad)) == status


def test_pointers_and_overlap(L):
    p, c = attention(), cache()
    for name in ("q", "k", "v", "out"):
        assert prefill(L, p, **{name: None}) == B.KDA_ERR_INVALID_ARG
        assert prefill(L, p, **{name: _addr(9) + 8}) == B.KDA_ERR_INVALID_ARG
    assert prefill(L, p, out=_addr(0)) == B.KDA_ERR_INVALID_ARG
    assert prefill(L, p, cu=_addr(4) + 16) == B.KDA_ERR_INVALID_ARG  # offsets inside the output
    # the whole strided range counts: k and v as views of one projection of which out is a part
    wide = attention(q_stride=512, k_stride=512, v_stride=512)
    assert prefill(L, wide, out=_addr(0) + 63 * 1024) == B.KDA_ERR_INVALID_ARG
    for name in ("k", "v", "lengths"):
        assert append(L, p, c, **{name: None}) == B.KDA_ERR_INVALID_ARG
        assert append(L, p, c, **{name: _addr(21) + 64}) == B.KDA_ERR_INVALID_ARG  # inside the cache
    assert append(L, p, c, check=_addr(4) + 4) == B.KDA_ERR_INVALID_ARG
    assert append(L, p, cache(v=_addr(20))) == B.KDA_ERR_INVALID_ARG
    for name in ("q", "lengths", "out"):
        assert decode(L, p, c, **{name: None}) == B.KDA_ERR_INVALID_ARG
    assert decode(L, p, c, out=_addr(0)) == B.KDA_ERR_INVALID_ARG
    assert decode(L, p, c, out=_addr(22)) == B.KDA_ERR_INVALID_ARG
    assert decode(L, p, c, lengths=_addr(2) + 4) == B.KDA_ERR_INVALID_ARG
    need = B.kda_attention_decode_workspace_bytes(p)
    assert decode(L, p, c, ws=None) == B.KDA_ERR_WORKSPACE
    assert decode(L, p, c, ws=_addr(30) + 128) == B.KDA_ERR_WORKSPACE
    assert decode(L, p, c, wsb=need - 1) == B.KDA_ERR_WORKSPACE
    assert decode(L, p, c, ws=_addr(1)) == B.KDA_ERR_INVALID_ARG


def test_binding_refuses():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    q, k = t(8, 4, 64), t(8, 2, 64)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(TypeError):
        B.kda_attention_prefill(q.half(), k.half(), k.half())
    with pytest.raises(TypeError):
        B.kda_attention_prefill(q, k.float(), k)
    with pytest.raises(ValueError):
        B.kda_attention_prefill(q, k, t(8, 3, 64))
    with pytest.raises(ValueError):
        B.kda_attention_prefill(q, k[:7], k)
    with pytest.raises(ValueError):  # channels not packed
        B.kda_attention_prefill(t(8, 64, 4).transpose(1, 2), k, k)
    with pytest.raises(ValueError):  # overlapping tokens
        B.kda_attention_prefill(torch.zeros(600, dtype=torch.bfloat16).as_strided((8, 4, 64), (32, 64, 1)), k, k)
    with pytest.raises(TypeError):
        B.kda_attention_prefill(q, k, k, cu_seqlens=torch.zeros(3, dtype=torch.int64))
    c = B.kda_cache_alloc(3, 16, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        B.kda_cache_append(k, k, B.KvCache(c.k.view(torch.uint8), c.v, c.k_scale, c.v_scale), i32(8, 1), i32(8))
    with pytest.raises(TypeError):
        B.kda_cache_append(k, k, c, i32(8, 1), torch.zeros(8, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.kda_cache_append(k, k, c, i32(7, 1), i32(8))
    with pytest.raises(ValueError):
        B.kda_cache_append(k, k, c, i32(8, 1), i32(8), check=i32(1))
    with pytest.raises(ValueError):
        B.kda_attention_decode(q, B.KvCache(c.k, c.v, c.k_scale[:2], c.v_scale), i32(8, 1), i32(8))
    with pytest.raises(ValueError):
        B.kda_attention_decode(q, c, i32(8), i32(8))


def test_reference_rounding_matches_torch():
    """The cache reference's rounding is e4m3's: torch's own conversion within its range."""
    x = torch.cat([torch.randn(4000, generator=torch.Generator().manual_seed(0)) * 2.0 ** e for e in range(-12, 9)]).clamp(-448, 448)
    assert torch.equal(ref.nearest(x.double(), torch.float8_e4m3fn), x.to(torch.float8_e4m3fn).double())


def test_reference_rows_are_what_a_loop_gives():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 2, 8, generator=g, dtype=torch.float64) for n in (6, 6, 6))
    got = ref.prefill(q, k, v, [4, 0, 2], scale=0.5)
    for t in range(6):
        s = 0 if t < 4 else 4
        for h in range(2):
            w = torch.stack([torch.exp(0.5 * (q[t, h] * k[j, h]).sum()) for j in range(s, t + 1)])
            want = sum(w[j - s] * v[j, h] for j in range(s, t + 1)) / w.sum()
            assert torch.allclose(got[t, h], want, atol=1e-14)
    assert torch.equal(ref.rows(q[:, 0], k[:, 0], v[:, 0], [0, -1, 1, 2, 3, 6], 1.0)[:2], torch.zeros(2, 8, dtype=torch.float64))
