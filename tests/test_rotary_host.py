"""What the rotary entry points refuse on the host, before any launch (no GPU: the fake addresses are never
dereferenced), and the float64 form that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import rotary_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_abi_host import L, _addr  # noqa: F401  (fixture)
from test_attention_host import BAD, BAD_Q, attention, cache
from test_stream_allocations import Side, refused, watched  # noqa: F401  (fixture)


def descriptor(**kw):
    r = B.KdaRotary.from_buffer_copy(B.make_rotary(64))  # equal arguments share one: change a copy
    for name, x in kw.items():
        if name in ("axis", "freq"):
            getattr(r, name)[x[0]] = x[1]
        else:
            setattr(r, name, x)
    return r


def rotary(L, p, r, inverse=0, **over):
    names = ("q", "k", "cu", "lengths", "positions", "q_out", "k_out")
    ptr = {n: _addr(i) for i, n in enumerate(names)}
    ptr.update(cu=None, lengths=None, positions=None)
    ptr.update(over)
    return L.kda_rotary(*[ptr[n] for n in names], ctypes.byref(p) if p else None, ctypes.byref(r) if r else None, inverse, None)


def append(L, p, c, r, **over):
    names = ("q", "k", "v", "cu", "lengths", "positions", "q_out")
    ptr = {n: _addr(i) for i, n in enumerate(names)}
    ptr.update(cu=None, positions=None, check=None)
    ptr.update(over)
    return L.kda_rotary_append(*[ptr[n] for n in names], ctypes.byref(c) if c else None, ctypes.byref(p) if p else None,
                               ctypes.byref(r) if r else None, ptr["check"], None)


@pytest.mark.parametrize("bad,status", [x for x in BAD + BAD_Q if "scale" not in x[0]])
def test_bad_descriptors(L, bad, status):  # noqa: F811
    assert rotary(L, attention(**bad), descriptor()) == status
    assert append(L, attention(**bad), cache(), descriptor()) == status


@pytest.mark.parametrize("bad,status", [
    (dict(rot_dim=0), B.KDA_ERR_INVALID_ARG), (dict(rot_dim=128), B.KDA_ERR_INVALID_ARG),
    (dict(rot_dim=24), B.KDA_ERR_UNSUPPORTED), (dict(axes=0), B.KDA_ERR_INVALID_ARG), (dict(axes=5), B.KDA_ERR_INVALID_ARG),
    (dict(adjacent=2), B.KDA_ERR_INVALID_ARG), (dict(reserved=1), B.KDA_ERR_INVALID_ARG),
    (dict(axis=(31, 1)), B.KDA_ERR_INVALID_ARG), (dict(freq=(3, math.inf)), B.KDA_ERR_INVALID_ARG),
    (dict(freq=(0, math.nan)), B.KDA_ERR_INVALID_ARG), (dict(freq=(0, -65537.0)), B.KDA_ERR_INVALID_ARG)])
def test_bad_rotary(L, bad, status):  # noqa: F811
    assert rotary(L, attention(), descriptor(**bad)) == status
    assert append(L, attention(), cache(), descriptor(**bad)) == status


def test_null_descriptors(L):  # noqa: F811
    assert rotary(L, None, descriptor()) == rotary(L, attention(), None) == B.KDA_ERR_INVALID_ARG
    assert append(L, None, cache(), descriptor()) == append(L, attention(), None, descriptor()) == B.KDA_ERR_INVALID_ARG
    assert append(L, attention(), cache(), None) == B.KDA_ERR_INVALID_ARG
    assert rotary(L, attention(), descriptor(), inverse=2) == B.KDA_ERR_INVALID_ARG
    assert rotary(L, attention(num_seqs=3), descriptor()) == append(L, attention(num_seqs=3), cache(), descriptor()) == B.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [0.0, -1.0, math.nan])
def test_scale_is_not_used(L, scale):  # noqa: F811
    good = rotary(L, attention(), descriptor())
    assert good != B.KDA_ERR_INVALID_ARG and rotary(L, attention(scale=scale), descriptor()) == good
    good = append(L, attention(), cache(), descriptor())
    assert good != B.KDA_ERR_INVALID_ARG and append(L, attention(scale=scale), cache(), descriptor()) == good


def test_pointers_and_overlap(L):  # noqa: F811
    p, r, c = attention(), descriptor(), cache()
    for name in ("q", "k", "q_out", "k_out"):  # a tensor and its output come together, on 16 bytes
        assert rotary(L, p, r, **{name: None}) == B.KDA_ERR_INVALID_ARG
        assert rotary(L, p, r, **{name: _addr(9) + 8}) == B.KDA_ERR_INVALID_ARG
    assert rotary(L, p, r, q=None, k=None, q_out=None, k_out=None) == B.KDA_ERR_INVALID_ARG
    for name in ("cu", "lengths", "positions"):
        assert rotary(L, p, r, **{name: _addr(9) + 2}) == B.KDA_ERR_INVALID_ARG
        assert rotary(L, p, r, **{name: _addr(5) + 16}) == B.KDA_ERR_INVALID_ARG  # inside an output
    assert rotary(L, p, r, q_out=_addr(0) + 64) == B.KDA_ERR_INVALID_ARG   # over its input, not in place
    assert rotary(L, p, r, k_out=_addr(0)) == B.KDA_ERR_INVALID_ARG
    assert rotary(L, p, r, k_out=_addr(5)) == B.KDA_ERR_INVALID_ARG
    # in place among the views of one projection: rows that touch are refused
    wide = attention(q_stride=512, k_stride=512)
    assert rotary(L, wide, r, q_out=_addr(0), k=_addr(0) + 128, k_out=_addr(0) + 128) == B.KDA_ERR_INVALID_ARG
    assert rotary(L, wide, r, q_out=_addr(0), k=_addr(0) + 512) == B.KDA_ERR_INVALID_ARG  # q in place, k's rows are read between
    for name in ("k", "v", "lengths", "q", "q_out"):
        assert append(L, p, c, r, **{name: None}) == B.KDA_ERR_INVALID_ARG
        assert append(L, p, c, r, **{name: _addr(21) + 64}) == B.KDA_ERR_INVALID_ARG  # inside the cache
    assert append(L, p, c, r, positions=_addr(20) + 64) == B.KDA_ERR_INVALID_ARG
    for name in ("k", "v", "lengths", "cu", "positions", "check"):
        assert append(L, p, c, r, **{name: _addr(6)}) == B.KDA_ERR_INVALID_ARG  # the turned queries
    assert append(L, p, c, r, check=_addr(9) + 4) == B.KDA_ERR_INVALID_ARG
    assert append(L, p, c, r, q_out=_addr(0), k=_addr(0) + 128) == B.KDA_ERR_INVALID_ARG
    assert append(L, p, c, r, q_out=_addr(0), lengths=_addr(0) + 128) == B.KDA_ERR_INVALID_ARG


def test_make_rotary():
    r = B.make_rotary(64, base=500.0, sections=(8, 12, 12))
    assert r.axes == 3 and list(r.axis[:32]) == [0] * 8 + [1] * 12 + [2] * 12
    assert all(abs(r.freq[i] - 500.0 ** (-i / 32)) < 1e-15 for i in range(32))
    assert B.make_rotary(32, axis=tuple(i % 3 for i in range(16))).axes == 3
    assert list(B.make_rotary(16, freqs=tuple(range(8))).freq[:8]) == list(range(8))
    for bad in (dict(rot_dim=15), dict(rot_dim=130), dict(rot_dim=64, sections=(8, 8)), dict(rot_dim=64, sections=(-1, 33)),
                dict(rot_dim=16, axis=(0,) * 7), dict(rot_dim=16, axis=(4,) * 8), dict(rot_dim=16, freqs=(1.0,)),
                dict(rot_dim=16, sections=(8,), axis=(0,) * 8), dict(rot_dim=16, sections=(2, 2, 2, 1, 1))):
        with pytest.raises(ValueError):
            B.make_rotary(**bad)


def test_binding_refuses():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    r, q, k = B.make_rotary(64), t(8, 4, 64), t(8, 2, 64)
    with pytest.raises(ValueError):
        B.kda_rotary(r)
    with pytest.raises(TypeError):
        B.kda_rotary(r, q.half())
    with pytest.raises(TypeError):
        B.kda_rotary(r, q, k.float())
    with pytest.raises(ValueError):
        B.kda_rotary(r, q, k[:7])
    with pytest.raises(ValueError):
        B.kda_rotary(r, q, positions=i32(2, 8))
    with pytest.raises(ValueError):
        B.kda_rotary(r, q, cu_seqlens=i32(3), lengths=i32(3))
    with pytest.raises(ValueError):  # neither packed nor q itself
        B.kda_rotary(r, q, q_out=t(16, 4, 64)[::2])
    c = B.kda_cache_alloc(3, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        B.kda_rotary_append(r, k, k, c, i32(8, 1), i32(8), q=q[:5])
    with pytest.raises(ValueError):
        B.kda_rotary_append(r, k, k, c, i32(8, 1), i32(8), positions=i32(8))
    with pytest.raises(TypeError):
        B.kda_rotary_append(r, k, k, c, i32(8, 1), torch.zeros(8, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.kda_rotary_append(r, k, k, c, i32(8, 1), i32(8), check=i32(1))


def test_allocations_on_another_stream(watched):  # noqa: F811
    where, recorded = watched
    side, r = Side(), B.make_rotary(64)
    q, k = torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    cache_, i32 = B.kda_cache_alloc(3, 16, 2, 64, device="cpu"), lambda *s: torch.zeros(*s, dtype=torch.int32)
    refused(B.kda_rotary, r, q, k, stream=side)
    refused(B.kda_rotary_append, r, k, k, cache_, i32(8, 1), i32(8), q=q, stream=side)
    assert where == [side] * 3 and recorded == ["current"] * 3


def test_reference_is_the_formula():
    """Pairs as complex numbers against sines and cosines written out; back again; and a far position."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 2, 32, generator=g, dtype=torch.float64)
    for adjacent in (False, True):
        r = B.make_rotary(16, base=100.0, axis=(0, 1, 0, 1, 0, 1, 1, 0), adjacent=adjacent)
        pos = torch.tensor([[0, 1, 2, -3, 4], [7, 7, 0, 5, 1000000]])
        y = ref.turned(x, r, pos)
        for t in range(5):
            for i in range(8):
                a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + 8)
                w = float(pos[r.axis[i], t]) * r.freq[i]
                want = x[t, 1, a] * math.cos(w) - x[t, 1, b] * math.sin(w)
                assert abs(float(y[t, 1, a] - want)) < 1e-9
                assert abs(float(y[t, 1, b] - (x[t, 1, b] * math.cos(w) + x[t, 1, a] * math.sin(w)))) < 1e-9
        assert torch.equal(y[..., 16:], x[..., 16:])
        assert torch.allclose(ref.turned(y, r, pos, inverse=True), x, atol=1e-14)
    one = B.make_rotary(16, freqs=(1.0,) * 8)  # 710 radians are 113 turns and 6.03e-5 less
    far = ref.angles(one, torch.tensor([[710, 2 ** 31 - 1]]))
    assert abs(float(far[0, 0]) - (710 - 113 * 2 * math.pi)) < 1e-12
    # 2 pi in 64 bits is off by at most 2^-62, and taken 2^31 / 2 pi times
    assert abs(math.sin(float(far[1, 0])) - math.sin(2 ** 31 - 1)) < 2.0 ** -33
