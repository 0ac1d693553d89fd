"""Rotary positions against float64 forms, alone and on the way into the 8-bit cache.

Tolerances, derived from the roundings that the kernels make (half a step relative to a value: bf16 2^-8, fp32 2^-24).
  turned values: y = a c - b s with two roundings in fp32 of terms below |a| + |b| (2^-23 of it together); the angle is off by
      2^-32 of a turn (2^-29.3 radians), by fp32's rounding of an eighth of a turn (2^-25.3), and by double's
      rounding of freq / 2 pi (2^-52 of position * freq: two roundings, of the constant and of the product); the sine and the cosine
      by a few units of fp32's last place (2^-23 each): together below 2^-21 (|a| + |b|) for |position freq| < 2^26, plus
      2^-52 |position freq| (|a| + |b|); then half a step of the io dtype.
  codes: the turned value (as above), then half a step of the code at the page's scale.
"""
import pytest
import torch

import attention_ref
import rotary_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_attention import offsets, tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def data(T, heads, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, heads, d, generator=g).to(dtype).to(DEV)


def close(got, x, rotary, pos, inverse=False):
    want = ref.turned(x, rotary, pos, inverse)
    far = float(pos.abs().max()) * max(abs(f) for f in rotary.freq[:rotary.rot_dim // 2]) if pos.numel() else 0.0
    tol = (2.0 ** -21 + 2.0 ** -52 * far) * ref.size(x, rotary) + HALF[x.dtype] * want.abs()
    bad = ~((got.detach().double().cpu() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), [tuple(i) for i in bad.nonzero()[:4].tolist()])
    assert torch.equal(got[..., rotary.rot_dim:], x[..., rotary.rot_dim:])


ROTARY = {32: [(32, False), (16, True)], 64: [(64, True), (48, False), (32, False)], 128: [(128, False), (128, True), (64, False), (80, True), (16, False)]}
LENS = [[1], [3, 1, 0, 2], [65, 0, 130, 7, 1], [1] * 70, [0, 0, 300]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,rot,adjacent", [(d, r, a) for d in ROTARY for r, a in ROTARY[d]])
def test_places_in_sequences(d, rot, adjacent, dtype):
    """Ragged sequences, beginning with these tokens or behind others; rows behind the last are left alone."""
    r = B.make_rotary(rot, adjacent=adjacent)
    for i, new in enumerate(LENS):
        T = sum(new)
        q, k = data(T + 5, 6, d, dtype, i), data(T + 5, 2, d, dtype, 50 + i)
        before = [(37 * j + 11) % 5000 for j in range(len(new))]
        lens = [a + b for a, b in zip(before, new)]
        for lengths, pos in ((None, ref.places(new, new)), (torch.tensor(lens, dtype=torch.int32, device=DEV), ref.places(lens, new))):
            qo, ko = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
            got = B.kda_rotary(r, q, k, cu_seqlens=offsets(new), lengths=lengths, q_out=qo, k_out=ko)
            assert got[0] is qo and got[1] is ko
            close(qo[:T], q[:T], r, pos)
            close(ko[:T], k[:T], r, pos)
            assert bool((qo[T:] == 3.0).all()) and bool((ko[T:] == 3.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_axes_views_in_place_and_back(dtype):
    """Three axes, views of one projection turned in place, and turned back."""
    r = B.make_rotary(96, base=500.0, sections=(12, 18, 18))
    T = 333
    x = data(T, 6 + 2 * 2, 128, dtype, 4)
    keep = x.clone()
    pos = torch.randint(-3000, 3000, (3, T), generator=torch.Generator().manual_seed(1))
    q, k = x[:, :6], x[:, 6:8]
    B.kda_rotary(r, q, k, positions=pos.to(torch.int32).to(DEV), q_out=q, k_out=k)
    close(q, keep[:, :6], r, pos)
    close(k, keep[:, 6:8], r, pos)
    assert torch.equal(x[:, 8:], keep[:, 8:])
    back, none = B.kda_rotary(r, q, positions=pos.to(torch.int32).to(DEV), inverse=True)
    assert none is None
    close(back, q, r, pos, inverse=True)
    kb = B.kda_rotary(r, k=k, positions=pos.to(torch.int32).to(DEV), inverse=True)[1]
    close(kb, k, r, pos, inverse=True)


def test_far_positions():
    """Positions up to the largest, with frequencies up to a hundred radians: the fraction of the turn is what counts."""
    r = B.make_rotary(64, freqs=tuple(100.0 / 3 ** i for i in range(32)))
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 1048576, 999999937, -1, 0]])
    q = data(6, 3, 64, torch.float32, 5)
    close(B.kda_rotary(r, q, positions=pos.to(torch.int32).to(DEV))[0], q, r, pos)


def test_gradient_is_the_turn_back():
    """The gradient of a turn against the formula's and against differences of the float64 form."""
    r = B.make_rotary(32, base=50.0, sections=(10, 6))
    T = 9
    pos = torch.randint(0, 400, (2, T), generator=torch.Generator().manual_seed(2))
    x, dy = data(T, 2, 64, torch.float32, 6), data(T, 2, 64, torch.float32, 7)
    got = B.kda_rotary(r, dy, positions=pos.to(torch.int32).to(DEV), inverse=True)[0]
    close(got, dy, r, pos, inverse=True)
    xd, w = x.double().cpu(), dy.double().cpu()
    for at in ((0, 0, 0), (4, 1, 17), (8, 0, 31), (3, 1, 40)):
        e = torch.zeros_like(xd)
        e[at] = 1e-3
        diff = ((ref.turned(xd + e, r, pos) - ref.turned(xd - e, r, pos)) * w).sum() / 2e-3
        # the form is linear: the difference is exact but for float64's rounding (2^-53 of sums of |w x| over 1152 values, / 1e-3)
        assert abs(float(got[at]) - float(diff)) < 2.0 ** -20 * float(ref.size(dy, r)[at] + w[at].abs()) + 1e-9


def test_nothing_to_turn():
    r = B.make_rotary(64)
    q = data(0, 4, 64, torch.bfloat16, 8)
    assert B.kda_rotary(r, q, q)[0].shape == (0, 4, 64)


def test_special_values_stay_with_their_pair():
    r = B.make_rotary(32)
    q = data(7, 2, 64, torch.bfloat16, 9)
    pos = torch.arange(7)[None] + 1
    clean = B.kda_rotary(r, q, positions=pos.to(torch.int32).to(DEV))[0]
    q2 = q.clone()
    q2[3, 1, 5], q2[2, 0, 60], q2[4, 1, 20] = float("nan"), float("nan"), float("inf")
    got = B.kda_rotary(r, q2, positions=pos.to(torch.int32).to(DEV))[0]
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[3, 1, [5, 21]] = hit[2, 0, 60] = hit[4, 1, [4, 20]] = True
    assert torch.equal(got[~hit], clean[~hit]) and not bool(torch.isfinite(got[hit]).any())


# ---------------------------------------------------------------- into the cache

def appended(q, k, v, old, new, page, dtype, r, pos=None, in_place=False):
    """The call's cache, turned queries and check word, from a cache filled with the tokens before."""
    N, hkv, d = len(new), k.shape[1], k.shape[2]
    lens = [a + b for a, b in zip(old, new)]
    table, pool = tables(lens, page, seed=3)
    cache = B.kda_cache_alloc(pool, page, hkv, d, dtype=dtype)
    before = data(sum(old), 2 * hkv, d, k.dtype, 77)
    if sum(old):
        B.kda_cache_append(before[:, :hkv], before[:, hkv:], cache, table, torch.tensor(old, dtype=torch.int32, device=DEV), cu_seqlens=offsets(old))
    start = B.KvCache(*[x.clone() for x in cache])
    check = torch.zeros(64, dtype=torch.int32, device=DEV)
    out = B.kda_rotary_append(r, k, v, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), q=q, positions=pos,
                              cu_seqlens=offsets(new), q_out=q if in_place else None, check=check)
    assert B.kda_workspace_status(check) == B.KDA_OK
    return start, cache, table, out


APPENDS = [([0], [1]), ([0, 0, 0], [130, 1, 33]), ([5, 64, 15, 700], [1, 1, 1, 1]), ([100, 0, 31, 16], [40, 7, 0, 300]), ([3] * 40, [2] * 40)]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("code", [torch.float8_e4m3fn, torch.int8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("d,rot,adjacent,page,axes", [(128, 128, False, 64, 0), (128, 64, True, 128, 3), (64, 64, True, 16, 0), (64, 16, False, 32, 3), (32, 32, False, 128, 0), (128, 128, False, 128, 0)])
def test_append(d, rot, adjacent, page, axes, code, io):
    r = B.make_rotary(rot, base=1000.0, adjacent=adjacent, axis=tuple(i % 3 for i in range(rot // 2)) if axes else None)
    for old, new in APPENDS:
        T, hkv = sum(new), 3
        x = data(T, 6 + 2 * hkv, d, io, d + T)
        q, k, v = x[:, :6], x[:, 6:6 + hkv], x[:, 6 + hkv:]
        lens = [a + b for a, b in zip(old, new)]
        pos = torch.randint(0, 2000, (3, T), generator=torch.Generator().manual_seed(T)) if axes else ref.places(lens, new)
        start, cache, table, out = appended(q, k, v, old, new, page, code, r, pos.to(torch.int32).to(DEV) if axes else None)
        close(out, q, r, pos)
        turned, size = ref.turned(k, r, pos), ref.size(k, r)
        want_k, want_v, want_ks, want_vs = attention_ref.append(turned, v, start, table, old, new)
        assert torch.equal(cache.v.cpu().to(torch.float64), want_v) and torch.equal(cache.v_scale.cpu().double(), want_vs)
        # the scale follows the largest turned value: the same but where that lies within fp32's error of a power's limit
        assert torch.equal(cache.k_scale.cpu().double(), want_ks)
        got = cache.k.cpu().to(torch.float64)
        # every code that this call did not write (or round again) is what it was, and the others' values are near
        at = 0
        differs = got != want_k
        for n, (a, m) in enumerate(zip(old, new)):
            for t in range(m):
                p, s = int(table[n, (a + t) // page]), (a + t) % page
                unit = cache.k_scale[p].cpu().double()[:, None]
                err = (got[p, :, s] * unit - turned[at + t]).abs()
                value = (turned[at + t] / unit).abs()
                step = torch.exp2(torch.frexp(value).exponent.double().sub(1).clamp(min=-6) - 3) if code == torch.float8_e4m3fn else torch.ones_like(value)
                assert bool((err <= 0.5 * step * unit + 2.0 ** -20 * size[at + t]).all()), (n, t)
                differs[p, :, s] = False
            at += m
        assert not bool(differs.any())


@pytest.mark.parametrize("code", [torch.float8_e4m3fn, torch.int8], ids=["e4m3", "int8"])
def test_append_without_a_turn_is_the_plain_append(code):
    """At position 0 a turn changes nothing: the same codes as kda_cache_append's, and q as it was, in place too."""
    r = B.make_rotary(128)
    old, new, hkv = [70, 0, 5], [60, 100, 1], 2
    T = sum(new)
    x = data(T, 4 + 2 * hkv, 128, torch.bfloat16, 21)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    keep = x.clone()
    pos = torch.zeros(1, T, dtype=torch.int32, device=DEV)
    start, cache, table, out = appended(q, k, v, old, new, 64, code, r, pos, in_place=True)
    assert out is q and torch.equal(x, keep)
    lens = torch.tensor([a + b for a, b in zip(old, new)], dtype=torch.int32, device=DEV)
    B.kda_cache_append(k, v, start, table, lens, cu_seqlens=offsets(new))
    for a, b in zip(start, cache):
        assert torch.equal(a.float(), b.float())


def test_append_equal_lengths_and_no_queries():
    r = B.make_rotary(64)
    N, hkv, d = 9, 2, 64
    k, v = data(N, hkv, d, torch.bfloat16, 30), data(N, hkv, d, torch.bfloat16, 31)
    old = [17 * i for i in range(N)]
    a = appended(None, k, v, old, [1] * N, 32, torch.float8_e4m3fn, r)
    lens = torch.tensor([o + 1 for o in old], dtype=torch.int32, device=DEV)
    cache = a[0]
    assert a[3] is None and B.kda_rotary_append(r, k, v, cache, a[2], lens) is None
    for x, y in zip(cache, a[1]):
        assert torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x, y.view(torch.uint8) if y.element_size() == 1 else y)


def test_bad_lengths_and_pages_are_skipped():
    """A sequence that does not fit its pages, or a page that is not there, is left out and reported; its queries turn."""
    r = B.make_rotary(64)
    new, hkv, d, page = [4, 5, 6], 2, 64, 16
    k, v, q = (data(15, h, d, torch.bfloat16, 40 + h) for h in (hkv, hkv, 4))
    table = torch.tensor([[0, 1], [2, 99], [3, 4]], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([40, 20, 20], dtype=torch.int32, device=DEV)  # 40 > 2 pages; 20 reaches the page that is not there
    cache = B.kda_cache_alloc(6, page, hkv, d)
    check = torch.zeros(64, dtype=torch.int32, device=DEV)
    out = B.kda_rotary_append(r, k, v, cache, table, lengths, q=q, cu_seqlens=offsets(new), check=check)
    assert B.kda_workspace_status(check) == B.KDA_ERR_DEVICE_CHECK
    close(out, q, r, torch.tensor([list(range(36, 40)) + list(range(15, 20)) + list(range(14, 20))]))
    used = cache.k.float().abs().sum((1, 2, 3)) > 0
    assert used.tolist() == [False, False, True, True, True, False]


def test_infinities_and_nans_set_no_scale():
    r = B.make_rotary(64)
    k, v = data(40, 1, 64, torch.float32, 50), data(40, 1, 64, torch.float32, 51)
    clean = appended(None, k, v, [0], [40], 64, torch.float8_e4m3fn, r)[1]
    k2 = k.clone()
    k2[7, 0, 3], k2[9, 0, 40] = float("nan"), float("inf")
    cache = appended(None, k2, v, [0], [40], 64, torch.float8_e4m3fn, r)[1]
    assert float(cache.k_scale.max()) <= float(clean.k_scale.max())
    assert bool(cache.k.float().isnan().any())  # NaN stays NaN in e4m3


def test_captured_and_on_another_stream():
    """The same bits when replayed from a graph and from another stream."""
    r = B.make_rotary(128)
    old, new = [100, 3, 64], [1, 1, 1]
    x = data(3, 8, 128, torch.bfloat16, 60)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    start, want, table, out = appended(q, k, v, old, new, 64, torch.float8_e4m3fn, r)
    lens = torch.tensor([a + b for a, b in zip(old, new)], dtype=torch.int32, device=DEV)
    same = lambda a, b: all(torch.equal(x.float(), y.float()) for x, y in zip(a, b))  # noqa: E731
    cache = B.KvCache(*[t.clone() for t in start])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = B.kda_rotary_append(r, k, v, cache, table, lens, q=q, stream=side)
    turned = B.kda_rotary(r, q, k, lengths=lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(cache, want) and torch.equal(got, out) and torch.equal(turned[0], out)
    cache = B.KvCache(*[t.clone() for t in start])
    q_out = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.kda_rotary_append(r, k, v, cache, table, lens, q=q, q_out=q_out)
    for a, b in zip(cache, start):
        a.copy_(b)
    graph.replay()
    assert same(cache, want) and torch.equal(q_out, out)


def test_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31."""
    r = B.make_rotary(128)
    T, heads = (1 << 31) // (128 * 64) + 300, 64
    q = torch.zeros(T, heads, 128, dtype=torch.bfloat16, device=DEV)
    q[-2:] = data(2, heads, 128, torch.bfloat16, 70)
    pos = torch.zeros(1, T, dtype=torch.int32, device=DEV)
    pos[0, -2:] = torch.tensor([12345, 54321])
    out = B.kda_rotary(r, q, positions=pos, q_out=q)[0]
    close(out[-2:], data(2, heads, 128, torch.bfloat16, 70), r, torch.tensor([[12345, 54321]]))
    assert not bool(out[:-2].any())
