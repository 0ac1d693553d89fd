"""Attention where it can go wrong, against the float64 forms: scales far apart, infinities and NaN, many tiles.

Tolerances are those of test_gpu_attention.py, whose head derives them.
"""
import pytest
import torch

import attention_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_attention import CODES, DEV, close, filled, make, offsets, same_codes, tables

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page,d,hq", [(16, 128, 1), (32, 128, 8), (64, 128, 3), (16, 64, 8), (32, 128, 12)])
def test_decode_page_scales_from_tile_to_tile(page, d, hq, dtype, code):
    """Neighbouring pages' scales differ by 2^4, over runs of many tiles a warp: each tile takes its own pages' scales."""
    lens = [5000, 3333] + [1400] * 600
    pool = -(-max(lens) // page)
    table = torch.arange(pool, dtype=torch.int32).repeat(len(lens), 1).to(DEV)  # the sequences share their pages
    c = filled(pool, 1, page, d, code, seed=page)
    even = (torch.arange(pool) % 2).float()[:, None].to(DEV)
    cache = B.KvCache(c.k, c.v, torch.exp2(-9 + 4 * even), torch.exp2(-3 - 4 * even))
    q = make(len(lens), hq, 1, d, dtype, 6)[0]
    out = B.kda_attention_decode(q, cache, table, i32(*lens))
    few = 4
    close(out[:few], ref.decode(q[:few], cache, table[:few], lens[:few]), ref.dequant(c.v, cache.v_scale), dtype, 2.0 ** -11)
    # the shorter sequences hold the same keys: one row of q at every place of the cut
    same = B.kda_attention_decode(q[2:3].expand(600, -1, -1).contiguous(), cache, table[2:], i32(*lens[2:]))
    want = ref.decode(q[2:3], cache, table[2:3], lens[2:3]).expand(600, -1, -1)
    close(same, want, ref.dequant(c.v, cache.v_scale), dtype, 2.0 ** -11)


@pytest.mark.parametrize("capacity", [0, 600], ids=["narrow_table", "wide_table"])  # many rows: one kernel or the other
@pytest.mark.parametrize("hq,window,dtype", [(4, 7, torch.bfloat16), (8, 7, torch.bfloat16), (2, 2, torch.bfloat16),
                                             (4, 7, torch.float32)], ids=["28", "56", "4", "28f32"])
def test_decode_a_row_of_q_leaves_the_others_alone(hq, window, dtype, capacity):
    """One row of q with a NaN, an infinity, or far larger or smaller than the rest: every other row stays as it was."""
    lens, page, d = [150, 95, 300], 16, 128
    table, pool = tables(lens, page, capacity=capacity)
    cache = filled(pool, 1, page, d, torch.float8_e4m3fn)
    q = make(len(lens) * window, hq, 1, d, dtype, 8)[0]
    clean = B.kda_attention_decode(q, cache, table, i32(*lens))
    v = ref.dequant(cache.v, cache.v_scale)
    for n, t, head, change in ((0, window - 1, 0, float("nan")), (1, 0, hq - 1, -float("inf")), (2, window // 2, 1, 2.0 ** 40),
                               (2, 0, 1, 2.0 ** -60), (0, window - 1, 1, 2.0 ** 90)):
        row, x = n * window + t, q.clone()
        if abs(change) < float("inf"):
            x[row, head] *= change
        else:
            x[row, head, 5] = change
        out = B.kda_attention_decode(x, cache, table, i32(*lens))
        others = torch.ones(out.shape[:2], dtype=torch.bool, device=DEV)
        others[row, head] = False
        assert torch.equal(out[others], clean[others]), (change, int((out[others] != clean[others]).sum()))
        if abs(change) < 1:
            close(out, ref.decode(x, cache, table, lens), v, dtype, 2.0 ** -11)
        elif not abs(change) < float("inf"):
            assert not out[row, head].isfinite().any()


def minus_infinity_first(d, dtype):
    """128 keys that every row scores at -inf, and more behind them: those count alone."""
    lens, hidden = [400, 150], 128
    q, k, v = make(sum(lens), 4, 2, d, dtype, 12)
    q, k = q.clone(), k.clone()
    q[:, :, 3] = q[:, :, 3].abs() + 0.1
    k[:hidden, 0, 3] = -float("inf")
    k[400:400 + hidden, 1, 3] = -float("inf")
    out = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens))
    start = 0
    for n, length in enumerate(lens):  # key head n has the hidden keys
        s = slice(start + hidden, start + length)
        heads = slice(2 * n, 2 * n + 2)
        want = ref.prefill(q[s, heads], k[s, n:n + 1], v[s, n:n + 1], [length - hidden])
        close(out[s, heads], want, v, dtype, 2.0 ** -8)
        start += length


@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefill_fp32_keys_with_infinities(d):
    """A key whose score is -inf weighs nothing; one whose score is +inf or NaN makes the rows that see it NaN."""
    minus_infinity_first(d, torch.float32)
    q, k, v = make(150, 2, 1, d, torch.float32, 16)
    q, k = q.clone(), k.clone()
    q[:, :, 3] = q[:, :, 3].abs() + 0.1
    q[:, :, 4] = 0
    clean = B.kda_attention_prefill(q, k, v)
    for bad, ch in ((float("inf"), 3), (float("nan"), 3), (-float("inf"), 4)):
        k2 = k.clone()
        k2[70, 0, ch] = bad
        out = B.kda_attention_prefill(q, k2, v)
        assert torch.equal(out[:70], clean[:70]) and bool(out[70:].isnan().all())


@pytest.mark.parametrize("copies", [1, 80], ids=["few_tiles", "many_tiles"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefill_fp32_largest_finite_values(d, copies):
    """The largest finite value in V reaches the rows that see it, as itself, and no other row."""
    top = torch.finfo(torch.float32).max
    lens = [150, 90] * copies
    q, k, v = make(sum(lens), 4, 2, d, torch.float32, 9)
    clean = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens))
    v2 = v.clone()
    v2[140, 1, 5], v2[150 + 60, 0, 7], v2[0, 0, 2] = top, -top, top
    out = B.kda_attention_prefill(q, k, v2, cu_seqlens=offsets(lens))
    same = torch.ones_like(out, dtype=torch.bool)
    same[140:150, 2:, 5] = same[150 + 60:240, :2, 7] = same[:150, :2, 2] = False
    assert torch.equal(out[same], clean[same]), int((out[same] != clean[same]).sum())
    want = ref.prefill(q[:240], k[:240], v2[:240], lens[:2])
    close(out[:240], want, v2, torch.float32, 0.0)


def test_prefill_fp32_largest_finite_keys():
    """The largest finite values in k and q: scores are what they are, here up to about 10."""
    top, lens = torch.finfo(torch.float32).max, [200]
    q, k, v = make(200, 2, 2, 64, torch.float32, 10)
    g = torch.Generator().manual_seed(1)
    x = torch.rand(200, 2, generator=g).to(DEV) * 2 - 1
    k, q = k.clone(), q.clone()
    q[:, 0, 3], k[:, 0, 3] = x[:, 0] * 1e-30, torch.where(x[:, 1] > 0, top, x[:, 1])
    q[:, 1, 3], k[:, 1, 3] = torch.where(x[:, 1] > 0, -top, x[:, 1]), x[:, 0] * 1e-30
    out = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens), scale=3e-8)
    close(out, ref.prefill(q, k, v, lens, scale=3e-8), v, torch.float32, 0.0)


def flat_tail(n, at, high, code, first):
    """A cache of one sequence's ``n`` keys of which one, at ``at``, scores ``high`` more in base 2 than the others for a q
    that is one in channel 0 (with scale ln 2); its value is zero, the others' one.  ``first``: the first page's
    values are zeros on a scale 64 times the others'."""
    page, d = 128, 128
    pages = n // page
    k, v = torch.zeros(pages, 1, page, d), torch.full((pages, 1, page, d), 64.0)
    vs = torch.full((pages, 1), 2.0 ** -6)
    k[at // page, 0, at % page, 0] = 2 * high
    v[at // page, 0, at % page] = 0
    if first:
        v[0], vs[0] = 0, 1.0
    return B.KvCache(k.to(code).to(DEV), v.to(code).to(DEV), torch.full((pages, 1), 0.5).to(DEV), vs.to(DEV))


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("hq,dtype,at,high,first", [
    (1, torch.float32, 0, 26, False), (12, torch.float32, 0, 26, False), (1, torch.float32, 256, 20, True),
    (12, torch.float32, 256, 20, True), (1, torch.bfloat16, 256, 20, True), (12, torch.bfloat16, 256, 20, True),
], ids=["f32", "f32_12", "f32_scale", "f32_12_scale", "bf16_scale", "bf16_12_scale"])
def test_decode_one_key_before_a_long_flat_tail(hq, dtype, at, high, first, code):
    """Thousands of weights far below the largest add up to something: 4095 of 2^-26 of it, or of 2^-20 after a page
    whose values are on a larger scale."""
    n, many = 4096, 2000
    cache = flat_tail(n, at, high, code, first)
    table = torch.arange(n // 128, dtype=torch.int32).repeat(many, 1).to(DEV)
    q = torch.zeros(many, hq, 128, dtype=dtype, device=DEV)
    q[:, :, 0] = 1
    ln2 = 0.6931471805599453
    out = B.kda_attention_decode(q, cache, table, i32(*[n] * many), scale=ln2)
    want = ref.decode(q[:1], cache, table[:1], [n], scale=ln2)
    assert float(want.max()) > (2.0 ** -17 if dtype == torch.float32 else 2.0 ** -11)  # not lost in the tolerance
    close(out, want.expand(many, -1, -1), ref.dequant(cache.v, cache.v_scale), dtype, 2.0 ** -11)


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
def test_decode_many_rows_one_key_before_a_long_flat_tail(code):
    """As above for the kernel that takes many rows, whose blocks of 128 keys alternate between two streams."""
    n, many, hq = 4096, 300, 28
    cache = flat_tail(n, 256, 20, code, True)
    table = torch.arange(n // 128, dtype=torch.int32).repeat(many, 1).to(DEV)
    q = torch.zeros(many, hq, 128, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1
    ln2 = 0.6931471805599453
    out = B.kda_attention_decode(q, cache, table, i32(*[n] * many), scale=ln2)
    want = ref.decode(q[:1], cache, table[:1], [n], scale=ln2)
    assert float(want.max()) > 2.0 ** -11
    close(out, want.expand(many, -1, -1), ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefill_scores_of_minus_infinity_come_first(d):
    minus_infinity_first(d, torch.bfloat16)


@pytest.mark.parametrize("capacity", [0, 600], ids=["narrow_table", "wide_table"])
def test_decode_scores_of_minus_infinity_alone(capacity):
    """A row whose every score is -inf has no weight: zeros, from either kernel, and the other rows as they were."""
    lens, page, d, hq, window = [150, 300], 16, 128, 4, 7
    table, pool = tables(lens, page, capacity=capacity)
    c = filled(pool, 1, page, d, torch.int8)
    k = c.k.clone()
    k[..., 0] = -3
    cache = B.KvCache(k, c.v, c.k_scale, c.v_scale)
    q = make(2 * window, hq, 1, d, torch.bfloat16, 13)[0]
    clean = B.kda_attention_decode(q, cache, table, i32(*lens))
    x = q.clone()
    x[9, 2, 0] = float("inf")
    out = B.kda_attention_decode(x, cache, table, i32(*lens))
    want = clean.clone()
    want[9, 2] = 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("up", [2.0 ** 13, 2.0 ** 17, 2.0 ** 45])
def test_prefill_huge_scores(up, d, dtype):
    """Scores up to 2^95, whose rounding alone is larger than fp32's exponents: the largest takes the weight."""
    lens = [300, 1, 130]
    q, k, v = make(sum(lens), 4, 2, d, dtype, 17)
    out = B.kda_attention_prefill(q * up, k * up, v, cu_seqlens=offsets(lens))
    close(out, ref.prefill(q * up, k * up, v, lens), v, dtype, 2.0 ** -8)


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("up", [2.0 ** 24, 2.0 ** 30, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("hq,window,dtype", [(2, 1, torch.bfloat16), (4, 3, torch.bfloat16), (4, 7, torch.bfloat16),
                                             (2, 2, torch.float32)], ids=["2", "12", "28", "4f32"])
def test_decode_huge_scores(hq, window, dtype, up, code):
    lens, page, d = [700, 40, 131], 32, 128
    table, pool = tables(lens, page, capacity=768)
    cache = filled(pool, 1, page, d, code, seed=9)
    q = make(len(lens) * window, hq, 1, d, dtype, 18)[0] * up
    out = B.kda_attention_decode(q, cache, table, i32(*lens))
    close(out, ref.decode(q, cache, table, lens), ref.dequant(cache.v, cache.v_scale), dtype, 2.0 ** -11)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (3, 3), (40, 2)], ids=["4of2", "3of3", "40of2"])
def test_prefill_more_tiles_than_sms(hq, hkv, d):
    """bf16, several hundred tiles: a CTA takes one after another.  NaN and infinities, in tiles of any turn, reach the rows
    that see them and no other."""
    dtype = torch.bfloat16
    lens = [5, 70, 0, 33, 131, 300] * (40 if hq == 3 else 24 if hq == 4 else 6) + [900, 1]
    q, k, v = make(sum(lens), hq, hkv, d, dtype, 14 + d, fused=True)
    out = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens))
    close(out, ref.prefill(q, k, v, lens), v, dtype, 2.0 ** -8)
    nan, inf, group = float("nan"), float("inf"), hq // hkv
    v2, want, start = v.clone(), out.clone(), 0
    for i, n in enumerate(lens):
        h, ch = i % hkv, (5 * i) % d
        rows = want[start:start + n, h * group:(h + 1) * group, ch]
        if n >= 33 and i % 3 != 2:  # one odd value, late in the sequence
            at, bad = n - 1 - i % 20, (nan, inf, -inf)[i % 5 % 3]
            v2[start + at, h, ch] = bad
            rows[at:] = bad
        elif n >= 131:  # one of each sign
            v2[start + n // 2, h, ch], v2[start + n - 3, h, ch] = inf, -inf
            rows[n // 2:], rows[n - 3:] = inf, nan
        start += n
    bad = B.kda_attention_prefill(q, k, v2, cu_seqlens=offsets(lens))
    same = (bad == want) | (bad.isnan() & want.isnan())
    assert bool(same.all()), (int((~same).sum()), [tuple(i) for i in (~same).nonzero()[:4].tolist()])
    # and the same again: nothing is left over
    assert torch.equal(out, B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("count,hkv,page,d", [(150, 9, 16, 64), (230, 9, 16, 128), (60, 17, 64, 32), (420, 5, 128, 128)])
def test_append_many_pages_and_heads(count, hkv, page, d, code, dtype):
    """Pages enough that a CTA takes several heads one after another, the last group of heads smaller than the others;
    partly filled pages, some of which grow."""
    before = [(7 * i) % (2 * page) for i in range(count)]
    fresh = [(13 * i) % min(2 * page + 9, 60) for i in range(count)]
    table, pool = tables([a + b for a, b in zip(before, fresh)], page)
    cache = filled(pool, hkv, page, d, code, seed=3)
    g = torch.Generator().manual_seed(15)
    size = torch.exp2(torch.randint(-6, 7, (sum(fresh), 1, 1), generator=g).float())
    kv = (torch.randn(sum(fresh), 2 * hkv, d, generator=g) * size).to(dtype)
    kv[::97, 0, 3], kv[::89, hkv, 5] = float("inf"), float("nan")
    kv = kv.to(DEV)
    k, v = kv[:, :hkv], kv[:, hkv:]
    want = ref.append(k, v, cache, table, before, fresh)
    check = torch.zeros(64, dtype=torch.int32, device=DEV)
    B.kda_cache_append(k, v, cache, table, i32(*[a + b for a, b in zip(before, fresh)]), cu_seqlens=offsets(fresh), check=check)
    same_codes(cache, want)
    assert B.kda_workspace_status(check) == B.KDA_OK


@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefill_waits_that_give_up_show(monkeypatch, d):
    """bf16: rows that a given-up wait left unfinished are NaN, all of them where no wait is tried; the next call is right."""
    lens = [900, 70, 131, 1, 300] * 24
    q, k, v = make(sum(lens), 8, 4, d, torch.bfloat16, 19)
    clean = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens))
    for tries in ("0", "1", "3"):
        monkeypatch.setenv("KDA_DEBUG_HANDOFF_TRIES", tries)
        out = torch.full_like(clean, 123.0)
        B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens), out=out)
        torch.cuda.synchronize()
        monkeypatch.delenv("KDA_DEBUG_HANDOFF_TRIES")
        lost = out.isnan().all(-1)
        assert torch.equal(out[~lost], clean[~lost]), (tries, int((out == 123.0).all(-1).sum()))
        assert tries != "0" or bool(lost.all())
        assert torch.equal(B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens)), clean)


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("up", [2.0 ** 8, 2.0 ** 20, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("hq,window", [(2, 1), (4, 7)], ids=["2", "28"])
def test_decode_huge_key_scales(hq, window, up, code):
    """Huge scores from the keys' scales, on some of the pages alone: those of the others count for nothing or all."""
    lens, page, d = [700, 40, 131], 32, 128
    table, pool = tables(lens, page, capacity=768)
    c = filled(pool, 1, page, d, code, seed=9)
    ks = c.k_scale.clone()
    ks[::3] *= up
    cache = B.KvCache(c.k, c.v, ks, c.v_scale)
    q = make(len(lens) * window, hq, 1, d, torch.bfloat16, 18)[0]
    out = B.kda_attention_decode(q, cache, table, i32(*lens))
    close(out, ref.decode(q, cache, table, lens), ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)
