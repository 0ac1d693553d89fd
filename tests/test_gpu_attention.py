"""Attention over prompts, the 8-bit paged cache and the tokens that read it against float64 forms.

Tolerances, derived from the roundings that the kernels make (half a step relative to a value:
bf16 2^-8, f16 2^-11, fp32 2^-24).  A row's output is a mean of values with weights p / sum p.
  prompts, bf16: each weight is rounded to bf16 once, so the mean moves by at most 2^-8 max|v|, the
      output is rounded once more: |err| <= 2^-8 max|v| + 2^-8 |o|; scores carry fp32 sums of 128
      exact products, below 2^-16 of a weight.
  tokens, bf16: weights in f16 (2^-11), the output rounded to bf16.
  fp32: operands as three bf16 (prompts) or two f16 parts (tokens): 2^-22 of a product; scores up to
      about 2^5 in base 2 with fp32 sums of 128 terms give a weight 2^5 * 2^-24 * a few; bound
      2^-17 max|v|.
"""
import pytest
import torch

import attention_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def close(got, want, v, dtype, weight):
    g = got.detach().double().cpu()
    top = float(v.detach().double().abs().max()) if v.numel() else 0.0
    if dtype == torch.float32:
        tol = torch.full_like(want, 2.0 ** -17 * top + 1e-30)
    else:
        tol = weight * top + 2.0 ** -8 * want.abs() + 2.0 ** -14 * top
    bad = ~((g - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((g - want).abs().max()), [tuple(i) for i in bad.nonzero()[:4].tolist()])


def make(T, hq, hkv, d, dtype, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hq + 2 * hkv, d, generator=g).to(dtype).to(DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(DEV)


PROMPTS = [
    ([1], 1, 1), ([2, 1, 0, 3], 2, 1), ([63, 64, 65], 4, 2), ([127, 0, 128, 129], 3, 3), ([33, 200, 1, 7], 12, 4),
    ([257, 511], 5, 1), ([300], 16, 2), ([130, 5], 40, 1), ([40], 128, 1), ([700, 90], 6, 2),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,hq,hkv", PROMPTS, ids=[f"{len(p[0])}x{max(p[0])}h{p[1]}of{p[2]}" for p in PROMPTS])
def test_prefill(lens, hq, hkv, d, dtype):
    q, k, v = make(sum(lens), hq, hkv, d, dtype, 1 + d + sum(lens), fused=True)
    out = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens))
    close(out, ref.prefill(q, k, v, lens), v, dtype, 2.0 ** -8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_prefill_equal_lengths_scale_and_out(dtype):
    q, k, v = make(4 * 77, 4, 2, 128, dtype, 3)
    out = torch.full_like(q, float("nan"))
    assert B.kda_attention_prefill(q, k, v, num_seqs=4, scale=0.3, out=out) is out
    close(out, ref.prefill(q, k, v, [77] * 4, scale=0.3), v, dtype, 2.0 ** -8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_hidden_infinities_and_nans_stay_hidden(d, dtype):
    """A later token's or another sequence's NaN or infinity reaches no row that does not see it."""
    lens = [150, 90, 300]
    q, k, v = make(sum(lens), 4, 2, d, dtype, 9)
    clean = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens))
    for at, bad in ((140, float("nan")), (150 + 60, float("inf")), (240 + 131, -float("inf"))):
        k2, v2 = k.clone(), v.clone()
        k2[at, 0, 3] = float("nan")
        v2[at, 1, 5] = bad
        out = B.kda_attention_prefill(q, k2, v2, cu_seqlens=offsets(lens))
        seq_end = next(e for e in (150, 240, 540) if at < e)
        # heads 0, 1 read key head 0, whose key is NaN; heads 2, 3 read the value
        want = clean.clone()
        want[at:seq_end, :2] = float("nan")
        want[at:seq_end, 2:, 5] = bad
        same = (out == want) | (out.isnan() & want.isnan())
        assert bool(same.all()), [tuple(i) for i in (~same).nonzero()[:4].tolist()]
    # +inf and -inf in one channel give NaN to the rows that see both
    v2 = v.clone()
    v2[20, 0, 1], v2[60, 0, 1] = float("inf"), -float("inf")
    out = B.kda_attention_prefill(q, k, v2, cu_seqlens=offsets(lens))
    col = out[:150, 0, 1].float().cpu()
    assert torch.isfinite(col[:20]).all() and (col[20:60] == float("inf")).all() and col[60:].isnan().all()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefill_fp32_many_tiles(d):
    """More tiles than the form for few of them takes: one CTA a tile."""
    lens = [5, 70, 0, 33, 131] * 36
    q, k, v = make(sum(lens), 4, 4, d, torch.float32, 11 + d, fused=True)
    out = B.kda_attention_prefill(q, k, v, cu_seqlens=offsets(lens))
    close(out, ref.prefill(q, k, v, lens), v, torch.float32, 0.0)
    # infinities of both signs in one channel, in different key tiles: NaN to the rows that see both, the first alone before
    start = sum(lens[:4])
    v2 = v.clone()
    v2[start + 9, 0, 1], v2[start + 77, 0, 1] = float("inf"), -float("inf")
    bad = B.kda_attention_prefill(q, k, v2, cu_seqlens=offsets(lens))
    want = out.clone()
    want[start + 9:start + 77, 0, 1], want[start + 77:start + 131, 0, 1] = float("inf"), float("nan")
    same = (bad == want) | (bad.isnan() & want.isnan())
    assert bool(same.all()), [tuple(i) for i in (~same).nonzero()[:4].tolist()]


def test_prefill_large_scores():
    """Scores of a few thousand: one key takes all the weight, nothing overflows."""
    q, k, v = make(400, 2, 2, 128, torch.bfloat16, 5)
    out = B.kda_attention_prefill(q * 30, k * 30, v)
    close(out, ref.prefill(q * 30, k * 30, v, [400]), v, torch.bfloat16, 2.0 ** -8 + 2.0 ** -8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_prefill_is_the_same_every_time_and_on_another_stream(dtype):
    q, k, v = make(1000, 8, 2, 128, dtype, 6)
    first = B.kda_attention_prefill(q, k, v, num_seqs=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(first)
    B.kda_attention_prefill(q, k, v, num_seqs=4, out=other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)


# ---------------------------------------------------------------- the cache

def tables(lens, page, extra=3, seed=0, capacity=0):
    """Shuffled pages; ``capacity`` keys at least a sequence in the table's columns."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + extra
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    cols = max(max(max(need), 1) + 1, -(-capacity // page))
    t = torch.full((len(lens), cols), -7, dtype=torch.int32)  # entries past the last page are not read
    at = 0
    for n, m in enumerate(need):
        t[n, :m] = order[at:at + m]
        at += m
    return t.to(DEV), pool


def filled(pool, hkv, page, d, code, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, pool, hkv, page, d, generator=g)
    c = [(x[i] * 90).clamp(-448, 448).to(code) if code == torch.float8_e4m3fn else (x[i] * 30).round().clamp(-127, 127).to(code)
         for i in range(2)]
    s = [torch.exp2(torch.randint(-8, -3, (pool, hkv), generator=g).float()) for _ in range(2)]
    return B.KvCache(*[t.to(DEV) for t in c], *[t.to(DEV) for t in s])


def same_codes(cache, want):
    for got, w in zip(cache, want):
        g = got.detach().cpu().to(torch.float64)
        assert bool(((g == w) | (g.isnan() & w.isnan())).all()), (int((g != w).sum()), g.numel())


CODES = [torch.float8_e4m3fn, torch.int8]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("page,d", [(16, 128), (32, 64), (64, 128), (128, 128), (128, 32)])
def test_append(page, d, code, dtype):
    """Prompts into empty and half-filled pages, then single tokens that grow a page's scale."""
    before, fresh = [0, 5, 64, 130, 33], [100, 1, 64, 200, 0]
    hkv = 3
    after = [a + b for a, b in zip(before, fresh)]
    table, pool = tables([n + 2 for n in after], page)
    cache = filled(pool, hkv, page, d, code)
    g = torch.Generator().manual_seed(4)
    kv = torch.randn(sum(fresh), 2 * hkv, d, generator=g) * torch.rand(sum(fresh), 1, 1, generator=g) * 8
    kv = kv.to(dtype).to(DEV)
    k, v = kv[:, :hkv], kv[:, hkv:]
    want = ref.append(k, v, cache, table, before, fresh)
    check = torch.zeros(64, dtype=torch.int32, device=DEV)
    lengths = torch.tensor(after, dtype=torch.int32, device=DEV)
    B.kda_cache_append(k, v, cache, table, lengths, cu_seqlens=offsets(fresh), check=check)
    same_codes(cache, want)
    for step in (1, 2):
        one = (torch.randn(len(after), 2 * hkv, d, generator=g) * 10.0 ** step).to(dtype).to(DEV)
        k, v = one[:, :hkv], one[:, hkv:]
        want = ref.append(k, v, cache, table, after, [1] * len(after))
        after = [n + 1 for n in after]
        lengths += 1
        B.kda_cache_append(k, v, cache, table, lengths, check=check)
        same_codes(cache, want)
    assert B.kda_workspace_status(check) == B.KDA_OK


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
def test_append_extremes(code):
    """Zeros, the smallest scale, infinities, NaN and values next to a border of the scale."""
    d, hkv = 64, 1
    top = ref.MAX[code]
    rows = [torch.zeros(d), torch.full((d,), 2.0 ** -80), torch.full((d,), top), torch.full((d,), top * 1.0001),
            torch.full((d,), 3e38), torch.full((d,), top * 0.50001), torch.linspace(-top, top, d)]
    odd = torch.randn(d, generator=torch.Generator().manual_seed(0))
    odd[3], odd[4], odd[5] = float("inf"), -float("inf"), float("nan")
    x = torch.stack(rows + [odd])[:, None].to(DEV)
    n = x.shape[0]
    table, pool = tables([1] * n, 16)
    cache = filled(pool, hkv, 16, d, code)
    want = ref.append(x, x, cache, table, [0] * n, [1] * n)
    B.kda_cache_append(x, x, cache, table, torch.ones(n, dtype=torch.int32, device=DEV))
    same_codes(cache, want)


def test_append_skips_what_is_out_of_range():
    """Bad lengths and pages write nothing and set the check word; the others are written."""
    hkv, d, page = 2, 64, 16
    table, pool = tables([32] * 4, page)
    table[1, 1], table[2, 1] = pool, -1
    cache = filled(pool, hkv, page, d, torch.int8)
    x = torch.randn(4, hkv, d, device=DEV)
    lengths = torch.tensor([20, 20, 20, 10_000], dtype=torch.int32, device=DEV)
    want = ref.append(x[:1], x[:1], cache, table, [19], [1])
    check = torch.zeros(64, dtype=torch.int32, device=DEV)
    B.kda_cache_append(x, x, cache, table, lengths, check=check)
    same_codes(cache, want)
    assert B.kda_workspace_status(check) == B.KDA_ERR_DEVICE_CHECK


TOKENS = [
    ([1], 1, 1, 1), ([0, 5, 31, 32, 33], 4, 1, 1), ([200, 0, 64, 1], 8, 2, 1), ([77, 300], 6, 2, 3), ([2, 600], 4, 4, 4),
    ([129, 4, 70], 20, 1, 1), ([100, 33], 16, 2, 7), ([1500], 3, 1, 1), ([40], 128, 1, 1), ([17] * 300, 2, 1, 1),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("page,d", [(16, 128), (32, 32), (64, 64), (128, 128)])
@pytest.mark.parametrize("lens,hq,hkv,window", TOKENS, ids=[f"{len(p[0])}x{max(p[0])}h{p[1]}of{p[2]}w{p[3]}" for p in TOKENS])
def test_decode(lens, hq, hkv, window, page, d, code, dtype):
    """Windows longer than the cached sequence leave rows that see nothing: zeros."""
    table, pool = tables(lens, page)
    cache = filled(pool, hkv, page, d, code, seed=page + d)
    q = make(len(lens) * window, hq, 1, d, dtype, 2, fused=True)[0]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)  # the workspace needs no preparation
    out = B.kda_attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), workspace=ws)
    v = ref.dequant(cache.v, cache.v_scale)
    close(out, ref.decode(q, cache, table, lens), v, dtype, 2.0 ** -11)
    assert B.kda_workspace_status(ws) == B.KDA_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,hq,hkv,window,d", [
    ([0, 1, 33, 100, 7] * 100, 8, 8, 1, 32), ([900] + [5] * 260, 16, 8, 1, 128), ([3, 0] * 250 + [700, 64], 8, 8, 3, 64),
    ([40, 31, 32, 65] * 70, 27, 9, 4, 128),
], ids=["mixed", "long_first", "long_last", "two_column_tiles"])
def test_decode_more_units_than_workers(lens, hq, hkv, window, d, dtype):
    """Short sequences, and a long one among them: the cut counts what a unit's start costs."""
    table, pool = tables(lens, 16)
    cache = filled(pool, hkv, 16, d, torch.int8, seed=8)
    q = make(len(lens) * window, hq, 1, d, dtype, 4, fused=True)[0]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)
    out = B.kda_attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), workspace=ws)
    close(out, ref.decode(q, cache, table, lens), ref.dequant(cache.v, cache.v_scale), dtype, 2.0 ** -11)
    assert B.kda_workspace_status(ws) == B.KDA_OK


MANY = [
    # lens, query heads, key heads, window: 17 rows and more a key head, up to several tiles of 32 rows
    ([1], 17, 1, 1), ([1], 25, 1, 1), ([0, 5, 127, 128, 129, 256], 8, 1, 4), ([3, 700], 16, 2, 7), ([1000, 64, 333], 24, 3, 5),
    ([90, 400], 8, 1, 40), ([1300], 128, 1, 2), ([17] * 300, 26, 1, 1), ([3000, 2900] * 20, 8, 2, 7), ([5], 4, 1, 30),
]


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("page,d", [(16, 128), (64, 64), (128, 128), (32, 128)])
@pytest.mark.parametrize("lens,hq,hkv,window", MANY, ids=[f"{len(p[0])}x{max(p[0])}h{p[1]}of{p[2]}w{p[3]}" for p in MANY])
def test_decode_many_rows(lens, hq, hkv, window, page, d, code):
    """Many rows a key head, which another kernel takes."""
    table, pool = tables(lens, page, capacity=600)
    cache = filled(pool, hkv, page, d, code, seed=page + d)
    q = make(len(lens) * window, hq, 1, d, torch.bfloat16, 2, fused=True)[0]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)
    out = B.kda_attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), workspace=ws)
    check_n = min(len(lens), 6)  # the float64 form of the first sequences; the rest against themselves
    few = ref.decode(q[:check_n * window], cache, table[:check_n], lens[:check_n])
    close(out[:check_n * window], few, ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)
    assert B.kda_workspace_status(ws) == B.KDA_OK
    assert torch.equal(out, B.kda_attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV)))
    n = len(lens) - 1  # the last sequence alone
    alone = B.kda_attention_decode(q[n * window:], cache, table[n:], torch.tensor(lens[n:], dtype=torch.int32, device=DEV))
    close(out[n * window:], alone.double().cpu(), ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("lens,hq,hkv,window", [
    ([0, 1, 700, 129, 40, 1500] * 30, 13, 1, 2), ([2000] + [9] * 160, 4, 1, 7), ([30, 0] * 90 + [1900], 26, 1, 1),
    ([400, 128, 0, 257] * 12, 10, 5, 14),
], ids=["mixed", "long_first", "long_last", "several_row_tiles"])
def test_decode_many_rows_mixed_lengths(lens, hq, hkv, window, code):
    """More units than CTAs, short and long: the cut counts what a unit's start costs."""
    table, pool = tables(lens, 32, capacity=2048)
    cache = filled(pool, hkv, 32, 128, code, seed=5)
    q = make(len(lens) * window, hq, 1, 128, torch.bfloat16, 3, fused=True)[0]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)
    out = B.kda_attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), workspace=ws)
    close(out, ref.decode(q, cache, table, lens), ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)
    assert B.kda_workspace_status(ws) == B.KDA_OK


@pytest.mark.parametrize("page", [16, 64])
def test_decode_many_rows_nan_past_the_end_and_in_hidden_keys(page):
    """As for few rows: stale NaN past the end reaches nothing, a drafted token's NaN the rows that see it alone."""
    lens, d, L, hq = [150, 95, 7, 300], 128, 7, 4
    table, pool = tables(lens, page, capacity=600)
    cache = filled(pool, 1, page, d, torch.float8_e4m3fn)
    q = make(4 * L, hq, 1, d, torch.bfloat16, 8)[0]
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean = B.kda_attention_decode(q, cache, table, lengths)
    raw = [c.view(torch.uint8).clone() for c in (cache.k, cache.v)]
    for n, length in enumerate(lens):
        last = int(table[n, (length - 1) // page])
        for c in raw:
            c[last, :, (length - 1) % page + 1:] = 0x7F
    dirty = B.KvCache(raw[0].view(torch.float8_e4m3fn), raw[1].view(torch.float8_e4m3fn), cache.k_scale, cache.v_scale)
    assert torch.equal(B.kda_attention_decode(q, dirty, table, lengths), clean)
    want = clean.clone()
    # the fourth of seven drafted tokens of sequence 0, and a token of sequence 3 that every row sees
    for n, key, ch in ((0, lens[0] - L + 3, 9), (3, lens[3] - L - 20, 77)):
        raw[1][int(table[n, key // page]), 0, key % page, ch] = 0xFF
        first = max(0, key - (lens[n] - L))
        want[n * L + first:(n + 1) * L, :, ch] = float("nan")
    out = B.kda_attention_decode(q, dirty, table, lengths)
    assert bool(((out == want) | (out.isnan() & want.isnan())).all())


def test_decode_many_rows_reports_bad_lengths_and_pages():
    page, d, L, hq = 16, 128, 7, 4
    table, pool = tables([200, 200, 200], page, capacity=600)
    cache = filled(pool, 1, page, d, torch.float8_e4m3fn)
    q = make(3 * L, hq, 1, d, torch.bfloat16, 8)[0]
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device=DEV)
    lengths = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    good = B.kda_attention_decode(q, cache, table, lengths(200, 200, 200), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_OK
    out = B.kda_attention_decode(q, cache, table, lengths(200, 10_000, 200), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_ERR_DEVICE_CHECK
    assert torch.equal(out[:L], good[:L]) and torch.equal(out[2 * L:], good[2 * L:]) and not out[L:2 * L].any()
    t2 = table.clone()
    t2[2, 3] = pool + 5  # keys 48 .. 63 of sequence 2 are not there
    out = B.kda_attention_decode(q, cache, t2, lengths(200, 200, 200), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_ERR_DEVICE_CHECK
    assert torch.equal(out[:2 * L], good[:2 * L])
    k, v = ref.cached(cache, table, 2, 200, 0)
    keep = torch.cat([torch.arange(48), torch.arange(64, 200)])
    x = q[2 * L:].detach().double().cpu().reshape(-1, d)
    seen = [200 - L + t + 1 - 16 for t in range(L) for _ in range(hq)]
    want = ref.rows(x, k[keep], v[keep], seen, d ** -0.5).view(L, hq, d)
    close(out[2 * L:], want, ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)


@pytest.mark.parametrize("hq,window", [(2, 1), (8, 5)], ids=["few", "many"])
@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
def test_decode_pages_without_scale(code, hq, window):
    """Pages whose values are zero, or whose keys are: their weight counts, their values add nothing."""
    lens, page, d = [640, 333], 16, 128
    table, pool = tables(lens, page)
    c = filled(pool, 1, page, d, code)
    vs, ks = c.v_scale.clone(), c.k_scale.clone()
    vs[::3], ks[1::4] = 0.0, 0.0
    cache = B.KvCache(c.k, c.v, ks, vs)
    q = make(2 * window, hq, 1, d, torch.bfloat16, 3)[0]
    out = B.kda_attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    close(out, ref.decode(q, cache, table, lens), ref.dequant(c.v, vs), torch.bfloat16, 2.0 ** -11)


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
def test_decode_scales_far_apart(code):
    """Pages whose scales differ by up to 2^50, zero scales among them."""
    lens, page, d = [640, 333], 16, 128
    table, pool = tables(lens, page)
    c = filled(pool, 2, page, d, code)
    g = torch.Generator().manual_seed(1)
    vs = torch.exp2(torch.randint(-50, 1, (pool, 2), generator=g).float())
    ks = torch.exp2(torch.randint(-12, -4, (pool, 2), generator=g).float())
    vs[::5], ks[::7] = 0.0, 0.0
    cache = B.KvCache(c.k, c.v, ks.to(DEV), vs.to(DEV))
    q = make(2, 4, 1, d, torch.bfloat16, 3)[0]
    out = B.kda_attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    close(out, ref.decode(q, cache, table, lens), ref.dequant(c.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)


@pytest.mark.parametrize("page", [16, 64])
def test_decode_nan_past_the_end_and_in_hidden_keys(page):
    """Stale codes past a sequence's end may be NaN; a drafted token's NaN reaches the rows that see it alone."""
    lens, d, L = [50, 95, 7], 128, 4
    table, pool = tables(lens, page)
    cache = filled(pool, 1, page, d, torch.float8_e4m3fn)
    q = make(3 * L, 2, 1, d, torch.bfloat16, 8)[0]
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean = B.kda_attention_decode(q, cache, table, lengths)
    raw = [c.view(torch.uint8).clone() for c in (cache.k, cache.v)]
    for n, length in enumerate(lens):
        last = int(table[n, (length - 1) // page])
        for c in raw:
            c[last, :, (length - 1) % page + 1:] = 0x7F
    dirty = B.KvCache(raw[0].view(torch.float8_e4m3fn), raw[1].view(torch.float8_e4m3fn), cache.k_scale, cache.v_scale)
    assert torch.equal(B.kda_attention_decode(q, dirty, table, lengths), clean)
    # the third of four drafted tokens of sequence 1 has a NaN value in channel 9
    key = lens[1] - L + 2
    raw[1][int(table[1, key // page]), 0, key % page, 9] = 0xFF
    out = B.kda_attention_decode(q, dirty, table, lengths)
    want = clean.clone()
    want[L + 2:2 * L, :, 9] = float("nan")
    assert bool(((out == want) | (out.isnan() & want.isnan())).all())


def test_decode_reports_bad_lengths_and_pages():
    """A bad length counts as an empty cache, a bad page as missing keys; both are reported."""
    page, d = 16, 64
    table, pool = tables([40, 40, 40], page)
    cache = filled(pool, 1, page, d, torch.float8_e4m3fn)
    q = make(3, 2, 1, d, torch.bfloat16, 8)[0]
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)
    good = B.kda_attention_decode(q, cache, table, torch.tensor([40, 40, 16], dtype=torch.int32, device=DEV), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_OK
    out = B.kda_attention_decode(q, cache, table, torch.tensor([40, -1, 16], dtype=torch.int32, device=DEV), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_ERR_DEVICE_CHECK
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and not out[1].any()
    t2 = table.clone()
    t2[2, 1], t2[2, 2] = pool, -1  # only the first page of sequence 2 is there
    out = B.kda_attention_decode(q, cache, t2, torch.tensor([40, 40, 40], dtype=torch.int32, device=DEV), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_ERR_DEVICE_CHECK
    assert torch.equal(out[:2], good[:2])
    close(out, ref.decode(q, cache, table, [40, 40, 16]), ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)
    assert B.kda_attention_decode(q, cache, table, torch.tensor([40, 40, 16], dtype=torch.int32, device=DEV), workspace=ws) is not None
    assert B.kda_workspace_status(ws) == B.KDA_OK


def test_prompts_then_tokens_in_a_graph():
    """A step (append, attend) captured once and replayed as the sequences grow."""
    page, d, hq, hkv, N = 64, 128, 8, 2, 3
    lens = [70, 1, 129]
    table, pool = tables([n + 8 for n in lens], page)
    cache = B.kda_cache_alloc(pool, page, hkv, d)
    q, k, v = make(sum(lens), hq, hkv, d, torch.bfloat16, 11, fused=True)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    B.kda_cache_append(k, v, cache, table, lengths, cu_seqlens=offsets(lens))
    q1, k1, v1 = make(N, hq, hkv, d, torch.bfloat16, 12)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q1)

    def step():
        lengths.add_(1)
        B.kda_cache_append(k1, v1, cache, table, lengths)
        B.kda_attention_decode(q1, cache, table, lengths, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x = make(N, hq, hkv, d, torch.bfloat16, 20 + i)
        for dst, src in zip((q1, k1, v1), x):
            dst.copy_(src)
        graph.replay()
        now = [n + 2 + i for n in lens]
        close(out, ref.decode(q1, cache, table, now), ref.dequant(cache.v, cache.v_scale), torch.bfloat16, 2.0 ** -11)
