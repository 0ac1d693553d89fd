"""Chunks of new tokens over the 8-bit paged cache against a float64 form.

Tolerances, derived from the roundings that the kernels make (half a step relative to a value: bf16 2^-8, f16 2^-11, fp32
2^-24).  A row's output is a mean of values with weights p / sum p.
  bf16: weights in f16 (2^-11 max|v|), the output rounded to bf16 (2^-8 |o|); scores carry fp32 sums of exact products.  Sums of
      the products' own may be cut off rather than rounded: a step of 16 keys moves the running sum by at most 2^-23 of
      it, so t keys by t 2^-27 max|v|.
  fp32: weights and q as two f16 parts (2^-22); scores of at most 2^5 in base 2 with 2 x 8 steps cut off at 2^-23 move a weight by
      2^5 x 2^-19 at most and, where signs differ, far less: bound 2^-15 max|v|.
"""
import pytest
import torch

import attention_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_attention import filled, offsets, tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = [torch.bfloat16, torch.float32]
CODES = [torch.float8_e4m3fn, torch.int8]


def want_of(q, cache, table, lens, new, scale=None):
    """The definition in float64, a sequence and head at a time."""
    d, group = q.shape[2], q.shape[1] // cache.k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    x = q.detach().double().cpu()
    out = torch.zeros(x.shape, dtype=torch.float64)
    s = 0
    for n, (length, m) in enumerate(zip(lens, new)):
        for h in range(cache.k.shape[1] if m and length > 0 else 0):
            k, v = ref.cached(cache, table, n, length, h)
            rows = x[s:s + m, h * group:(h + 1) * group].reshape(-1, d)
            seen = (torch.arange(m) + length - m + 1).repeat_interleave(group)
            z = (rows @ k.T) * scale
            z = z.masked_fill(torch.arange(length)[None] >= seen[:, None], -float("inf"))
            p = torch.exp(z - z.amax(1, keepdim=True).clamp(min=-1e300))
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
            out[s:s + m, h * group:(h + 1) * group] = (p @ v).view(m, group, d)
        s += m
    return out


def close(got, want, cache, longest, more=0.0):
    top = float((cache.v.float().nan_to_num().abs().amax((2, 3)) * cache.v_scale).max())
    if got.dtype == torch.float32:
        tol = torch.full_like(want, 2.0 ** -15 * top)
    else:
        tol = (2.0 ** -11 + 2.0 ** -14 + longest * 2.0 ** -27 + more) * top + 2.0 ** -8 * want.abs()
    bad = ~((got.detach().double().cpu() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((got.detach().double().cpu() - want).abs().max() / top), [tuple(i) for i in bad.nonzero()[:4].tolist()])


def case(lens, new, hq, hkv, d, page, code, io, seed=0, extra_rows=0):
    table, pool = tables(lens, page, seed=seed)
    cache = filled(pool, hkv, page, d, code, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = (1.5 * torch.randn(sum(new) + extra_rows, hq, d, generator=g)).to(io).to(DEV)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


CASES = [  # keys of each sequence, new tokens of each, query and key heads, page
    ([1], [1], 1, 1, 16), ([5, 1, 17], [5, 1, 3], 4, 2, 16), ([127, 128, 129], [127, 1, 2], 2, 1, 32),
    ([300, 0, 64, 9], [37, 0, 64, 0], 6, 2, 64), ([777], [130], 16, 4, 64), ([260, 513, 1000], [1, 257, 90], 3, 3, 128),
    ([2000, 40, 700, 700, 1], [33, 40, 1, 512, 1], 8, 2, 32), ([500], [60], 40, 1, 64), ([300, 310], [4, 9], 128, 1, 16),
    ([1500], [900], 10, 2, 128),
]


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens,new,hq,hkv,page", CASES, ids=[f"{max(c[0])}n{max(c[1])}h{c[2]}of{c[3]}p{c[4]}" for c in CASES])
def test_chunks(lens, new, hq, hkv, page, d, code, io):
    q, cache, table, lengths = case(lens, new, hq, hkv, d, page, code, io, seed=d + sum(new))
    out = B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=offsets(new))
    close(out, want_of(q, cache, table, lens, new), cache, max(lens))


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
def test_many_sequences_of_all_kinds(io):
    """A serving step: single tokens, chunks, slots without a sequence; more units than SMs."""
    lens = [(i * 37) % 900 + 1 for i in range(150)]
    new = [1 if i % 5 else min(lens[i], 40 + i) for i in range(150)]
    for i in (3, 77, 149):
        lens[i] = new[i] = 0
    q, cache, table, lengths = case(lens, new, 8, 4, 64, 16, torch.float8_e4m3fn, io, seed=5)
    close(B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=offsets(new)), want_of(q, cache, table, lens, new), cache, 900)


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
@pytest.mark.parametrize("n,new", [(1, 1), (1, 300), (2, 64)])
def test_long_contexts_are_cut_among_sms(n, new, io):
    lens = [20011 - 4321 * i for i in range(n)]
    q, cache, table, lengths = case(lens, [new] * n, 4, 2, 128, 64, torch.int8, io, seed=6)
    close(B.kda_attention_extend(q, cache, table, lengths), want_of(q, cache, table, lens, [new] * n), cache, 20011)


def test_strided_queries_scale_and_out():
    lens, new = [400, 90], [200, 3]
    q, cache, table, lengths = case(lens, new, 4, 2, 128, 64, torch.float8_e4m3fn, torch.bfloat16, seed=7, extra_rows=9)
    wide = torch.zeros(q.shape[0], 9, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, 3:7] = q
    out = torch.full_like(q, 7.0)
    assert B.kda_attention_extend(wide[:, 3:7], cache, table, lengths, cu_seqlens=offsets(new), scale=0.21, out=out) is out
    T = sum(new)
    close(out[:T], want_of(q[:T], cache, table, lens, new, scale=0.21), cache, 400)
    assert bool((out[T:] == 7.0).all())  # rows behind the last sequence's


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
def test_rows_that_see_nothing_are_zero(io):
    """More new tokens than keys: the first ones see none.  A length out of range counts as none and is reported."""
    lens, new = [3, 0, 200, 130], [10, 5, 300, 1]
    q, cache, table, lengths = case([max(n, 300) for n in lens], new, 4, 2, 64, 32, torch.float8_e4m3fn, io, seed=8)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, float("nan"))
    B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=offsets(new), out=out)
    want = want_of(q, cache, table, lens, new)
    assert not bool(want[:7].any()) and not bool(out[:7].any()) and not bool(out[10:15].any()) and not bool(out[15:115].any())
    close(out, want, cache, 300)
    for bad in (-1, 2 ** 30):
        lengths[2] = bad
        ws = torch.zeros(B.kda_attention_extend_workspace_bytes(B.KdaAttention(4, sum(new), 4, 2, 64, B._IO[io], 1.0, 0, 0, 0)), dtype=torch.uint8, device=DEV)
        B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=offsets(new), out=out, workspace=ws)
        assert B.kda_workspace_status(ws) == B.KDA_ERR_DEVICE_CHECK
        close(out, want_of(q, cache, table, [3, 0, 0, 130], new), cache, 300)
        lengths[2] = 200
        B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=offsets(new), out=out, workspace=ws)
        assert B.kda_workspace_status(ws) == B.KDA_OK


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_pages_that_are_not_there(page, io):
    """Keys of a page outside the pool are not there for any row, and the call reports it."""
    lens, new = [700, 650], [140, 2]
    q, cache, table, lengths = case(lens, new, 4, 2, 64, page, torch.float8_e4m3fn, io, seed=9)
    gone = table.clone()
    at = 256 // page  # a whole page of sequence 0, and the same of sequence 1
    gone[0, at], gone[1, at] = -3, 1 << 30
    ws = torch.zeros(B.kda_attention_extend_workspace_bytes(B.KdaAttention(2, sum(new), 4, 2, 64, B._IO[io], 1.0, 0, 0, 0)), dtype=torch.uint8, device=DEV)
    out = B.kda_attention_extend(q, cache, gone, lengths, cu_seqlens=offsets(new), workspace=ws)
    assert B.kda_workspace_status(ws) == B.KDA_ERR_DEVICE_CHECK
    x, want, s = q.double().cpu(), torch.zeros(q.shape, dtype=torch.float64), 0
    for n, (length, m) in enumerate(zip(lens, new)):
        keep = torch.cat([torch.arange(at * page), torch.arange((at + 1) * page, length)])
        for h in range(2):
            k, v = (y[keep] for y in ref.cached(cache, table, n, length, h))
            rows = x[s:s + m, 2 * h:2 * h + 2].reshape(-1, 64)
            seen = torch.tensor([int((keep <= length - m + t).sum()) for t in range(m) for _ in range(2)])
            want[s:s + m, 2 * h:2 * h + 2] = ref.rows(rows, k, v, seen, 64 ** -0.5).view(m, 2, 64)
        s += m
    close(out, want, cache, 700)


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 128])
def test_hidden_nans_stay_hidden(d, io):
    """A NaN in a key or value that a row does not see leaves it as it is; a row that sees it has it in that channel."""
    lens, new = [400, 390], [150, 200]
    q, cache, table, lengths = case(lens, new, 4, 2, d, 64, torch.float8_e4m3fn, io, seed=10)
    cu = offsets(new)
    clean = B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=cu)
    nan = torch.tensor(0x7f, dtype=torch.uint8, device=DEV)
    for n, key, ch in ((0, 300, 5), (0, 399, 0), (1, 191, d - 1), (1, 250, 17), (0, 20, 3)):
        c = B.KvCache(cache.k.clone(), cache.v.clone(), cache.k_scale, cache.v_scale)
        page = int(table[n, key // 64])
        c.k.view(torch.uint8)[page, 0, key % 64, ch] = nan      # heads 0, 1 read key head 0
        c.v.view(torch.uint8)[page, 1, key % 64, ch] = nan
        out = B.kda_attention_extend(q, c, table, lengths, cu_seqlens=cu)
        want = clean.clone()
        start, ctx = sum(new[:n]), lens[n] - new[n]
        first = start + max(0, key - ctx)
        want[first:start + new[n], :2] = float("nan")
        want[first:start + new[n], 2:, ch] = float("nan")
        same = (out == want) | (out.isnan() & want.isnan())
        assert bool(same.all()), (n, key, [tuple(i) for i in (~same).nonzero()[:4].tolist()])


def test_odd_rows_of_q_change_no_other():
    """A NaN, an infinity, a huge or a tiny row of q is that row's own affair."""
    lens, new = [500], [140]
    q, cache, table, lengths = case(lens, new, 4, 2, 128, 64, torch.float8_e4m3fn, torch.bfloat16, seed=11)
    clean = B.kda_attention_extend(q, cache, table, lengths)
    q2 = q.clone()
    q2[3, 1, 7], q2[60, 0, 0], q2[139, 3] = float("nan"), float("inf"), q[139, 3] * 2.0 ** 100
    q2[100, 2] = q[100, 2] * 2.0 ** -120
    out = B.kda_attention_extend(q2, cache, table, lengths)
    rest = torch.ones(140, 4, dtype=torch.bool, device=DEV)
    rest[3, 1] = rest[60, 0] = rest[139, 3] = rest[100, 2] = False
    assert torch.equal(out[rest], clean[rest]) and bool(out[3, 1].isnan().all()) and bool(out[60, 0].isnan().all())
    # scores near zero: a plain mean; enormous ones: the largest takes all
    k, v = ref.cached(cache, table, 0, 500, 1)
    mean = v[:500 - 140 + 101].mean(0)
    top = float(v.abs().max())
    assert float((out[100, 2].double().cpu() - mean).abs().max()) < (2.0 ** -11 + 2.0 ** -14 + 500 * 2.0 ** -27) * top + 2.0 ** -8 * float(mean.abs().max())
    z = k @ q2[139, 3].double().cpu()
    assert float((out[139, 3].double().cpu() - v[z.argmax()]).abs().max()) <= (2.0 ** -8 + 2.0 ** -11) * top


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
def test_large_scores_and_scales_far_apart(io):
    """Scores of thousands, and pages whose value scales lie 2^30 apart."""
    lens, new = [900, 257], [300, 257]
    q, cache, table, lengths = case(lens, new, 4, 2, 64, 32, torch.int8, io, seed=12)
    big = want_of(q * 40, cache, table, lens, new)
    # a score's rounding: 2^-24 of up to 2^13 in base 2 moves a weight by 2^-11; cut-off sums by up to 2^4 times that
    if io == torch.bfloat16:
        close(B.kda_attention_extend(q * 40, cache, table, lengths, cu_seqlens=offsets(new)), big, cache, 900, more=2.0 ** -7)
    c = B.KvCache(cache.k, cache.v, cache.k_scale, cache.v_scale.clone())
    c.v_scale[::3] *= 2.0 ** -30
    c.v_scale[1::3] *= 2.0 ** 8
    close(B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(new)), want_of(q, c, table, lens, new), c, 900)


@pytest.mark.parametrize("io", IO, ids=["bf16", "f32"])
def test_like_prompts_and_like_tokens(io):
    """A whole prompt as one chunk is the prompt over the cache's values; single tokens are kda_attention_decode's."""
    lens, hq, hkv, d, page = [300, 65, 1], 8, 2, 128, 64
    q, cache, table, lengths = case(lens, lens, hq, hkv, d, page, torch.float8_e4m3fn, io, seed=13)
    k, v = (torch.cat([torch.stack([ref.cached(cache, table, n, length, h)[i] for h in range(hkv)], 1) for n, length in enumerate(lens)]).to(io).to(DEV) for i in range(2))
    out = B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=offsets(lens))
    close(out, ref.prefill(q, k, v, lens), cache, 300)
    one = torch.stack([q[sum(lens[:n + 1]) - 1] for n in range(3)])
    got, tokens = B.kda_attention_extend(one, cache, table, lengths), B.kda_attention_decode(one, cache, table, lengths)
    close(got, tokens.double().cpu(), cache, 300, more=2.0 ** -8)


def test_the_same_every_time_on_another_stream_and_in_a_graph():
    lens, new = [5000, 300, 77], [200, 1, 77]
    q, cache, table, lengths = case(lens, new, 8, 2, 128, 64, torch.float8_e4m3fn, torch.bfloat16, seed=14)
    cu = offsets(new)
    first = B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=cu)
    assert all(torch.equal(first, B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=cu)) for _ in range(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=cu, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=cu, out=out)
    for x, y in ((lens, new), ([4000, 250, 60], [160, 40, 60]), (lens, new)):  # other lengths through the same graph
        lengths.copy_(torch.tensor(x, dtype=torch.int32))
        cu.copy_(offsets(y))
        graph.replay()
        if x is lens:
            assert torch.equal(out, first)


def test_nothing_new():
    q, cache, table, lengths = case([40, 50], [0, 0], 4, 2, 64, 32, torch.float8_e4m3fn, torch.bfloat16, seed=15)
    assert B.kda_attention_extend(q, cache, table, lengths).shape == (0, 4, 64)


def test_a_run_of_calls_as_they_are_used():
    """A prompt in pieces and then tokens, with positions: rotary append, then extend, against the definition over the
    cache as the calls left it."""
    r = B.make_rotary(128, base=5000.0)
    hq, hkv, d, page = 8, 2, 128, 32
    pieces = [[50, 7], [130, 0], [1, 200], [1, 1], [1, 1]]
    total = [sum(p[i] for p in pieces) for i in range(2)]
    g = torch.Generator().manual_seed(16)
    table, pool = tables(total, page, seed=16)
    cache = B.kda_cache_alloc(pool, page, hkv, d)
    lens = [0, 0]
    for new in pieces:
        lens = [a + b for a, b in zip(lens, new)]
        x = torch.randn(sum(new), hq + 2 * hkv, d, generator=g).bfloat16().to(DEV)
        lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = offsets(new)
        q = B.kda_rotary_append(r, x[:, hq:hq + hkv], x[:, hq + hkv:], cache, table, lengths, q=x[:, :hq], cu_seqlens=cu)
        out = B.kda_attention_extend(q, cache, table, lengths, cu_seqlens=cu)
        close(out, want_of(q, cache, table, lens, new), cache, max(lens))
