"""Chunks over the 8-bit cache where they can go wrong: odd page scales, scales and scores far apart, the largest values,
long sums of one sign, a graph's other lengths.

Tolerances are those of test_gpu_extend.py, whose head derives them; what differs is derived beside the test."""
import math

import pytest
import torch

import attention_ref as ref
from linear_attention_recurrence_kda_gb300 import binding as B
from test_gpu_attention import filled, offsets, tables
from test_gpu_extend import CODES, DEV, IO, case, close, want_of

pytestmark = pytest.mark.gpu
IDS = dict(ids=["bf16", "f32"])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def with_scales(c, ks=None, vs=None):
    return B.KvCache(c.k, c.v, c.k_scale if ks is None else ks.to(DEV), c.v_scale if vs is None else vs.to(DEV))


LENS, NEW = [900, 257, 40], [300, 257, 1]


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("d,page", [(64, 32), (128, 64), (128, 16)])
def test_scales_that_are_no_power_of_two(d, page, code, io):
    """Over two and a half decades.  (A value's scale enters as 2^(log2 of it): 2^-22 of a weight and half a step of a logarithm below
    2^5, 2^-20; far below the tolerances' other parts.)"""
    q, c, table, lengths = case(LENS, NEW, 4, 2, d, page, code, io, seed=21)
    g = torch.Generator().manual_seed(22)
    spread = lambda: torch.exp(torch.empty(c.k_scale.shape).uniform_(-6.0, 0.0, generator=g)) / 30  # noqa: E731
    c = with_scales(c, spread() / 4, spread())
    close(B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(NEW)), want_of(q, c, table, LENS, NEW), c, 900)


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
def test_scales_of_zero_and_below(code, io):
    """A scale of zero makes keys that score zero, or values of zero whose weights count; a negative one turns signs."""
    q, c, table, lengths = case(LENS, NEW, 4, 2, 64, 16, code, io, seed=23)
    ks, vs = c.k_scale.clone(), c.v_scale.clone()
    ks[::5], ks[1::7], vs[::4], vs[1::3] = 0.0, -ks[1::7], 0.0, -vs[1::3]
    c = with_scales(c, ks, vs)
    out = B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(NEW))
    close(out, want_of(q, c, table, LENS, NEW), with_scales(c, ks, vs.abs()), 900)
    c = with_scales(c, ks, torch.zeros_like(vs))
    assert not bool(B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(NEW)).any())


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("of", ["k", "v"])
def test_scales_that_are_no_number(of, bad, io):
    """A page whose scale is infinite or NaN leaves the rows that do not see it as the definition has them, and gives no
    finite value to those that see all of it (with infinite scales a row's scores there are infinities, of either sign)."""
    lens, new = [300, 200], [120, 40]
    q, c, table, lengths = case(lens, new, 4, 2, 64, 16, torch.int8, io, seed=24)
    want = want_of(q, c, table, lens, new)
    for n, page in ((0, 15), (0, 18), (1, 12)):
        ks, vs = c.k_scale.clone(), c.v_scale.clone()
        (ks if of == "k" else vs)[table[n, page], 1] = bad  # heads 2 and 3 read key head 1
        out = B.kda_attention_extend(q, with_scales(c, ks, vs), table, lengths, cu_seqlens=offsets(new))
        first = sum(new[:n]) + 16 * page - (lens[n] - new[n])
        sees = torch.zeros(out.shape, dtype=torch.bool)
        sees[first:sum(new[:n + 1]), 2:] = True
        close(torch.where(sees.to(DEV), 0, out), torch.where(sees, 0.0, want), c, 300)
        whole = out[min(first + 15, sum(new[:n + 1]) - 1):sum(new[:n + 1]), 2:]
        assert whole.numel() > 0 and not bool(torch.isfinite(whole).any())


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_scale_that_is_no_number_alone(bad, io):
    """No other page gives the outputs a unit."""
    q, c, table, lengths = case([16], [3], 4, 2, 64, 16, torch.int8, io, seed=25)
    out = B.kda_attention_extend(q, with_scales(c, vs=torch.full_like(c.v_scale, bad)), table, lengths)
    assert not bool(torch.isfinite(out).any())


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("low,high", [(-50, 1), (-60, 70), (-126, 0), (-60, 118), (-140, -100)])
def test_value_scales_far_apart(low, high, io):
    """Pages side by side whose value scales differ by up to 2^178, zeros among them."""
    q, c, table, lengths = case(LENS, NEW, 4, 2, 64, 16, torch.int8, io, seed=26)
    g = torch.Generator().manual_seed(27)
    vs = torch.exp2(torch.randint(low, high + 1, c.v_scale.shape, generator=g).float())
    vs[::3] = 2.0 ** low
    vs[1::5], vs[2::7] = 2.0 ** high, 0.0
    c = with_scales(c, vs=vs)
    close(B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(NEW)), want_of(q, c, table, LENS, NEW), c, 900)


@pytest.mark.parametrize("io", IO, **IDS)
def test_weights_of_values_on_a_tiny_scale_count(io):
    """One key on a scale of 1 scores 12 more in base 2 than 4095 keys whose values are on a scale of 2^-120: half of the
    weight is theirs."""
    n, page, d = 4096, 128, 64
    k, v = torch.zeros(n // page, 1, page, d), torch.ones(n // page, 1, page, d)
    k[0, 0, 0, 0] = 24
    vs = torch.full((n // page, 1), 2.0 ** -120)
    vs[0] = 1.0
    v[0, 0, 1:] = 0
    c = B.KvCache(k.to(torch.int8).to(DEV), v.to(torch.int8).to(DEV), torch.full((n // page, 1), 0.5).to(DEV), vs.to(DEV))
    for order in (torch.arange(n // page), torch.arange(n // page).flip(0)):  # first, and last of all
        table = order.to(torch.int32)[None].to(DEV)
        q = torch.zeros(1, 2, d, dtype=io, device=DEV)
        q[:, :, 0] = 1
        out = B.kda_attention_extend(q, c, table, i32([n]), scale=math.log(2.0))
        want = want_of(q, c, table, [n], [1], scale=math.log(2.0))
        assert abs(float(want[0, 0, 0]) - 0.5) < 1e-3
        close(out, want, c, n)


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("up", [2.0 ** 13, 2.0 ** 24, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("io", IO, **IDS)
def test_huge_scores(io, up, code):
    """All rows' scores, and one row's among ordinary ones: the largest takes all (two scores a rounding apart would share)."""
    lens, new = [700, 40, 131], [60, 1, 131]
    q, c, table, lengths = case(lens, new, 4, 2, 128, 32, code, io, seed=28)
    cu = offsets(new)
    close(B.kda_attention_extend(q * up, c, table, lengths, cu_seqlens=cu), want_of(q * up, c, table, lens, new), c, 700)
    x = q.clone()
    x[7, 1], x[100, 3] = q[7, 1] * up, q[100, 3] * up
    out = B.kda_attention_extend(x, c, table, lengths, cu_seqlens=cu)
    close(out, want_of(x, c, table, lens, new), c, 700)


@pytest.mark.parametrize("up", [2.0 ** 8, 2.0 ** 20, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("io", IO, **IDS)
def test_huge_key_scales(io, up):
    lens, new = [700, 40, 131], [60, 1, 131]
    q, c, table, lengths = case(lens, new, 4, 2, 128, 32, torch.float8_e4m3fn, io, seed=29)
    ks = c.k_scale.clone()
    ks[::3] *= up
    c = with_scales(c, ks)
    # with 2^8: scores of 2^14 in base 2, in 2 x 8 steps cut off at 2^-23 of them: 2^-5 of a weight, for fp32
    want = want_of(q, c, table, lens, new)
    if io == torch.float32 and up == 2.0 ** 8:
        top = float((c.v.float().abs().amax((2, 3)) * c.v_scale).max())
        out = B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(new)).double().cpu()
        assert float((out - want).abs().max()) <= 2.0 ** -4 * top
    else:
        close(B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(new)), want, c, 700, more=2.0 ** -4 if up == 2.0 ** 8 else 0.0)


def test_large_scores_in_full_precision():
    """Scores of up to 2^13 in base 2: 2 x 4 steps of the products cut off at 2^-23 and one rounding move a score by 2^-7 + 2^-11
    and the mean by 2 ln 2 times that."""
    lens, new = [900, 257], [300, 257]
    q, c, table, lengths = case(lens, new, 4, 2, 64, 32, torch.int8, torch.float32, seed=12)
    out = B.kda_attention_extend(q * 40, c, table, lengths, cu_seqlens=offsets(new))
    top = float((c.v.float().abs().amax((2, 3)) * c.v_scale).max())
    assert float((out.double().cpu() - want_of(q * 40, c, table, lens, new)).abs().max()) <= 1.5 * (2.0 ** -7 + 2.0 ** -11) * top


@pytest.mark.parametrize("code", CODES, ids=["e4m3", "int8"])
@pytest.mark.parametrize("io,at,high,first", [(torch.float32, 0, 26, False), (torch.float32, 256, 20, True), (torch.bfloat16, 256, 20, True)],
                         ids=["f32", "f32_scale", "bf16_scale"])
def test_one_key_before_a_long_flat_tail(io, at, high, first, code):
    """Thousands of weights far below the largest add up: 4095 of 2^-26 of it, or of 2^-20 after a page on a larger scale."""
    n, many, hq = 4096, 40, 12
    page, d = 128, 128
    k, v = torch.zeros(n // page, 1, page, d), torch.full((n // page, 1, page, d), 64.0)
    vs = torch.full((n // page, 1), 2.0 ** -6)
    k[at // page, 0, at % page, 0] = 2 * high
    v[at // page, 0, at % page] = 0
    if first:
        v[0], vs[0] = 0, 1.0
    c = B.KvCache(k.to(code).to(DEV), v.to(code).to(DEV), torch.full((n // page, 1), 0.5).to(DEV), vs.to(DEV))
    table = torch.arange(n // page, dtype=torch.int32).repeat(many, 1).to(DEV)
    q = torch.zeros(many, hq, d, dtype=io, device=DEV)
    q[:, :, 0] = 1
    out = B.kda_attention_extend(q, c, table, i32([n] * many), scale=math.log(2.0))
    want = want_of(q[:1], c, table[:1], [n], [1], scale=math.log(2.0))
    assert float(want.max()) > (2.0 ** -15 if io == torch.float32 else 2.0 ** -11)  # not lost in the tolerance
    # (weights of 2^-26 of the largest and sums in fp32: 2^-17 where test_gpu_extend.py grants products of signs 2^-15)
    tol = 2.0 ** -17 if io == torch.float32 else 2.0 ** -11 + 2.0 ** -14 + n * 2.0 ** -27
    err = (out.double().cpu() - want).abs() - 2.0 ** -8 * (io == torch.bfloat16) * want.abs()
    assert float(err.max()) <= tol * float(v.max() * 2.0 ** -6)


@pytest.mark.parametrize("io", IO, **IDS)
def test_scores_of_minus_infinity_alone(io):
    """A row whose every score is -inf has no weight: zeros, and the other rows as they were."""
    lens, new = [150, 300], [7, 130]
    q, c, table, lengths = case(lens, new, 4, 1, 128, 16, torch.int8, io, seed=30)
    k = c.k.clone()
    k[..., 0] = -3
    c = B.KvCache(k, c.v, c.k_scale, c.v_scale)
    clean = B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(new))
    x = q.clone()
    x[9, 2, 0] = float("inf")
    out = B.kda_attention_extend(x, c, table, lengths, cu_seqlens=offsets(new))
    want = clean.clone()
    want[9, 2] = 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("keys,many", [(300, 200), (300, 1), (20011, 1)], ids=["whole", "few_pieces", "many_pieces"])
def test_values_near_the_largest(keys, many, io):
    """Values up to 2^127, in units that one CTA holds and in units that many share: their means are finite."""
    q, c, table, lengths = case([keys] * many, [2] * many, 4, 2, 64, 64, torch.int8, io, seed=31)
    c = B.KvCache(c.k, (c.v.float().abs() + 1).clamp(max=127).to(torch.int8), c.k_scale, torch.full_like(c.v_scale, 2.0 ** 120))
    out = B.kda_attention_extend(q, c, table, lengths).double().cpu() * 2.0 ** -120
    small = with_scales(c, vs=torch.ones_like(c.v_scale))
    want = want_of(q, small, table, [keys] * many, [2] * many)
    close(out.float() if io == torch.float32 else out.bfloat16(), want, small, keys)


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("d", [64, 128])
def test_long_sums_of_one_sign(d, io):
    """Units enough to fill the SMs, 400,000 keys each, which a CTA adds up by itself; every value of some channels is 1, of others
    positive.  The tolerance does not grow with the length."""
    keys, page, hkv, many = 400_000, 128, 8, 40
    pages = 64
    g = torch.Generator().manual_seed(32)
    k = torch.randn(pages, hkv, page, d, generator=g).mul(30).round().clamp(-127, 127)
    v = torch.randint(1, 128, (pages, hkv, page, d), generator=g).float()
    v[..., ::3] = 127
    c = B.KvCache(k.to(torch.int8).to(DEV), v.to(torch.int8).to(DEV), torch.full((pages, hkv), 2.0 ** -6).to(DEV), torch.full((pages, hkv), 2.0 ** -7).to(DEV))
    cols = keys // page
    table = (torch.arange(cols, dtype=torch.int32) % pages).repeat(many, 1).to(DEV)
    q = torch.randn(many, hkv, d, generator=g).to(io).to(DEV)
    q[::2] *= 0.01  # weights nearly alike
    out = B.kda_attention_extend(q, c, table, i32([cols * page] * many))
    # the pages repeat: their keys' weights are counted as often as they stand in the table
    often = torch.bincount(table[0].long().cpu(), minlength=pages).double().repeat_interleave(page)
    want = torch.zeros(out.shape, dtype=torch.float64)
    kd, vd = ref.dequant(c.k, c.k_scale), ref.dequant(c.v, c.v_scale)
    for h in range(hkv):
        kk, vv = kd[:, h].reshape(-1, d), vd[:, h].reshape(-1, d)
        z = q[:, h].double().cpu() @ kk.T * d ** -0.5
        p = torch.exp(z - z.amax(1, keepdim=True)) * often
        want[:, h] = (p / p.sum(1, keepdim=True)) @ vv
    worst = ((out.double().cpu() - want).abs() / want.abs()).max()
    print(f"largest relative distance {float(worst):.2e}, mean {float(((out.double().cpu() - want) / want).mean()):.2e}")
    # as for few keys: weights in f16 (2^-11, of either sign), sums cut off for 2^12 steps at most, by 2^-23 each, the output's half a
    # step; fp32: 2^-15 as for scores of signs
    assert float(worst) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11 if io == torch.bfloat16 else 2.0 ** -15)
    # and on the whole no more bias than those steps': f16's and bf16's roundings are of either sign, what is cut off is not
    bias = float(((out.double().cpu() - want) / want).mean())
    assert abs(bias) <= (2.0 ** -11 if io == torch.bfloat16 else 2.0 ** -17)


def test_other_lengths_through_the_same_graph():
    """Replays with other lengths and offsets give what direct calls give; rows behind the last sequence stay."""
    lens, new = [5000, 300, 77], [200, 1, 77]
    q, c, table, lengths = case(lens, new, 8, 2, 128, 64, torch.float8_e4m3fn, torch.bfloat16, seed=14)
    cu = offsets(new)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    B.kda_attention_extend(q, c, table, lengths, cu_seqlens=cu, out=out)
    with torch.cuda.graph(graph):
        B.kda_attention_extend(q, c, table, lengths, cu_seqlens=cu, out=out)
    for x, y in ((lens, new), ([4000, 250, 60], [160, 40, 60]), ([1, 0, 77], [1, 0, 3]), ([2048, 300, 5], [0, 200, 0]), (lens, new)):
        lengths.copy_(torch.tensor(x, dtype=torch.int32))
        cu.copy_(offsets(y))
        out.fill_(9.0)
        graph.replay()
        direct = torch.full_like(out, 9.0)
        B.kda_attention_extend(q, c, table, lengths, cu_seqlens=cu, out=direct)
        T = sum(y)
        assert torch.equal(out, direct) and bool((out[T:] == 9.0).all())
        close(out[:T], want_of(q[:T], c, table, x, y), c, max(x))


@pytest.mark.parametrize("io", IO, **IDS)
@pytest.mark.parametrize("lens,new", [([777], [37]), ([9000, 300, 4000, 1], [700, 1, 64, 1])])
def test_what_a_workspace_held_does_not_count(lens, new, io):
    """The same bits from a workspace of zeros and one of NaN."""
    q, c, table, lengths = case(lens, new, 16, 4, 128, 64, torch.float8_e4m3fn, io, seed=33)
    need = B.kda_attention_extend_workspace_bytes(B.KdaAttention(len(lens), sum(new), 16, 4, 128, B._IO[io], 1.0, 0, 0, 0))
    got = []
    for fill in (0, 255, 127, 0):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        got.append(B.kda_attention_extend(q, c, table, lengths, cu_seqlens=offsets(new), workspace=ws))
        assert B.kda_workspace_status(ws) == B.KDA_OK
    assert all(torch.equal(got[0], x) for x in got[1:])
