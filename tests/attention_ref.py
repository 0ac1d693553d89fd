"""Softmax attention in float64 for the GPU tests: prompts, the 8-bit cache's rounding and the tokens
that read it, each row over exactly the keys that it sees."""
import numpy as np
import torch

MAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def rows(q, k, v, seen, scale):
    """q [r, d] over k, v [t, d] (float64), row i over the first seen[i] keys; none: zeros."""
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
    for i in range(q.shape[0]):
        n = int(seen[i])
        if n <= 0:
            continue
        z = (k[:n] @ q[i]) * scale
        p = torch.exp(z - z.max())
        out[i] = (p / p.sum()) @ v[:n]
    return out


def prefill(q, k, v, lens, scale=None):
    q, k, v = (x.detach().double().cpu() for x in (q, k, v))
    T, hq, d = q.shape
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(T, hq, d, dtype=torch.float64)
    s = 0
    for n in lens:
        if n:
            mask = torch.ones(n, n).tril().bool()
            for h in range(hq):
                z = (q[s:s + n, h] @ k[s:s + n, h // group].T) * scale
                p = torch.softmax(z.masked_fill(~mask, -np.inf), -1)
                out[s:s + n, h] = p @ v[s:s + n, h // group]
        s += n
    return out


def dequant(codes, scale):
    return codes.detach().cpu().to(torch.float64) * scale.detach().cpu().double()[..., None, None]


def cached(cache, table, n, length, h):
    """Keys and values [length, d] (float64) of head h of sequence n."""
    page = cache.k.shape[2]
    ids = table[n, :-(-length // page)].long().cpu()
    return [dequant(c[ids.to(c.device), h:h + 1].squeeze(1)[:, None], s[ids.to(s.device), h:h + 1]).squeeze(1).reshape(-1, c.shape[3])[:length]
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


def decode(q, cache, table, lengths, scale=None):
    N = len(lengths)
    T, hq, d = q.shape
    L, group = T // N, hq // cache.k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    x = q.detach().double().cpu()
    out = torch.zeros(T, hq, d, dtype=torch.float64)
    for n, length in enumerate(lengths):
        for h in range(cache.k.shape[1]):
            if length <= 0:
                continue
            k, v = cached(cache, table, n, length, h)
            seen = [length - L + t + 1 for t in range(L) for _ in range(group)]
            part = x[n * L:(n + 1) * L, h * group:(h + 1) * group].reshape(-1, d)
            out[n * L:(n + 1) * L, h * group:(h + 1) * group] = rows(part, k, v, seen, scale).view(L, group, d)
    return out


def nearest(x, dtype):
    """float64 values to the nearest code, ties to even; infinities saturate, NaN stays (int8: 0)."""
    if dtype == torch.int8:
        return torch.nan_to_num(torch.round(x).clamp(-127, 127), nan=0.0)
    e = torch.frexp(x).exponent.double() - 1
    step = torch.exp2(e.clamp(min=-6.0) - 3)
    fin = torch.isfinite(x)
    y = torch.where(fin, torch.round(x / step) * step, x)
    return y.clamp(-448.0, 448.0)


def append(k, v, cache, table, lens_before, fresh):
    """The cache after the append, as (codes k, codes v, scale k, scale v) in float64, by the definition."""
    dtype, page = cache.k.dtype, cache.k.shape[2]
    res = []
    for x, c, sc in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        x, c, sc = x.detach().double().cpu(), c.detach().cpu().to(torch.float64), sc.detach().cpu().double()
        s = 0
        for n, (old, new) in enumerate(zip(lens_before, fresh)):
            for p in range(old // page, -(-(old + new) // page)):
                a, b = max(old, p * page), min(old + new, (p + 1) * page)
                at = int(table[n, p])
                for h in range(c.shape[1]):
                    y = x[s + a - old:s + b - old, h]
                    fin = y[torch.isfinite(y)].abs()
                    amax = float(fin.max()) if fin.numel() else 0.0
                    e = -60
                    while amax > MAX[dtype] * 2.0 ** e:
                        e += 1
                    unit = 2.0 ** e
                    if a > p * page:
                        was = float(sc[at, h])
                        if unit > was:
                            c[at, h] = nearest(c[at, h] * was / unit, dtype)
                        unit = max(unit, was)
                    sc[at, h] = unit
                    c[at, h, a - p * page:b - p * page] = nearest(y / unit, dtype)
            s += new
        res.append((c, sc))
    return res[0][0], res[1][0], res[0][1], res[1][1]
