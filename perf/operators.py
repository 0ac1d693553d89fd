"""Attention next to KDA layers: prompts, an 8-bit paged cache, and tokens that read it.

Three operators of a serving path, each in a plain form of elementary torch operations and through
the framework's entry points:

* ``prefill``  causal attention over packed prompts with grouped heads (``kda_attention_prefill``);
* ``append``   keys and values of new tokens into a paged cache of 8-bit codes with one scale for
               each page and head (``kda_cache_append``);
* ``decode``   the newest tokens of every sequence attend to that cache (``kda_attention_decode``).
"""
import math

import torch

own = False

MAX_CODE = {"e4m3": 448.0, "int8": 127.0}
MIN_EXP = -60  # smallest exponent of a page's scale
IO = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _prefill(name, lens, hq, hkv, d=128, io="bf16", fused=False):
    """lens: "AxB" for A prompts of B tokens, or "A:lo-hi" for A prompts of lo to hi tokens (drawn)."""
    return {"name": name, "op": "prefill", "lens": lens, "hq": hq, "hkv": hkv, "d": d, "io": io, "fused": fused}


def _append(name, lens, new, hkv, d=128, page=64, code="e4m3", io="bf16"):
    """lens: tokens already cached; new: tokens appended to every sequence (0: the whole of ``lens``, from empty)."""
    return {"name": name, "op": "append", "lens": lens, "new": new, "hkv": hkv, "d": d, "page": page, "code": code,
            "io": io}


def _decode(name, lens, hq, hkv, window=1, d=128, page=64, code="e4m3", io="bf16"):
    return {"name": name, "op": "decode", "lens": lens, "hq": hq, "hkv": hkv, "window": window, "d": d, "page": page,
            "code": code, "io": io}


def listed():
    return [
        # a few chat turns arriving together: short prompts, where latency counts
        _prefill("prompts_short", "6:1-90", 16, 4),
        # the benchmark's prompt, 4096 tokens, 16 heads, read from one fused projection
        _prefill("prompt_4096", "1x4096", 16, 4, fused=True),
        # the benchmark's ragged batch, 8 prompts of 1024 to 16384 tokens, 32 heads
        _prefill("prompts_ragged", "8:1024-16384", 32, 8),
        # many middling prompts of a small model: 64 channels, one key head per query head
        _prefill("prompts_d64", "40:100-1500", 12, 12, d=64),
        # the fp32 form, used to check a model in full precision
        _prefill("prompts_fp32", "3:200-1300", 10, 2, io="fp32"),
        # prompts enter the cache
        _append("append_prompts", "8:1024-16384", 0, 8),
        # one token of each of 256 sequences enters the cache
        _append("append_step", "256:512-576", 1, 8),
        # one user, a short context: latency
        _decode("step_one_user", "1x777", 16, 4),
        # 256 sequences after a 512-token prompt and some 64 tokens, 32 heads
        _decode("step_256", "256:512-576", 32, 8),
        # long ragged contexts in int8
        _decode("step_ragged", "48:1024-32768", 32, 8, code="int8"),
        # one 1,048,576-token context
        _decode("step_1m", "1x1048576", 32, 8, page=128),
        # a drafted window of 7 tokens verified for each of 64 sequences
        _decode("verify_7", "64:300-6000", 32, 8, window=7, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "append", "decode", "decode"))
    d = rng.choice((128, 128, 64, 32))
    io = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    code = rng.choice(("e4m3", "int8"))
    page = rng.choice((16, 32, 64, 128))
    hkv = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 8))
    if op == "prefill":
        hi = _log(rng, 1, 16384 if io == "bf16" else 2048)
        n = _log(rng, 1, max(1, min(64, 131072 // hi)))
        # not more than the largest listed prompt batch
        while n > 1 and n * hi * hi * hkv * group * d > 3.0e12:
            n //= 2
        lo = max(1, hi // rng.choice((1, 2, 8)))
        case = _prefill("", "%d:%d-%d" % (n, lo, hi), hkv * group, hkv, d, io, rng.random() < 0.5)
    elif op == "append":
        n = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(16384, 65536 // n)))
        lo = max(1, hi // rng.choice((1, 2, 8)))
        case = _append("", "%d:%d-%d" % (n, lo, hi), rng.choice((0, 1, 1, 5)), hkv, d, page, code, io)
    else:
        n = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(1 << 20, (1 << 20) // n)))
        lo = max(1, hi // rng.choice((1, 2, 16)))
        window = rng.choice((1, 1, 1, 2, 7))
        case = _decode("", "%d:%d-%d" % (n, lo, hi), hkv * group, hkv, window, d, page, code, io)
    del case["name"]
    return case


def _lengths(text):
    """The lengths of a case, the same for every seed: an even spread over the range, shuffled by a fixed rule."""
    if "x" in text:
        n, length = (int(v) for v in text.split("x"))
        return [length] * n
    n, span = text.split(":")
    n, (lo, hi) = int(n), (int(v) for v in span.split("-"))
    return [lo + (hi - lo) * ((i * 7 + 3) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def work(case):
    lens, d = _lengths(case["lens"]), case["d"]
    io = 4 if case["io"] == "fp32" else 2
    if case["op"] == "prefill":
        t = sum(lens)
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 2 * t * (case["hq"] + case["hkv"]) * d * io, "flops": 4 * d * case["hq"] * pairs}
    pages = sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "append":
        t = len(lens) * case["new"] or sum(lens)
        touched = len(lens) if case["new"] else pages
        return {"bytes": 2 * t * case["hkv"] * d * (io + 1) + 8 * touched * case["hkv"], "flops": 4 * t * case["hkv"] * d}
    w = case["window"]
    pairs = sum(max(0, n - w + 1 + i) for n in lens for i in range(w))
    return {"bytes": 2 * sum(lens) * case["hkv"] * d + 8 * pages * case["hkv"] + 4 * pages
            + 2 * len(lens) * w * case["hq"] * d * io, "flops": 4 * d * case["hq"] * pairs}


# ---------------------------------------------------------------- inputs

def _cache(case, pages, gen, dev):
    """A filled cache: codes as a trained model's keys and values leave them, scales that are powers of two."""
    shape = (pages, case["hkv"], case["page"], case["d"])
    out = {}
    for name in ("k", "v"):
        if case["code"] == "e4m3":
            codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        else:
            codes = torch.empty(shape, dtype=torch.int8, device=dev)
        step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
        for a in range(0, pages, step):
            x = torch.randn((min(step, pages - a),) + shape[1:], generator=gen, device=dev)
            x.mul_(MAX_CODE[case["code"]] / 5).clamp_(-MAX_CODE[case["code"]], MAX_CODE[case["code"]])
            codes[a:a + step] = x.to(codes.dtype) if case["code"] == "e4m3" else x.round_().to(codes.dtype)
        unit = 2 if case["code"] == "int8" else 4  # a page's values have a spread of about a half to two
        e = torch.randint(-unit - 4, -unit - 1, (pages, case["hkv"]), generator=gen, device=dev)
        out[name], out[name + "_scale"] = codes, torch.exp2(e.float())
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    io, d, lens = IO[case["io"]], case["d"], _lengths(case["lens"])
    s = {"case": case, "lens": lens}
    if case["op"] == "prefill":
        t, hq, hkv = sum(lens), case["hq"], case["hkv"]
        qkv = torch.randn(t, hq + 2 * hkv, d, generator=gen, device=dev)
        qkv[:, :hq] *= 2.0  # scores spread over a few units, so that some keys stand out
        qkv = qkv.to(io)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        s.update(q=q, k=k, v=v, cu=cu.to(dev), max_len=max(lens))
        return s
    # the page table: every sequence's pages in an order drawn from the pool
    grown = [n + case["new"] for n in lens] if case["op"] == "append" else lens
    need = [-(-n // case["page"]) for n in grown]
    cols, pool = max(need), sum(need)
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), cols, dtype=torch.int32, device=dev)
    at = torch.tensor([0] + need).cumsum(0)
    rows = torch.arange(cols, device=dev)[None, :]
    inside = rows < torch.tensor(need, device=dev)[:, None]
    table[inside] = order[(at[:-1].to(dev)[:, None] + rows)[inside]]
    s.update(_cache(case, pool, gen, dev), table=table, lengths=torch.tensor(grown, dtype=torch.int32, device=dev),
             max_len=max(grown))
    if case["op"] == "append":
        fresh = [case["new"] or n for n in lens]
        t = sum(fresh)
        cu = torch.tensor([0] + fresh, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
        s.update(cu=None if case["new"] else cu)
        s["new_k"] = torch.randn(t, case["hkv"], d, generator=gen, device=dev).to(io)
        s["new_v"] = torch.randn(t, case["hkv"], d, generator=gen, device=dev).to(io)
    else:
        s["q"] = (2.0 * torch.randn(len(lens) * case["window"], case["hq"], d, generator=gen, device=dev)).to(io)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_prefill(s):
    """Prompts padded to the longest, a block of queries at a time so that the scores fit."""
    q, k, v, cu, longest = s["q"], s["k"], s["v"], s["cu"].long(), s["max_len"]
    n, (t, hq, d), hkv = cu.numel() - 1, q.shape, k.shape[1]
    at = torch.arange(longest, device=q.device)
    here = at[None, :] < (cu[1:] - cu[:-1])[:, None]
    idx = torch.clamp(cu[:-1, None] + at[None, :], max=t - 1)
    qf = q.float()[idx].view(n, longest, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    kf = k.float()[idx].permute(0, 2, 3, 1)[:, :, None]
    vf = v.float()[idx].permute(0, 2, 1, 3)[:, :, None]
    of = torch.empty(n, hkv, hq // hkv, longest, d, device=q.device)
    rows = max(1, min(longest, (1 << 30) // (n * hq * longest)))
    for a in range(0, longest, rows):
        b = min(longest, a + rows)
        p = torch.matmul(qf[..., a:b, :], kf[..., :b])
        p.mul_(d ** -0.5).masked_fill_(at[None, :b] > at[a:b, None], -math.inf)
        p = p.sub_(p.amax(-1, keepdim=True)).exp_()
        torch.matmul(p, vf[..., :b, :], out=of[..., a:b, :])
        of[..., a:b, :] /= p.sum(-1, keepdim=True)
    out = torch.empty(t, hq, d, dtype=q.dtype, device=q.device)
    out[idx[here]] = of.permute(0, 3, 1, 2, 4)[here].reshape(-1, hq, d).to(q.dtype)
    return out


def _codes(x, code):
    top = MAX_CODE[code]
    x = x.clamp(-top, top)
    return x.to(torch.float8_e4m3fn) if code == "e4m3" else torch.nan_to_num(x.round()).to(torch.int8)


def _plain_append(s):
    code, page = s["case"]["code"], s["case"]["page"]
    lengths, table = s["lengths"].long(), s["table"].long()
    n, dev = lengths.numel(), lengths.device
    t = s["new_k"].shape[0]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device=dev) * (t // n)
    seq = torch.searchsorted(cu[1:], torch.arange(t, device=dev), right=True)
    first = lengths - (cu[1:] - cu[:-1])  # a sequence's tokens before this call
    pos = first[seq] + torch.arange(t, device=dev) - cu[seq]
    pages, slot = table[seq, pos // page], pos % page
    begun = table[torch.arange(n, device=dev), first // page]  # the page that the first new token enters
    held = first % page != 0                                   # and whether it holds earlier tokens
    for x, codes, scale in ((s["new_k"], s["k"], s["k_scale"]), (s["new_v"], s["v"], s["v_scale"])):
        xf = x.float()
        amax = torch.where(torch.isfinite(xf), xf, 0.0).abs().amax(-1)
        m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1)
        mt, et = math.frexp(MAX_CODE[code])
        e = torch.where(amax > 0, e - et + (m > mt), MIN_EXP).clamp(min=MIN_EXP)
        old = scale[begun]
        new = torch.zeros_like(scale)
        new.scatter_reduce_(0, pages[:, None].expand(-1, scale.shape[1]), torch.exp2(e.float()), "amax")
        kept = torch.where(held[:, None], old, 0.0)
        grown = torch.maximum(new[begun], kept)
        # every sequence owns its pages, so each row of `begun` is written once
        new[begun] = grown
        ratio = torch.where(held[:, None], old / grown, 1.0)[:, :, None, None]
        codes[begun] = _codes(codes[begun].float() * ratio, code)
        scale[pages] = new[pages]
        q = xf / scale[pages][:, :, None]
        h = torch.arange(scale.shape[1], device=dev)[None, :]
        codes[pages[:, None], h, slot[:, None]] = _codes(q, code)
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _plain_decode(s):
    case, table = s["case"], s["table"].long()
    n, cols = table.shape
    w, hq, hkv, d = case["window"], case["hq"], case["hkv"], case["d"]

    def rows(codes, scale):  # [n, hkv, tokens, d]
        x = codes[table].float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, cols * case["page"], d)

    q = s["q"].float().view(n, w, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
    p = torch.matmul(q, rows(s["k"], s["k_scale"]).transpose(2, 3)).mul_(d ** -0.5)
    seen = s["lengths"].long()[:, None] - w + 1 + torch.arange(w, device=q.device)[None, :]
    hidden = torch.arange(p.shape[3], device=q.device)[None, None, :] >= seen[:, :, None]
    p.masked_fill_(hidden.repeat_interleave(hq // hkv, 1)[:, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = torch.matmul(p, rows(s["v"], s["v_scale"])) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(n, hkv, w, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n * w, hq, d).to(s["q"].dtype)


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"prefill": _plain_prefill, "append": _plain_append, "decode": _plain_decode}[op](s)
    from linear_attention_recurrence_kda_gb300 import binding as kda
    if op == "prefill":
        return kda.kda_attention_prefill(s["q"], s["k"], s["v"], cu_seqlens=s["cu"])
    cache = kda.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if op == "append":
        kda.kda_cache_append(s["new_k"], s["new_v"], cache, s["table"], s["lengths"], cu_seqlens=s["cu"])
        return s["k"], s["v"], s["k_scale"], s["v_scale"]
    return kda.kda_attention_decode(s["q"], cache, s["table"], s["lengths"])


# ---------------------------------------------------------------- 64 bits

def _softmax_read(q, k, v, seen):
    """Rows of q [r, d] over k, v [t, d], row i reading the first seen[i] of them, in 64 bits."""
    z = (q @ k.T) / math.sqrt(q.shape[1])
    z = torch.where(torch.arange(k.shape[0], device=q.device) < seen[:, None], z, -math.inf)
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, (e @ v) / total, 0.0)


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    dev, d = s["q"].device, case["d"]
    group = case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    w = case.get("window", 0)
    start = 0
    for n, length in enumerate(s["lens"]):
        if case["op"] == "decode":
            pages = s["table"][n, :-(-length // case["page"])].long()
        for h in range(case["hkv"]):
            heads = slice(h * group, (h + 1) * group)
            if case["op"] == "prefill":
                k, v = (s[x][start:start + length, h].double() for x in ("k", "v"))
                step = max(1, (1 << 27) // (length * group))
                for a in range(0, length, step):
                    b = min(length, a + step)
                    q = s["q"][start + a:start + b, heads].double().reshape(-1, d)
                    seen = torch.arange(a + 1, b + 1, device=dev).repeat_interleave(group)
                    out[start + a:start + b, heads] = _softmax_read(q, k[:b], v[:b], seen).view(-1, group, d)
            else:
                k, v = ((s[x][pages, h].double() * s[x + "_scale"][pages, h].double()[:, None, None])
                        .reshape(-1, d)[:length] for x in ("k", "v"))
                q = s["q"][n * w:(n + 1) * w, heads].double().reshape(-1, d)
                seen = (length - w + 1 + torch.arange(w, device=dev)).repeat_interleave(group)
                out[n * w:(n + 1) * w, heads] = _softmax_read(q, k, v, seen).view(-1, group, d)
        start += length
    return out


def _exact_append(s):
    """The definition taken page by page: each page's largest finite value sets the scale, then every value is rounded."""
    case, (top, page) = s["case"], (MAX_CODE[s["case"]["code"]], s["case"]["page"])
    lens, new = s["lens"], s["case"]["new"]
    if sum(lens if not new else [new] * len(lens)) // page + 2 * len(lens) > 4000:
        return None
    answers = []
    for x, name in ((s["new_k"], "k"), (s["new_v"], "v")):
        codes, scale = s[name].double(), s[name + "_scale"].double()
        start = 0
        for n, length in enumerate(lens):
            old, count = (length, new) if new else (0, length)
            first = old
            while first < old + count:
                last = min(old + count, (first // page + 1) * page)
                at, slot = int(s["table"][n, first // page]), first % page
                rows = x[start + first - old:start + last - old].double().transpose(0, 1)
                amax = rows.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / top))
                e = torch.where(top * torch.exp2(e - 1) >= amax, e - 1, torch.where(top * torch.exp2(e) < amax, e + 1, e))
                unit = torch.exp2(torch.where(amax > 0, e, float(MIN_EXP)).clamp(min=MIN_EXP))
                if slot:
                    unit = torch.maximum(unit, scale[at])
                    codes[at] = _nearest(codes[at] * (scale[at] / unit)[:, None, None], case["code"])
                scale[at] = unit
                codes[at, :, slot:slot + last - first] = _nearest(rows / unit[:, None, None], case["code"])
                first = last
            start += count
        answers.append((codes, scale))
    (k, ks), (v, vs) = answers
    if case["code"] == "int8":
        k, v = k.to(torch.int8), v.to(torch.int8)
    return k, v, ks, vs


def _nearest(x, code):
    """x in 64 bits to the nearest value that the code can hold, ties to even."""
    if code == "int8":
        return torch.round(x)
    step = torch.exp2(torch.clamp(torch.frexp(x).exponent.double() - 1, min=-6.0) - 3)  # three bits after the first
    return torch.clamp(torch.round(x / step) * step, -448.0, 448.0)
