"""Rotary positions and chunks of new tokens over the 8-bit paged cache.

Three operators of a serving path (the first also of training), each in a plain form of elementary
torch operations and through the framework's entry points:

* ``rotary``  queries and keys turned by their positions, one or several axes; its gradient is the
              same with the angles negated (``kda_rotary``);
* ``append``  keys turned by their positions and rounded into a paged cache of 8-bit codes with one
              scale for each page and head, values beside them, queries turned in the same call
              (``kda_rotary_append``);
* ``extend``  the new tokens of every sequence, a chunk of any length each, attend to that cache,
              which holds their keys and values already (``kda_attention_extend``).
"""
import math

import torch

own = False

MAX_CODE = {"e4m3": 448.0, "int8": 127.0}
MIN_EXP = -60  # smallest exponent of a page's scale
IO = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _rotary(name, lens, new, hq, hkv, d=128, rot=0, axes=0, adjacent=False, inverse=False, io="bf16", fused=False):
    """lens: tokens of every sequence with the new ones, "AxB" or "A:lo-hi" for A sequences; new: those that the call
    brings (see _news); rot: channels that turn, 0 for all; axes: 0, positions from the lengths, or 3."""
    return {"name": name, "op": "rotary", "lens": lens, "new": new, "hq": hq, "hkv": hkv, "d": d, "rot": rot or d,
            "axes": axes, "adjacent": adjacent, "inverse": inverse, "io": io, "fused": fused}


def _append(name, lens, new, hq, hkv, d=128, rot=0, axes=0, adjacent=False, page=64, io="bf16"):
    """hq: query heads that turn in the same call, 0 for none.  (Codes are e4m3, which come back as the values they
    stand for; an int8 code next to a tie may be either neighbour, and whole numbers have no tolerance.)"""
    return {"name": name, "op": "append", "lens": lens, "new": new, "hq": hq, "hkv": hkv, "d": d, "rot": rot or d,
            "axes": axes, "adjacent": adjacent, "page": page, "code": "e4m3", "io": io}


def _extend(name, lens, new, hq, hkv, d=128, page=64, code="e4m3", io="bf16"):
    return {"name": name, "op": "extend", "lens": lens, "new": new, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "code": code, "io": io}


def listed():
    return [
        # the benchmark's ragged batch, 8 prompts of 1024 to 16384 tokens, 32 heads, read from one fused projection
        _rotary("rotate_prompts", "8:1024-16384", "all", 32, 8, fused=True),
        # the gradient through positions of three axes: a few images with their text
        _rotary("rotate_axes_gradient", "3:900-5000", "all", 16, 4, axes=3, inverse=True),
        # a few tokens far into a long context, in full precision, a quarter of the channels in adjacent pairs: latency
        _rotary("rotate_far_fp32", "2:1000000-1048576", "77", 10, 2, d=64, rot=16, adjacent=True, io="fp32"),
        # one token of each of 256 sequences, some 64 tokens after a 512-token prompt
        _append("append_step", "256:513-576", "1", 32, 8),
        # prompts enter the cache, their queries turned on the way
        _append("append_prompts", "8:1024-16384", "all", 32, 8),
        # image tokens of a small model behind their text: three axes, small pages, odd lengths, full precision
        _append("append_axes_fp32", "5:300-2900", "3-701", 0, 3, d=64, axes=3, page=16, io="fp32"),
        # the next sentence of a chat, one user, a short context: latency
        _extend("chat_turn", "1x777", "37", 16, 4),
        # a chunk of 2048 tokens of a prompt of 32768, 32 heads
        _extend("chunk_2048", "1x32768", "2048", 32, 8),
        # a question of 256 tokens at the end of a 1,048,576-token context
        _extend("question_1m", "1x1048576", "256", 32, 8, page=128),
        # a serving step: most of 96 sequences bring one token, every eighth a chunk of its prompt
        _extend("mixed_step", "96:300-6000", "mix:8:64-512", 32, 8, page=32),
        # int8, 64 channels, a key head for every query head, small pages, chunks of odd lengths
        _extend("chunks_d64_int8", "7:1500-9000", "5-900", 12, 12, d=64, page=16, code="int8"),
        # full precision, used to check a model
        _extend("chunks_fp32", "3:700-2600", "40-333", 10, 2, io="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "append", "extend", "extend", "extend"))
    d = rng.choice((128, 128, 64, 32))
    io = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    page = rng.choice((16, 32, 64, 128))
    hkv = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 3, 4, 5, 8))
    rot = rng.choice([r for r in (16, 32, 64, 128) if r <= d])
    axes = rng.choice((0, 0, 3))
    n = _log(rng, 1, 256)
    if op == "extend":
        hi = _log(rng, 1, max(1, min(1 << 19, (1 << 20) // n)))
        most = max(1, min(4096, hi, (1 << 16) // n))
        # not more than the largest listed chunk
        while most > 1 and n * most * hi * hkv * group * d > 8.0e11 * (1 if io == "bf16" else 0.25):
            most = most // 2
        top = _log(rng, 1, most)
        new = rng.choice(("%d" % top, "%d-%d" % (max(1, top // 8), top), "0-%d" % top, "mix:%d:%d-%d" % (rng.choice((3, 8)), max(1, top // 4), top)))
        lo = max(1, hi // rng.choice((1, 2, 16)))
        case = _extend("", "%d:%d-%d" % (n, lo, hi), new, hkv * group, hkv, d, page, rng.choice(("e4m3", "int8")), io)
    else:
        hi = _log(rng, 1, max(1, min(16384, 65536 // n)))
        lo = max(1, hi // rng.choice((1, 2, 8)))
        new = rng.choice(("all", "all", "1", "%d-%d" % (max(1, hi // 5), max(1, hi // 2))))
        lens = "%d:%d-%d" % (n, lo, hi)
        if op == "rotary":
            case = _rotary("", lens, new, hkv * group, hkv, d, rot, axes, rng.random() < 0.4, rng.random() < 0.4, io, rng.random() < 0.5)
        else:
            case = _append("", lens, new, rng.choice((0, hkv * group)), hkv, d, rot, axes, rng.random() < 0.4, page, io)
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


def _news(text, lens):
    """New tokens of each sequence: "all" of them, "A", "lo-hi", or "mix:K:lo-hi", one token but for every K-th."""
    if text == "all":
        return list(lens)
    every = 1
    if text.startswith("mix:"):
        _, every, text = text.split(":")
        every = int(every)
    lo, hi = (int(v) for v in text.split("-")) if "-" in text else (int(text), int(text))
    n = len(lens)
    new = [1 if i % every else lo + (hi - lo) * ((i * 5 + 4) % n) // max(1, n - 1) if n > 1 else hi for i in range(n)]
    return [min(a, b) for a, b in zip(new, lens)]


def work(case):
    lens = _lengths(case["lens"])
    new = _news(case["new"], lens)
    t, d, hq, hkv = sum(new), case["d"], case["hq"], case["hkv"]
    io = 4 if case["io"] == "fp32" else 2
    if case["op"] == "rotary":
        return {"bytes": 2 * t * (hq + hkv) * d * io + 4 * t * case["axes"], "flops": 3 * t * (hq + hkv) * case["rot"]}
    if case["op"] == "append":
        touched = sum(-(-n // case["page"]) - (n - m) // case["page"] for n, m in zip(lens, new))
        return {"bytes": 2 * t * hkv * d * (io + 1) + 2 * t * hq * d * io + 8 * touched * hkv + 4 * t * case["axes"],
                "flops": 4 * t * hkv * d + 3 * t * (hq + hkv) * case["rot"]}
    read = [n for n, m in zip(lens, new) if m]
    pages = sum(-(-n // case["page"]) for n in read)
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
    return {"bytes": 2 * sum(read) * hkv * d + 8 * pages * hkv + 4 * pages + 2 * t * hq * d * io, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------- inputs

def _cache(case, pages, gen, dev):
    """A filled cache: codes as a trained model's keys and values leave them, scales that are powers of two."""
    shape = (pages, case["hkv"], case["page"], case["d"])
    out = {}
    for name in ("k", "v"):
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn if case["code"] == "e4m3" else torch.int8, device=dev)
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
    io, d, lens, hq, hkv = IO[case["io"]], case["d"], _lengths(case["lens"]), case["hq"], case["hkv"]
    new = _news(case["new"], lens)
    t = sum(new)
    cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
    s = {"case": case, "lens": lens, "new": new, "cu": cu, "lengths": torch.tensor(lens, dtype=torch.int32, device=dev)}
    if case["op"] != "extend":
        if case["axes"]:
            # tokens of images, rows and columns of 32, behind a start that grows with the sequence
            at = torch.arange(t, device=dev) + torch.randint(0, 2000, (1,), generator=gen, device=dev)
            s["positions"] = torch.stack([at // 1024, at // 32 % 32 + at // 1024, at % 32 + at // 1024]).to(torch.int32)
        else:
            s["positions"] = None
        qkv = 1.45 * torch.randn(t, hq + 2 * hkv, d, generator=gen, device=dev)
        qkv = qkv.to(io)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if not case.get("fused", False):
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        s.update(q=q if hq else None, new_k=k, new_v=v)
    if case["op"] != "rotary":
        # the page table: every sequence's pages in an order drawn from the pool
        need = [-(-n // case["page"]) for n in lens]
        cols, pool = max(need), sum(need)
        order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
        table = torch.zeros(len(lens), cols, dtype=torch.int32, device=dev)
        at = torch.tensor([0] + need).cumsum(0)
        rows = torch.arange(cols, device=dev)[None, :]
        inside = rows < torch.tensor(need, device=dev)[:, None]
        table[inside] = order[(at[:-1].to(dev)[:, None] + rows)[inside]]
        s.update(_cache(case, pool, gen, dev), table=table)
    if case["op"] == "extend":
        s["q"] = (2.0 * torch.randn(t, hq, d, generator=gen, device=dev)).to(io)
    return s


# ---------------------------------------------------------------- plain forms

def _sections(case):
    """Pairs of channels of each axis: a quarter for time, three eighths for rows and columns each."""
    p = case["rot"] // 2
    return (p - 2 * (3 * p // 8), 3 * p // 8, 3 * p // 8)


def _angles(s):
    """The angle of every token and pair of channels, in 64 bits."""
    case, cu, dev = s["case"], s["cu"].long(), s["cu"].device
    pairs = case["rot"] // 2
    freq = 10000.0 ** (-2.0 * torch.arange(pairs, dtype=torch.float64, device=dev) / case["rot"])
    if s["positions"] is None:
        t = int(sum(s["new"]))
        seq = torch.searchsorted(cu[1:], torch.arange(t, device=dev), right=True)
        pos = (s["lengths"].long() - cu[1:])[seq] + torch.arange(t, device=dev)
        angle = pos.double()[:, None] * freq
    else:
        axis = torch.repeat_interleave(torch.arange(3, device=dev), torch.tensor(_sections(case), device=dev), output_size=pairs)
        angle = s["positions"].double().T[:, axis] * freq
    return -angle if case.get("inverse", False) else angle


def _turn(x, cos, sin, case):
    """x [tokens, heads, d] turned pair by pair; channels past ``rot`` as they are."""
    rot = case["rot"]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if case["adjacent"] else (slice(0, rot // 2), slice(rot // 2, rot))
    y = x.clone()
    y[..., a] = x[..., a] * cos[:, None] - x[..., b] * sin[:, None]
    y[..., b] = x[..., b] * cos[:, None] + x[..., a] * sin[:, None]
    return y


def _plain_rotary(s):
    angle = _angles(s)
    cos, sin = angle.cos().float(), angle.sin().float()
    return tuple(_turn(x.float(), cos, sin, s["case"]).to(x.dtype) for x in (s["q"], s["new_k"]))


def _plain_append(s):
    case, page, top = s["case"], s["case"]["page"], MAX_CODE[s["case"]["code"]]
    lengths, table, cu = s["lengths"].long(), s["table"].long(), s["cu"].long()
    n, dev, t = lengths.numel(), lengths.device, s["new_k"].shape[0]
    angle = _angles(s)
    cos, sin = angle.cos().float(), angle.sin().float()
    seq = torch.searchsorted(cu[1:], torch.arange(t, device=dev), right=True)
    first = lengths - (cu[1:] - cu[:-1])  # a sequence's tokens before this call
    pos = first[seq] + torch.arange(t, device=dev) - cu[seq]
    pages, slot = table[seq, pos // page], pos % page
    begun = table[torch.arange(n, device=dev), first.clamp(max=lengths - 1) // page]  # the page that the first new token enters
    held = first % page != 0                                                          # and whether it holds earlier tokens
    for x, codes, scale in ((_turn(s["new_k"].float(), cos, sin, case), s["k"], s["k_scale"]), (s["new_v"].float(), s["v"], s["v_scale"])):
        amax = x.abs().amax(-1)
        m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1)
        mt, et = math.frexp(top)
        e = torch.where(amax > 0, e - et + (m > mt), MIN_EXP).clamp(min=MIN_EXP)
        old = scale[begun]
        fresh = torch.zeros_like(scale)
        fresh.scatter_reduce_(0, pages[:, None].expand(-1, scale.shape[1]), torch.exp2(e.float()), "amax")
        grown = torch.maximum(fresh[begun], torch.where(held[:, None], old, 0.0))
        # every sequence owns its pages, so each row of `begun` is written once
        fresh[begun] = grown
        ratio = torch.where(held[:, None], old / grown, 1.0)[:, :, None, None]
        codes[begun] = (codes[begun].float() * ratio).to(codes.dtype)
        scale[pages] = fresh[pages]
        h = torch.arange(scale.shape[1], device=dev)[None, :]
        codes[pages[:, None], h, slot[:, None]] = (x / scale[pages][:, :, None]).clamp(-top, top).to(codes.dtype)
    q = None if s["q"] is None else _turn(s["q"].float(), cos, sin, case).to(s["q"].dtype)
    return q, s["k"], s["v"], s["k_scale"], s["v_scale"]


def _plain_extend(s):
    """Chunks padded to the longest, a block of their rows at a time so that the scores fit."""
    case, table, cu = s["case"], s["table"].long(), s["cu"].long()
    n, cols = table.shape
    (t, hq, d), hkv, page = s["q"].shape, case["hkv"], case["page"]
    dev, group, longest = s["q"].device, hq // hkv, max(s["new"])

    def rows(codes, scale):  # [n, hkv, 1, tokens, d]
        x = codes[table].float().mul_(scale[table][..., None, None])
        return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, 1, cols * page, d)

    k, v = rows(s["k"], s["k_scale"]).transpose(3, 4), rows(s["v"], s["v_scale"])
    at = torch.arange(longest, device=dev)
    here = at[None, :] < (cu[1:] - cu[:-1])[:, None]
    idx = torch.clamp(cu[:-1, None] + at[None, :], max=t - 1)
    qf = s["q"].float()[idx].view(n, longest, hkv, group, d).permute(0, 2, 3, 1, 4)
    seen = s["lengths"].long()[:, None] - (cu[1:] - cu[:-1])[:, None] + 1 + at[None, :]
    key = torch.arange(cols * page, device=dev)
    of = torch.empty(n, hkv, group, longest, d, device=dev)
    step = max(1, min(longest, (3 << 30) // (n * hq * cols * page)))
    for a in range(0, longest, step):
        b = min(longest, a + step)
        p = torch.matmul(qf[..., a:b, :], k)
        p.mul_(d ** -0.5).masked_fill_((key >= seen[:, a:b, None])[:, None, None], -math.inf)
        p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
        torch.matmul(p, v, out=of[..., a:b, :])
        of[..., a:b, :] /= p.sum(-1, keepdim=True).clamp(min=1e-30)
    out = torch.empty(t, hq, d, dtype=s["q"].dtype, device=dev)
    out[idx[here]] = of.permute(0, 3, 1, 2, 4)[here].reshape(-1, hq, d).to(out.dtype)
    return out


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if not own:
        return {"rotary": _plain_rotary, "append": _plain_append, "extend": _plain_extend}[case["op"]](s)
    from linear_attention_recurrence_kda_gb300 import binding as kda
    if case["op"] == "extend":
        cache = kda.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        return kda.kda_attention_extend(s["q"], cache, s["table"], s["lengths"], cu_seqlens=s["cu"])
    rotary = kda.make_rotary(case["rot"], base=10000.0, sections=_sections(case) if case["axes"] else None, adjacent=case["adjacent"])
    if case["op"] == "rotary":
        return kda.kda_rotary(rotary, s["q"], s["new_k"], positions=s["positions"], lengths=s["lengths"], cu_seqlens=s["cu"],
                              inverse=case["inverse"])
    cache = kda.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    q = kda.kda_rotary_append(rotary, s["new_k"], s["new_v"], cache, s["table"], s["lengths"], q=s["q"], positions=s["positions"],
                              cu_seqlens=s["cu"])
    return q, s["k"], s["v"], s["k_scale"], s["v_scale"]


# ---------------------------------------------------------------- 64 bits

def _exact_turn(x, s):
    """Pairs as complex numbers, each multiplied by exp(i angle)."""
    case, rot = s["case"], s["case"]["rot"]
    y = x.double().clone()
    part = y[..., :rot].unflatten(-1, (-1, 2)) if case["adjacent"] else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
    pairs = torch.view_as_complex(part.contiguous())
    angle = torch.cat([_exact_angles(s, n) for n in range(len(s["new"]))])
    pairs = torch.view_as_real(pairs * torch.polar(torch.ones_like(angle), angle)[:, None])
    y[..., :rot] = (pairs if case["adjacent"] else pairs.transpose(-1, -2)).flatten(-2)
    return y


def _exact_angles(s, n):
    case, new, dev = s["case"], s["new"], s["cu"].device
    freq = torch.tensor([10000.0 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)], dtype=torch.float64, device=dev)
    if s["positions"] is None:
        place = torch.arange(s["lens"][n] - new[n], s["lens"][n], device=dev).double()[:, None].expand(-1, len(freq))
    else:
        start, (a, b, _) = sum(new[:n]), _sections(case)
        axis = [0 if i < a else 1 if i < a + b else 2 for i in range(len(freq))]
        place = s["positions"][axis, start:start + new[n]].double().T
    return (-1.0 if case.get("inverse", False) else 1.0) * place * freq


def exact(case, seed):
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_turn(s["q"], s), _exact_turn(s["new_k"], s)
    if case["op"] == "append":
        return _exact_append(s)
    dev, d, hq = s["q"].device, case["d"], case["hq"]
    group = hq // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    start = 0
    for n, (length, new) in enumerate(zip(s["lens"], s["new"])):
        pages = s["table"][n, :-(-length // case["page"])].long()
        for h in range(case["hkv"] if new else 0):
            k, v = ((s[x][pages, h].double() * s[x + "_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:length]
                    for x in ("k", "v"))
            step = max(1, (1 << 27) // (length * group))
            for a in range(0, new, step):
                b = min(new, a + step)
                q = s["q"][start + a:start + b, h * group:(h + 1) * group].double().reshape(-1, d)
                seen = torch.arange(length - new + a + 1, length - new + b + 1, device=dev).repeat_interleave(group)
                z = (q @ k.T) / math.sqrt(d)
                z = torch.where(torch.arange(length, device=dev) < seen[:, None], z, -math.inf)
                e = torch.exp(z - z.max(1, keepdim=True).values)
                out[start + a:start + b, h * group:(h + 1) * group] = ((e @ v) / e.sum(1, keepdim=True)).view(-1, group, d)
        start += new
    return out


def _exact_append(s):
    """The definition taken page by page: each page's largest value sets the scale, then every value is rounded."""
    case, top, page = s["case"], MAX_CODE[s["case"]["code"]], s["case"]["page"]
    if sum(s["new"]) // page + 2 * len(s["new"]) > 4000:
        return None
    answers = [None if s["q"] is None else _exact_turn(s["q"], s)]
    scales = []
    for x, name in ((_exact_turn(s["new_k"], s), "k"), (s["new_v"].double(), "v")):
        codes, scale = s[name].double(), s[name + "_scale"].double()
        start = 0
        for n, (length, new) in enumerate(zip(s["lens"], s["new"])):
            first = length - new
            while first < length:
                last = min(length, (first // page + 1) * page)
                at, slot = int(s["table"][n, first // page]), first % page
                rows = x[start:start + last - first].transpose(0, 1)
                amax = rows.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / top))
                e = torch.where(top * torch.exp2(e - 1) >= amax, e - 1, torch.where(top * torch.exp2(e) < amax, e + 1, e))
                unit = torch.exp2(torch.where(amax > 0, e, float(MIN_EXP)).clamp(min=MIN_EXP))
                if slot:
                    unit = torch.maximum(unit, scale[at])
                    codes[at] = _nearest(codes[at] * (scale[at] / unit)[:, None, None])
                scale[at] = unit
                codes[at, :, slot:slot + last - first] = _nearest(rows / unit[:, None, None])
                start += last - first
                first = last
        answers.append(codes)
        scales.append(scale)
    return tuple(answers + scales)


def _nearest(x):
    """x in 64 bits to the nearest value of e4m3, ties to even."""
    step = torch.exp2(torch.clamp(torch.frexp(x).exponent.double() - 1, min=-6.0) - 3)  # three bits after the first
    return torch.clamp(torch.round(x / step) * step, -448.0, 448.0)
