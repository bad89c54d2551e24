"""Cases of appending to a paged KV cache and of attention over its pages by chunks and with a window, with their plain forms.

The operators: packed query, key and value rows normed per head (optionally), rotated by their positions, the queries
returned and keys and values put into their pages; attention of each sequence's last rows (a prompt's chunk, tokens to be
verified, single ones) over the pages, with or without a sliding window and a few first positions that stay visible; and
attention of one new token per sequence with such a window.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of four requests of the 2.3B model: rotated, a row each appended
        dict(name="append-step-4", op="append", rows="f16", cache="f16", batch=4, lo=1, hi=1, before=1000, hq=20, hkv=4, hd=128,
             rot=128, norm=False, theta=1e4, page=16, seed=1),
        # ragged prompts of the 8B-class model with normed queries and keys, quantised as they are appended
        dict(name="append-prompts-norm-e4m3", op="append", rows="bf16", cache="e4m3", batch=9, lo=33, hi=1024, before=0, hq=32,
             hkv=8, hd=128, rot=128, norm=True, theta=5e5, page=32, seed=2),
        # long prompts, up to the 8B-class model's whole context, half of every head rotated
        dict(name="append-long-bf16", op="append", rows="bf16", cache="bf16", batch=5, lo=5001, hi=8192, before=300, hq=32, hkv=8,
             hd=128, rot=64, norm=False, theta=5e5, page=64, seed=3),
        # the tiny model: 16 tokens behind a short cached prefix, latency
        dict(name="chunk-tiny", op="chunk", rows="f16", cache="f16", batch=1, lo=16, hi=16, least=61, before=61, hq=4, hkv=2,
             hd=64, window=0, sinks=0, page=16, seed=4),
        # 32 requests verify up to eight proposed tokens each over quantised caches
        dict(name="chunk-verify-32-e4m3", op="chunk", rows="bf16", cache="e4m3", batch=32, lo=2, hi=8, least=500, before=8000,
             hq=32, hkv=8, hd=128, window=0, sinks=0, page=64, seed=5),
        # a server's mixed pass of the 2.3B model: prompts' chunks and single tokens
        dict(name="chunk-mixed-f16", op="chunk", rows="f16", cache="f16", batch=16, lo=1, hi=601, least=0, before=3000, hq=20,
             hkv=4, hd=128, window=0, sinks=0, page=16, seed=6),
        # the last 2,048 tokens of a prompt as long as the 8B-class model's context
        dict(name="chunk-2048-bf16", op="chunk", rows="bf16", cache="bf16", batch=1, lo=2048, hi=2048, least=6144, before=6144,
             hq=32, hkv=8, hd=128, window=0, sinks=0, page=32, seed=7),
        # a long document's chunk with a window and four first positions
        dict(name="chunk-window-bf16", op="chunk", rows="bf16", cache="bf16", batch=2, lo=1001, hi=2001, least=20000,
             before=30000, hq=32, hkv=8, hd=128, window=4096, sinks=4, page=64, seed=8),
        # four requests of the 2.3B model with a short window: latency
        dict(name="window-decode-4", op="decode", rows="f16", cache="f16", batch=4, lo=1, hi=1, least=500, before=1023, hq=20,
             hkv=4, hd=128, window=256, sinks=4, page=16, seed=9),
        # a full server: contexts from nothing to four windows, quantised
        dict(name="window-decode-64-e4m3", op="decode", rows="bf16", cache="e4m3", batch=64, lo=1, hi=1, least=0, before=16000,
             hq=32, hkv=8, hd=128, window=4096, sinks=4, page=64, seed=10),
        # one request, far behind its window
        dict(name="window-decode-1-long", op="decode", rows="bf16", cache="bf16", batch=1, lo=1, hi=1, least=131010,
             before=131010, hq=32, hkv=8, hd=128, window=32768, sinks=64, page=32, seed=11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(4, 2), (20, 4), (32, 8), (16, 4), (8, 8), (8, 1), (14, 2), (24, 2)])
    rows = rng.choice(["f16", "bf16"])
    c = dict(op=rng.choice(["append", "chunk", "chunk", "decode"]), rows=rows, cache=rng.choice([rows, "e4m3"]), hq=hq, hkv=hkv,
             hd=rng.choice([64, 128]), page=rng.choice([8, 16, 32, 64, 128]), seed=rng.randrange(1 << 20))
    if c["op"] == "append":
        c["hi"] = _log_int(rng, 1, 8192)
        c["lo"] = rng.randint(1, c["hi"])
        c["before"] = rng.choice([0, rng.randint(1, 2000)])
        c["rot"] = rng.choice([c["hd"], c["hd"], c["hd"] // 2])
        c["norm"] = rng.random() < 0.5
        c["theta"] = rng.choice([1e4, 5e5])
        c["batch"] = _log_int(rng, 1, max(1, min(64, int(1.5e8 / ((hq + 2 * hkv) * c["hd"] * c["hi"])))))
        return c
    c["window"] = rng.choice([0, _log_int(rng, 1, 8192)])
    c["sinks"] = rng.choice([0, rng.randint(1, 80)]) if c["window"] else 0
    if c["op"] == "decode":
        c["window"] = c["window"] or _log_int(rng, 16, 8192)
        c["lo"] = c["hi"] = 1
        c["before"] = _log_int(rng, 1, 32768)
        c["least"] = rng.randint(0, c["before"])
        c["batch"] = _log_int(rng, 1, max(1, min(128, int(2.0e8 / (hkv * c["hd"] * c["before"] * BYTES[c["cache"]])))))
        return c
    c["hi"] = _log_int(rng, 1, 2048)
    c["lo"] = rng.randint(1, c["hi"])
    c["before"] = _log_int(rng, 1, 16384)
    c["least"] = rng.randint(0, c["before"])
    most = min(4.0e8 / (hq * c["hi"] * (c["hi"] + c["before"])), 1.0e8 / (hkv * c["hd"] * (c["hi"] + c["before"])))
    c["batch"] = _log_int(rng, 1, max(1, min(48, int(most))))
    return c


def _rows(c):
    """New rows of every sequence, the first one's the most."""
    r = random.Random(c["seed"])
    return [c["hi"]] + [r.randint(c["lo"], c["hi"]) if c["op"] != "chunk" or r.random() > 0.4 else c["lo"] for _ in range(c["batch"] - 1)]


def _before(c):
    """Cached positions in front of every sequence's new rows."""
    r = random.Random(c["seed"] + 1)
    return [r.randint(c.get("least", 0), c["before"]) for _ in range(c["batch"])]


def _pairs(c):
    """Pairs of a row and a position that it sees, and the positions that some row sees."""
    pairs = seen = 0
    w, first = c["window"], c["sinks"]
    for m, b in zip(_rows(c), _before(c)):
        if not w:
            pairs += m * b + m * (m + 1) // 2
            seen += b + m
            continue
        for p in range(b, b + m):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(first, low)
        low = max(0, b - w + 1)
        seen += b + m - low + min(first, low)
    return pairs, seen


def work(case):
    c, n = case, sum(_rows(case))
    cell = c["hd"] * BYTES[c["cache"]] + (4 if c["cache"] == "e4m3" else 0)
    if c["op"] == "append":
        table = max(m + b for m, b in zip(_rows(c), _before(c))) * c["rot"] * 4
        return {"bytes": n * ((2 * c["hq"] + 2 * c["hkv"]) * c["hd"] * BYTES[c["rows"]] + 2 * c["hkv"] * cell) + table,
                "flops": n * (c["hq"] + c["hkv"]) * (3 * c["rot"] + (4 * c["hd"] if c["norm"] else 0))}
    pairs, seen = _pairs(c)
    return {"bytes": 2 * seen * c["hkv"] * cell + 2 * n * c["hq"] * c["hd"] * BYTES[c["rows"]],
            "flops": 4 * pairs * c["hq"] * c["hd"]}


# ---------------------------------------------------------------- inputs

def _cumulative(lens, dev):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=dev)


def _quantise(x):
    """e4m3 codes and their scale per row, from fp32 rows [..., hd]."""
    s = (x.abs().amax(-1, keepdim=True) / E4M3_MAX).clamp(min=SCALE_MIN)
    return (x / s).to(torch.float8_e4m3fn), s.squeeze(-1)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rows(*shape):
        # a few channels are larger than the rest, as queries and keys of real models have them
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
        x[..., 3::32] *= 3.0
        return x.to(DT[c["rows"]])

    new, before = _rows(c), _before(c)
    total = [m + b for m, b in zip(new, before)]
    hkv, hd, ps = c["hkv"], c["hd"], c["page"]
    need = [-(-m // ps) for m in total]
    n_pages = sum(need) + 7
    width = max(1, max(need))
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    at = _cumulative(need, dev)
    col = torch.arange(width, device=dev)
    held = col[None, :] < (at[1:] - at[:-1])[:, None]
    index = (at[:-1, None] + col[None, :]).clamp(max=n_pages - 1)
    table = torch.where(held, order[index.long()], -1).to(torch.int32)  # unused entries name no page

    s = dict(case=c, table=table, lens=torch.tensor(total, dtype=torch.int32, device=dev), cu=_cumulative(new, dev), n=sum(new),
             most=max(new), k_scale=None, v_scale=None, q_gain=None, k_gain=None)
    for name in ("k", "v"):
        pages = rows(n_pages, hkv, ps, hd)
        if c["cache"] == "e4m3":
            s[name + "_pages"], s[name + "_scale"] = _quantise(pages.float())
        else:
            s[name + "_pages"] = pages
        del pages
    if c["op"] != "append":
        s["q"] = rows(s["n"], c["hq"], hd)
        return s
    # the rows of one fused projection
    qkv = rows(s["n"], c["hq"] + 2 * hkv, hd)
    s["q"], s["k"], s["v"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + hkv], qkv[:, c["hq"] + hkv:]
    half = c["rot"] // 2
    turn = torch.arange(half, device=dev, dtype=torch.float64) * (-2.0 / c["rot"])
    angle = torch.arange(max(total), device=dev, dtype=torch.float64)[:, None] * torch.pow(c["theta"], turn)[None, :]
    s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
    if c["norm"]:
        for name in ("q_gain", "k_gain"):
            s[name] = (1 + 0.2 * torch.randn(hd, generator=g, device=dev)).to(DT[c["rows"]])
    return s


# ---------------------------------------------------------------- one pass

def _bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _positions(s):
    """Sequence and position of every packed row: the last positions of each sequence."""
    i = torch.arange(s["n"], device=s["table"].device)
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    return b, s["lens"].long()[b] - cu[b + 1] + i


def _normed(x, gain):
    if gain is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()


def _rotated(x, cos, sin):
    """Elements i and i + r of every head are turned by the position's angle i (r angles); the rest stays."""
    r = cos.shape[-1]
    a, b = x[..., :r], x[..., r:2 * r]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * r:]], -1)


def _plain_append(s):
    b, pos = _positions(s)
    ps = s["case"]["page"]
    page, slot = s["table"][b, pos // ps].long(), pos % ps
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotated(_normed(s["q"].float(), s["q_gain"]), cos, sin).to(s["q"].dtype)
    k = _rotated(_normed(s["k"].float(), s["k_gain"]), cos, sin)
    for name, x in (("k", k), ("v", s["v"].float())):
        pages = s[name + "_pages"]
        if pages.dtype == torch.float8_e4m3fn:
            codes, scale = _quantise(x)
            _bits(pages)[page, :, slot] = _bits(codes)
            s[name + "_scale"][page, :, slot] = scale
        else:
            pages[page, :, slot] = x.to(pages.dtype)
    return q


def _plain_attention(s):
    """Rows padded per sequence against the positions that some row may see: the first ones, then the window's span."""
    c = s["case"]
    b, lq = c["batch"], s["most"]
    hq, hkv, hd, ps = c["hq"], c["hkv"], c["hd"], c["page"]
    cu, lens = s["cu"].long(), s["lens"].long()
    n_q = cu[1:] - cu[:-1]
    dev = cu.device
    i = torch.arange(lq, device=dev)
    at = (lens - n_q)[:, None] + i[None, :]  # position of every padded row
    width = s["table"].shape[1] * ps
    if c["window"]:
        low = (lens - n_q - c["window"] + 1).clamp(min=0)
        near = low[:, None] + torch.arange(min(width, lq + c["window"] - 1), device=dev)[None, :]
        first = torch.arange(c["sinks"], device=dev)[None, :].expand(b, -1)
        key = torch.cat([torch.where(first < low[:, None], first, width), near], 1)  # (those in the span already: once)
    else:
        key = torch.arange(width, device=dev)[None, :].expand(b, -1)
    held = key < lens[:, None]
    key = key.clamp(max=width - 1)
    page, slot = s["table"].long().gather(1, key // ps).clamp(min=0), key % ps

    def gathered(name):
        pages = s[name + "_pages"]
        x = _bits(pages)[page, :, slot].view(pages.dtype).float()  # [b, keys, hkv, hd]
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"][page, :, slot][..., None]
        return x.transpose(1, 2)

    seen = held[:, None, :] & (key[:, None, :] <= at[:, :, None])
    if c["window"]:
        seen &= (key[:, None, :] > at[:, :, None] - c["window"]) | (key[:, None, :] < c["sinks"])
    q = s["q"][(cu[:-1, None] + i[None, :]).clamp(max=s["n"] - 1)].float()
    q = q.view(b, lq, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, hd)
    scores = (q @ gathered("k").transpose(-1, -2)).view(b, hkv, hq // hkv, lq, -1).mul_(1 / math.sqrt(hd))
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True).clamp(min=-1e30)
    scores.exp_()
    total = scores.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (scores.view(b, hkv, (hq // hkv) * lq, -1) @ gathered("v")).view(b, hkv, hq // hkv, lq, hd) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(b * lq, hq, hd)
    # back to the packed rows
    r = torch.arange(s["n"], device=dev)
    of = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    return o[of * lq + r - cu[of]].to(s["q"].dtype)


def _own(s):
    from autoregressive_decode_persistent_gb300 import ops

    c = s["case"]
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "append":
        return ops.paged_kv_append(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["q"], s["k"], s["v"], s["cos"],
                                   s["sin"], q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS, **scales)
    if c["op"] == "decode":
        return ops.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], window=c["window"],
                                   sinks=c["sinks"], **scales)
    return ops.paged_chunk_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"],
                                     window=c["window"] or None, sinks=c["sinks"], **scales)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        out = _own(s)
    else:
        out = _plain_append(s) if op == "append" else _plain_attention(s)
    if op == "append":
        return {"q": out, **{k: s[k] for k in ("k_pages", "v_pages", "k_scale", "v_scale") if s[k] is not None}}
    return {"out": out}


# ---------------------------------------------------------------- 64-bit values

def _e4m3_nearest(y):
    """The e4m3 value nearest to each y (ties to the even code), |y| <= 448."""
    e = torch.frexp(y)[1].clamp(min=-5)  # y = m 2^e with m in [0.5, 1): 4 bits of it are kept; 2^-9 is the least step
    step = torch.ldexp(torch.ones_like(y), e - 4)
    return torch.round(y / step) * step


def _turned(x, gain, cos, sin):
    """Rows [n, heads, hd] in 64 bits: normed where there is a gain, then every pair of elements times e^(i angle)."""
    if gain is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * gain.double()
    r = cos.shape[-1]
    z = torch.complex(x[..., :r], x[..., r:2 * r]) * torch.complex(cos, sin)[:, None]
    out = x.clone()
    out[..., :r], out[..., r:2 * r] = z.real, z.imag
    return out


def _exact_append(c, s):
    lens, cu, table = s["lens"].tolist(), s["cu"].tolist(), s["table"].tolist()
    where = [(b, p) for b in range(c["batch"]) for p in range(lens[b] - (cu[b + 1] - cu[b]), lens[b])]
    pos = torch.tensor([p for _, p in where], device="cuda")
    page = torch.tensor([table[b][p // c["page"]] for b, p in where], device="cuda")
    slot = pos % c["page"]
    cos, sin = s["cos"].double()[pos], s["sin"].double()[pos]
    out = {"q": _turned(s["q"].double(), s["q_gain"], cos, sin)}
    for name, x in (("k", _turned(s["k"].double(), s["k_gain"], cos, sin)), ("v", s["v"].double())):
        new = s[name + "_pages"].double()
        if c["cache"] == "e4m3":
            scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
            new[page, :, slot] = _e4m3_nearest(x / scale[..., None])
            scales = s[name + "_scale"].double()
            scales[page, :, slot] = scale
            out[name + "_scale"] = scales
        else:
            new[page, :, slot] = x
        out[name + "_pages"] = new
    return out


def _exact_attention(c, s):
    lens, cu, table = s["lens"].tolist(), s["cu"].tolist(), s["table"].tolist()
    out = torch.zeros(s["n"], c["hq"], c["hd"], dtype=torch.float64, device="cuda")
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(lens):
        if cu[b + 1] == cu[b]:
            continue
        ids = torch.tensor(table[b][:-(-n // c["page"])], device="cuda")
        kv = []
        for name in ("k", "v"):
            x = _bits(s[name + "_pages"]).index_select(0, ids).view(s[name + "_pages"].dtype).double()
            if s[name + "_scale"] is not None:
                x = x * s[name + "_scale"].index_select(0, ids).double().unsqueeze(-1)
            kv.append(x.transpose(0, 1).flatten(1, 2)[:, :n])  # [hkv, n, hd]
        for r0 in range(cu[b], cu[b + 1], 512):
            r1 = min(cu[b + 1], r0 + 512)
            p = n - (cu[b + 1] - torch.arange(r0, r1, device="cuda"))  # positions of these rows
            top = int(p[-1]) + 1
            low = max(0, int(p[0]) - c["window"] + 1) if c["window"] else 0
            keys = torch.cat([torch.arange(min(c["sinks"], low), device="cuda"), torch.arange(low, top, device="cuda")])
            hide = keys[None] > p[:, None]
            if c["window"]:
                hide |= (keys[None] <= p[:, None] - c["window"]) & (keys[None] >= c["sinks"])
            for h in range(c["hkv"]):
                q = s["q"][r0:r1, h * group:(h + 1) * group].double().transpose(0, 1)  # [group, rows, hd]
                w = torch.softmax((q @ kv[0][h, keys].T * c["hd"] ** -0.5).masked_fill(hide[None], -math.inf), -1)
                out[r0:r1, h * group:(h + 1) * group] = (w @ kv[1][h, keys]).transpose(0, 1)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attention(case, s)
