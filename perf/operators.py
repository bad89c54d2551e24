"""Cases of the paged KV cache operators and of packed prompt attention, with their plain forms.

The operators: writing packed K/V rows into a paged cache (16-bit, or e4m3 with a scale per row and head), reading
cached rows back, attention of one new token per sequence over the pages, and causal attention over packed prompts.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of four requests appends a row each
        dict(name="write-step-4", op="write", rows="f16", cache="f16", batch=4, lo=1, hi=1, before=1000, hkv=4, hd=128,
             page=16, seed=1),
        # ragged prompts of the 8B-class model (up to its prompt length) into an e4m3 cache
        dict(name="write-prompts-e4m3", op="write", rows="bf16", cache="e4m3", batch=9, lo=33, hi=1024, before=0, hkv=8,
             hd=128, page=32, seed=2),
        # long prompts (the model's whole context each) quantised as they are written
        dict(name="write-long-e4m3", op="write", rows="bf16", cache="e4m3", batch=5, lo=5001, hi=8192, before=300, hkv=8,
             hd=128, page=64, seed=3),
        # a short cached prefix back in 16 bits
        dict(name="read-prefix-e4m3", op="read", rows="f16", cache="e4m3", batch=1, lo=517, hi=517, before=0, hkv=4,
             hd=128, page=16, seed=4),
        # the caches of many requests gathered for a chunk of prompts
        dict(name="read-many-bf16", op="read", rows="bf16", cache="bf16", batch=12, lo=600, hi=8192, before=0, hkv=8,
             hd=128, page=32, seed=5),
        # the tiny model, one request: latency
        dict(name="decode-tiny", op="decode", rows="f16", cache="f16", batch=1, lo=77, hi=77, hq=4, hkv=2, hd=64,
             page=16, seed=6),
        # four requests of the 2.3B model at contexts 513 to 1024
        dict(name="decode-4-f16", op="decode", rows="f16", cache="f16", batch=4, lo=513, hi=1024, hq=20, hkv=4, hd=128,
             page=16, seed=7),
        # one request with a long context
        dict(name="decode-1-long", op="decode", rows="bf16", cache="bf16", batch=1, lo=131011, hi=131011, hq=32, hkv=8,
             hd=128, page=32, seed=8),
        # a full server: 64 slots, some empty, ragged contexts, quantised cache
        dict(name="decode-64-e4m3", op="decode", rows="bf16", cache="e4m3", batch=64, lo=0, hi=8192, hq=32, hkv=8,
             hd=128, page=64, seed=9),
        # the tiny model's 16-token prompt: latency
        dict(name="prompt-16", op="prompt", rows="f16", batch=1, lo=16, hi=16, prefix=0, hq=4, hkv=2, hd=64, seed=10),
        # ragged prompts of the 2.3B model, some continuing a cached prefix
        dict(name="prompts-ragged-f16", op="prompt", rows="f16", batch=12, lo=19, hi=1024, prefix=512, hq=20, hkv=4,
             hd=128, seed=11),
        # one long prompt of the 8B-class model (its whole context)
        dict(name="prompt-8192-bf16", op="prompt", rows="bf16", batch=1, lo=8192, hi=8192, prefix=0, hq=32, hkv=8,
             hd=128, seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(4, 2), (20, 4), (32, 8), (16, 4), (8, 8), (8, 1), (14, 2), (24, 2)])
    c = dict(op=rng.choice(["write", "read", "decode", "prompt"]), rows=rng.choice(["f16", "bf16"]),
             hkv=hkv, hd=rng.choice([64, 128]), seed=rng.randrange(1 << 20))
    if c["op"] == "prompt":
        c["hq"] = hq
        c["hi"] = _log_int(rng, 1, 4096)
        c["lo"] = rng.randint(max(1, c["hi"] // 8), c["hi"])
        c["prefix"] = rng.choice([0, 0, _log_int(rng, 1, 2048)])
        most = int(2.0e9 / (hq * c["hi"] * (c["hi"] + c["prefix"])))
        c["batch"] = _log_int(rng, 1, max(1, min(24, most)))
        return c
    c["cache"] = rng.choice([c["rows"], "e4m3"])
    c["page"] = rng.choice([8, 16, 32, 64, 128])
    if c["op"] == "decode":
        c["hq"] = hq
        c["hi"] = _log_int(rng, 1, 32768)
        c["lo"] = rng.randint(0, c["hi"])
        most = int(2.6e8 / (hkv * c["hd"] * c["hi"] * BYTES[c["cache"]]))
        c["batch"] = _log_int(rng, 1, max(1, min(256, most)))
        return c
    c["hi"] = _log_int(rng, 1, 8192)
    c["lo"] = rng.randint(1, c["hi"])
    c["before"] = rng.choice([0, rng.randint(1, 700)]) if c["op"] == "write" else 0
    c["batch"] = _log_int(rng, 1, max(1, min(64, int(3.0e7 / (hkv * c["hd"] * c["hi"])))))
    return c


def _lens(c):
    """Length of every sequence (new or cached rows), the first the longest."""
    r = random.Random(c["seed"])
    return [c["hi"]] + [r.randint(c["lo"], c["hi"]) if c["lo"] or r.random() > 0.1 else 0 for _ in range(c["batch"] - 1)]


def _more(c, key):
    """Cached positions in front of every sequence's own rows."""
    r = random.Random(c["seed"] + 1)
    return [r.randint(0, c[key]) for _ in range(c["batch"])]


def work(case):
    c, n = case, sum(_lens(case))
    if c["op"] in ("write", "read"):
        cached = c["hkv"] * (c["hd"] * BYTES[c["cache"]] + (4 if c["cache"] == "e4m3" else 0))
        return {"bytes": 2 * n * (c["hkv"] * c["hd"] * BYTES[c["rows"]] + cached), "flops": 0}
    if c["op"] == "decode":
        cached = c["hkv"] * (c["hd"] * BYTES[c["cache"]] + (4 if c["cache"] == "e4m3" else 0))
        return {"bytes": 2 * n * cached + 2 * c["batch"] * c["hq"] * c["hd"] * BYTES[c["rows"]],
                "flops": 4 * n * c["hq"] * c["hd"]}
    pre = _more(c, "prefix")
    pairs = sum(m * p + m * (m + 1) // 2 for m, p in zip(_lens(c), pre))
    return {"bytes": 2 * c["hd"] * BYTES[c["rows"]] * (n * c["hq"] + (n + sum(pre)) * c["hkv"]),
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
        # a few channels are larger than the rest, as keys and values of real models have them
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
        x[..., 3::32] *= 3.0
        return x.to(DT[c["rows"]])

    lens = _lens(c)
    hkv, hd = c["hkv"], c["hd"]
    if c["op"] == "prompt":
        k_lens = [m + p for m, p in zip(lens, _more(c, "prefix"))]
        return dict(case=c, q=rows(sum(lens), c["hq"], hd), k=rows(sum(k_lens), hkv, hd), v=rows(sum(k_lens), hkv, hd),
                    cu_q=_cumulative(lens, dev), cu_k=_cumulative(k_lens, dev), max_q=max(lens), max_k=max(k_lens))

    before = _more(c, "before") if c["op"] == "write" else [0] * c["batch"]
    total = [m + p for m, p in zip(lens, before)]
    ps = c["page"]
    need = [-(-m // ps) for m in total]
    n_pages = sum(need) + 7
    width = max(1, max(need))
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    at = _cumulative(need, dev)
    col = torch.arange(width, device=dev)
    held = col[None, :] < (at[1:] - at[:-1])[:, None]
    index = (at[:-1, None] + col[None, :]).clamp(max=n_pages - 1)
    table = torch.where(held, order[index.long()], -1).to(torch.int32)  # unused entries name no page

    s = dict(case=c, table=table, lens=torch.tensor(total, dtype=torch.int32, device=dev),
             cu=_cumulative(lens, dev), n=sum(lens), k_scale=None, v_scale=None)
    for name in ("k", "v"):
        pages = rows(n_pages, hkv, ps, hd)
        if c["cache"] == "e4m3":
            s[name + "_pages"], s[name + "_scale"] = _quantise(pages.float())
        else:
            s[name + "_pages"] = pages
    if c["op"] == "write":
        s["k"], s["v"] = rows(s["n"], hkv, hd), rows(s["n"], hkv, hd)
    if c["op"] == "decode":
        s["q"] = rows(c["batch"], c["hq"], hd)
    return s


# ---------------------------------------------------------------- one pass

def _row_places(s):
    """Page and slot of every packed row: the last rows of each sequence's positions."""
    i = torch.arange(s["n"], device=s["table"].device)
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    pos = s["lens"].long()[b] - cu[b + 1] + i
    ps = s["case"]["page"]
    return s["table"][b, pos // ps].long(), pos % ps


def _bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_write(s):
    page, slot = _row_places(s)
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        if pages.dtype == torch.float8_e4m3fn:
            codes, scale = _quantise(s[name].float())
            _bits(pages)[page, :, slot] = _bits(codes)
            s[name + "_scale"][page, :, slot] = scale
        else:
            pages[page, :, slot] = s[name].float().to(pages.dtype)


def _plain_read(s):
    page, slot = _row_places(s)
    out = []
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        x = _bits(pages)[page, :, slot].view(pages.dtype).float()
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"][page, :, slot][..., None]
        out.append(x.to(DT[s["case"]["rows"]]))
    return out


def _softmax_sum(scores, seen, v):
    """softmax over the seen keys (0 where none is) times v, in fp32."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, 1.0, total)


def _plain_decode(s):
    c = s["case"]
    b, width = s["table"].shape
    hkv, hd, ps = c["hkv"], c["hd"], c["page"]
    page = s["table"].long().clamp(min=0)
    seen = torch.arange(width * ps, device=page.device)[None, :] < s["lens"][:, None]

    def gathered(name):
        pages = s[name + "_pages"]
        x = _bits(pages)[page].view(pages.dtype).float()  # [b, width, hkv, ps, hd]
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"][page][..., None]
        return x.transpose(1, 2).reshape(b, hkv, width * ps, hd)

    q = s["q"].float().view(b, hkv, c["hq"] // hkv, hd)
    scores = (q @ gathered("k").transpose(-1, -2)) / math.sqrt(hd)
    return _softmax_sum(scores, seen[:, None, None, :], gathered("v")).reshape(b, c["hq"], hd).to(s["q"].dtype)


def _plain_prompt(s):
    c = s["case"]
    b, hq, hkv, hd = c["batch"], c["hq"], c["hkv"], c["hd"]
    lq, lk = s["max_q"], s["max_k"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    n_q, n_k = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(lq, device=cu_q.device), torch.arange(lk, device=cu_q.device)

    def padded(x, cu, at):
        return x[(cu[:-1, None] + at[None, :]).clamp(max=x.shape[0] - 1)].float()  # [b, l, h, hd]

    q = padded(s["q"], cu_q, i).view(b, lq, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, hd)
    k = padded(s["k"], cu_k, j).transpose(1, 2)
    v = padded(s["v"], cu_k, j).transpose(1, 2)
    seen = (j[None, None, :] <= i[None, :, None] + (n_k - n_q)[:, None, None]) & (j[None, :] < n_k[:, None])[:, None, :]
    scores = (q @ k.transpose(-1, -2)).view(b, hkv, hq // hkv, lq, lk) / math.sqrt(hd)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True).clamp(min=-1e30)
    scores.exp_()
    total = scores.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (scores.view(b, hkv, -1, lk) @ v).view(b, hkv, hq // hkv, lq, hd) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(b * lq, hq, hd)
    # back to the packed rows
    r = torch.arange(s["q"].shape[0], device=cu_q.device)
    at = torch.searchsorted(cu_q[1:].contiguous(), r, right=True)
    return o[at * lq + r - cu_q[at]].to(s["q"].dtype)


def _own(s):
    from autoregressive_decode_persistent_gb300 import ops

    op = s["case"]["op"]
    if op == "prompt":
        return ops.packed_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
    if op == "decode":
        return ops.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "read":
        return ops.paged_kv_read(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["n"],
                                 dtype=DT[s["case"]["rows"]], k_scale=s["k_scale"], v_scale=s["v_scale"])
    ops.paged_kv_write(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["k"], s["v"],
                       k_scale=s["k_scale"], v_scale=s["v_scale"])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        out = _own(s)
    else:
        out = {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "prompt": _plain_prompt}[op](s)
    if op == "write":
        return {k: s[k] for k in ("k_pages", "v_pages", "k_scale", "v_scale") if s[k] is not None}
    return {"k": out[0], "v": out[1]} if op == "read" else {"out": out}


# ---------------------------------------------------------------- 64-bit values

def _e4m3_nearest(y):
    """The e4m3 value nearest to each y (ties to the even code), |y| <= 448."""
    e = torch.frexp(y)[1].clamp(min=-5)  # y = m 2^e with m in [0.5, 1): 4 bits of it are kept; 2^-9 is the least step
    step = torch.ldexp(torch.ones_like(y), e - 4)
    return torch.round(y / step) * step


def _exact_cache(c, s):
    """Per sequence, the K and V positions in 64 bits [len, hkv, hd], by its own table row."""
    table, lens = s["table"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        got = []
        for name in ("k", "v"):
            x = torch.zeros(n, c["hkv"], c["hd"], dtype=torch.float64, device="cuda")
            if n:
                ids = torch.tensor(table[b][:-(-n // c["page"])], device="cuda")
                x = s[name + "_pages"].view(torch.uint8).index_select(0, ids).view(s[name + "_pages"].dtype).double()
                if s[name + "_scale"] is not None:
                    x = x * s[name + "_scale"].index_select(0, ids).double().unsqueeze(-1)
                x = x.permute(0, 2, 1, 3).flatten(0, 1)[:n]
            got.append(x)
        yield got


def _attend(q, k, v, first):
    """Rows of q [m, hq, hd] at positions first.. over k, v [n, hkv, hd]; row i sees keys up to first + i."""
    m, hq, hd = q.shape
    hkv = k.shape[1]
    out = torch.zeros(m, hq, hd, dtype=torch.float64, device=q.device)
    for at in range(0, m, 1024):
        end = min(m, at + 1024)
        n = min(k.shape[0], first + end)
        if n <= 0:
            continue
        for h in range(hq):
            kh, vh = k[:n, h * hkv // hq], v[:n, h * hkv // hq]
            w = (q[at:end, h] @ kh.T) * hd ** -0.5
            last = first + torch.arange(at, end, device=q.device)
            hide = torch.arange(n, device=q.device)[None, :] > last[:, None]
            w[hide] = -math.inf
            o = torch.softmax(w, 1) @ vh
            o[last < 0] = 0
            out[at:end, h] = o
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "prompt":
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        return {"out": torch.cat([
            _attend(s["q"][cq[b]:cq[b + 1]].double(), s["k"][ck[b]:ck[b + 1]].double(), s["v"][ck[b]:ck[b + 1]].double(),
                    (ck[b + 1] - ck[b]) - (cq[b + 1] - cq[b])) for b in range(c["batch"])])}
    if c["op"] == "decode":
        out = [_attend(s["q"][b:b + 1].double(), k, v, k.shape[0] - 1) for b, (k, v) in enumerate(_exact_cache(c, s))]
        return {"out": torch.cat(out)}
    if c["op"] == "read":
        got = list(_exact_cache(c, s))
        return {"k": torch.cat([k for k, _ in got]), "v": torch.cat([v for _, v in got])}
    out = {}
    table, cu, lens = s["table"].tolist(), s["cu"].tolist(), s["lens"].tolist()
    page, slot = [], []
    for b in range(c["batch"]):
        for p in range(lens[b] - (cu[b + 1] - cu[b]), lens[b]):
            page.append(table[b][p // c["page"]])
            slot.append(p % c["page"])
    page, slot = torch.tensor(page, device="cuda"), torch.tensor(slot, device="cuda")
    for name in ("k", "v"):
        x = s[name].double()
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
