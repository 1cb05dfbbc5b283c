"""Operators of a low-bit key/value cache: quantizing it as it is written, reading it back, and
attention over it.

Three operators, each as a user's program calls it:

  store   the keys and values of new tokens, quantized into the cache's pages, and read back from there
          as the values the codes stand for
  load    rows of the cache as values
  attend  softmax(scale Q K^T) V over the cached tokens of every sequence, and the logarithm of each
          row's sum, for one new token per sequence, a few, or a chunk of a prompt

A token's key (or value) of one head is D codes of 4 or 8 bits; `group` consecutive dimensions share a
fp16 scale s and offset o, and a code c stands for c s + o.  Pages hold [heads][page] such rows:
codes [pages][heads][page][D bits / 8] bytes, parameters fp16 [pages][heads][page][2][D / group]
(scales, then offsets).  Dimension d is the code at position (d % W) (D / W) + d / W of its row, least
significant bits first, with W = 4 for keys and 16 for values.

`own` False computes them in elementary torch operations in 32 bits, True through the framework's
entry points.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LIMIT = 57344.0  # values are clamped to this magnitude


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of one request on phi4 heads: latency only
        dict(name="attend_b1", op="attend", B=1, L=1500, least=1.0, q=1, heads=40, kv=10, D=128, bits=4, group=64,
             page=16, window=0, sinks=False, type="bf16"),
        # a decode batch of 32 requests of very different lengths, odd ones among them
        dict(name="attend_b32", op="attend", B=32, L=8191, least=0.001, q=1, heads=40, kv=10, D=128, bits=4,
             group=64, page=64, window=0, sinks=False, type="f16"),
        # a large decode batch at long context: the cache is what is read
        dict(name="attend_b64_long", op="attend", B=64, L=16384, least=0.5, q=1, heads=40, kv=10, D=128, bits=4,
             group=64, page=64, window=0, sinks=False, type="bf16"),
        # a GPT-OSS sliding-window layer with sinks, 64 heads of 64 dimensions
        dict(name="attend_window", op="attend", B=48, L=4000, least=0.1, q=1, heads=64, kv=8, D=64, bits=4, group=32,
             page=32, window=128, sinks=True, type="f16"),
        # four tokens of every sequence at once (drafted tokens being checked), 8-bit cache
        dict(name="attend_q4", op="attend", B=16, L=6001, least=0.2, q=4, heads=32, kv=4, D=128, bits=8, group=128,
             page=16, window=0, sinks=False, type="bf16"),
        # one key/value head of 256 dimensions, a few very long sequences, fine groups
        dict(name="attend_d256", op="attend", B=3, L=40000, least=0.3, q=1, heads=8, kv=1, D=256, bits=4, group=32,
             page=128, window=0, sinks=False, type="f16"),
        # the last 2048 tokens of an 8192-token prompt on phi4 heads
        dict(name="attend_prompt", op="attend", B=1, L=8192, least=1.0, q=2048, heads=40, kv=10, D=128, bits=4,
             group=64, page=64, window=0, sinks=False, type="bf16"),
        # prompts of odd lengths together, 64 dimensions with sinks, 8-bit cache
        dict(name="attend_prompts", op="attend", B=5, L=3001, least=0.05, q=777, heads=64, kv=8, D=64, bits=8,
             group=64, page=16, window=0, sinks=True, type="f16"),
        # a decode step's 32 new tokens, taken from the fp32 output of the fused projection
        dict(name="store_t32", op="store", T=32, heads=40, kv=10, D=128, bits=4, group=64, page=64, order="mixed",
             type="f32"),
        # a prompt of 8191 tokens, 8-bit
        dict(name="store_t8191", op="store", T=8191, heads=32, kv=4, D=128, bits=8, group=128, page=16,
             order="runs", type="bf16"),
        # a few hundred tokens read back, scattered
        dict(name="load_t333", op="load", T=333, heads=64, kv=8, D=64, bits=4, group=32, page=16, order="mixed",
             type="f16"),
        # the whole of a long sequence read back
        dict(name="load_t65536", op="load", T=65536, heads=40, kv=10, D=128, bits=4, group=64, page=64, order="runs",
             type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    D = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8, 10])
    case = dict(op=rng.choice(["attend", "attend", "attend", "store", "load"]), heads=kv * rng.choice([1, 2, 4, 5, 8]),
                kv=kv, D=D, bits=rng.choice([4, 4, 8]), group=rng.choice([g for g in (32, 64, 128) if g <= D]),
                page=rng.choice([16, 32, 64, 256]), type=rng.choice(["f16", "bf16"]))
    if case["op"] != "attend":
        case.update(T=_log(rng, 1, 8192), order=rng.choice(["mixed", "runs"]))
        if rng.random() < 0.3:
            case["type"] = "f32"
        return case
    kind = rng.choice(["one", "one", "few", "prompt"])
    if kind == "prompt":
        B, L = rng.randint(1, 4), _log(rng, 17, 4096)
        q = min(L, _log(rng, 16, 1024), (1 << 35) // (B * L * case["heads"] * D))
    else:
        B, L = _log(rng, 1, 64), _log(rng, 1, 16384)
        L = min(L, (1 << 31) // (B * kv * D * case["bits"]))
        q = 1 if kind == "one" else rng.randint(2, 8)
    case.update(B=B, L=L, q=q, least=rng.choice([0.01, 0.3, 1.0]), sinks=rng.choice([False, False, True]),
                window=rng.choice([0, 0, 0, 128, _log(rng, 1, 2000)]))
    return case


def _lengths(case):
    """(tokens in the cache, new ones among them) of every sequence: the first has the greatest number."""
    rng = random.Random(case["B"] * 1000003 + case["L"])
    lens, news = [], []
    for b in range(case["B"]):
        n = case["L"] if b == 0 else max(1, int(case["L"] * rng.uniform(case["least"], 1.0)))
        lens.append(n)
        # chunks of a prompt differ in length, drafted tokens do not
        news.append(min(n, case["q"] if b == 0 or case["q"] <= 8 else rng.randint(1, case["q"])))
    return lens, news


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pools(case, pages):
    """Empty pages: codes and parameters of keys and values."""
    H, page, D = case["kv"], case["page"], case["D"]
    codes = [torch.zeros(pages, H, page, D * case["bits"] // 8, dtype=torch.uint8, device="cuda") for _ in range(2)]
    params = [torch.zeros(pages, H, page, 2, D // case["group"], dtype=torch.float16, device="cuda")
              for _ in range(2)]
    return dict(k=codes[0], v=codes[1], k_params=params[0], v_params=params[1], bits=case["bits"],
                group=case["group"])


def _heads(case, rows, g, which):
    """Rows of keys (some dimensions far from zero in every token, as keys have them) or values."""
    x = torch.randn(rows, case["kv"], case["D"], generator=g, device="cuda")
    if which == "k":
        bias = torch.randn(case["kv"], case["D"], generator=g, device="cuda")
        x += torch.where(bias > 1.5, 2.0 * bias, torch.zeros_like(bias))
    return x


def _fill(case, s, g):
    """Every page filled with quantized rows."""
    c = s["cache"]
    pages, H, page = c["k"].shape[:3]
    step = max(1, (1 << 26) // (H * page * case["D"]))
    for which, W in (("k", 4), ("v", 16)):
        for i in range(0, pages, step):
            j = min(pages, i + step)
            x = _heads(case, (j - i) * page, g, which)
            code, scale, offset = _quantize(x, case["bits"], case["group"], torch.float32)
            rows = _pack(code, case["bits"], W)
            c[which][i:j] = rows.view(j - i, page, H, -1).transpose(1, 2)
            p = torch.stack([scale, offset], 2).to(torch.float16)
            c[which + "_params"][i:j] = p.view(j - i, page, H, 2, -1).transpose(1, 2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    ty = TYPES[case["type"]]
    s = dict(case=case, type=ty)
    H, D, page = case["kv"], case["D"], case["page"]
    if case["op"] != "attend":
        T = case["T"]
        pages = -(-T // page) + 3
        s["cache"] = _pools(case, pages)
        if case["order"] == "runs":  # page after page, in any order of pages
            order = torch.randperm(pages, generator=g, device="cuda")
            at = torch.arange(T, device="cuda") + int(torch.randint(0, page, (1,), generator=g, device="cuda"))
            slots = order[at // page] * page + at % page
        else:
            slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
        hole = torch.rand(T, generator=g, device="cuda") < (0.02 if T > 8 else 0.0)
        s["slots"] = torch.where(hole, torch.full_like(slots, -1), slots).to(torch.int32)
        if case["op"] == "load":
            _fill(case, s, g)
            return s
        # keys and values as slices of the fused projection's output
        fused = torch.empty(T, (case["heads"] + 2 * H) * D, dtype=ty, device="cuda")
        fused[:, :case["heads"] * D] = 1.0
        k, v = (fused[:, (case["heads"] + i * H) * D:(case["heads"] + (i + 1) * H) * D] for i in range(2))
        k.copy_(_heads(case, T, g, "k").view(T, H * D))
        v.copy_(_heads(case, T, g, "v").view(T, H * D))
        s["K"], s["V"] = k.view(T, H, D), v.view(T, H, D)
        return s
    lens, news = _lengths(case)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    s["cache"] = _pools(case, pages)
    _fill(case, s, g)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(case["B"], max(need), dtype=torch.int32, device="cuda")
    i = 0
    for b, n in enumerate(need):
        table[b, :n] = order[i:i + n]
        i += n
    s["table"] = table
    s["lens"], s["news"] = lens, news
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    s["cu_q"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    # queries as a slice of the fused projection's output
    T = starts[-1]
    fused = torch.randn(T, (case["heads"] + 2 * H) * D, generator=g, device="cuda").to(ty)
    s["Q"] = fused[:, :case["heads"] * D].view(T, case["heads"], D)
    s["sinks"] = torch.randn(case["heads"], generator=g, device="cuda") if case["sinks"] else None
    return s


# ---------------------------------------------------------------------------
# the operators in elementary operations, in 32 bits
# ---------------------------------------------------------------------------

def _quantize(x, bits, group, wide=torch.float64):
    """Codes [T, H, D], scales and offsets [T, H, D / group] of rows x; the rounding of a code in 64 bits."""
    T, H, D = x.shape
    x = x.float().view(T, H, D // group, group)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    x = torch.clamp(torch.where(bad, torch.zeros_like(x), x), -LIMIT, LIMIT)
    offset = x.amin(-1, keepdim=True).to(torch.float16).float()
    span = x.amax(-1, keepdim=True) - offset
    scale = (span / torch.full_like(span, 2 ** bits - 1)).to(torch.float16).float()
    scale = torch.clamp(scale, min=0.0)
    some = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = torch.round((x.to(wide) - offset.to(wide)) / some.to(wide)).clamp(0, 2 ** bits - 1)
    code = torch.where(scale > 0, code, torch.zeros_like(code))
    offset = torch.where(bad, torch.full_like(offset, float("nan")), offset)
    scale = torch.where(bad, torch.zeros_like(scale), scale)
    return code.to(torch.uint8).view(T, H, D), scale[..., 0], offset[..., 0]


def _pack(code, bits, W):
    """Bytes [T, H, D bits / 8] of codes in the order of the rows."""
    T, H, D = code.shape
    code = code.view(T, H, D // W, W).transpose(2, 3).reshape(T, H, D)
    if bits == 8:
        return code
    pair = code.view(T, H, D // 2, 2)
    return pair[..., 0] | (pair[..., 1] << 4)


def _values(rows, params, bits, W):
    """Values (..., D) in 32 bits of rows of bytes and their parameters (..., 2, D / group)."""
    if bits == 4:
        rows = torch.stack([rows & 15, rows >> 4], -1).flatten(-2)
    D = rows.shape[-1]
    code = rows.unflatten(-1, (W, D // W)).transpose(-1, -2).flatten(-2).float()
    p = params.float()
    G = p.shape[-1]
    return (code.unflatten(-1, (G, D // G)) * p[..., 0, :, None] + p[..., 1, :, None]).flatten(-2)


def _plain_load(s):
    c, slots = s["cache"], s["slots"].long()
    page = c["k"].shape[2]
    has = (slots >= 0)
    at = torch.where(has, slots, torch.zeros_like(slots))
    out = []
    for which, W in (("k", 4), ("v", 16)):
        rows = c[which][at // page, :, at % page]
        x = _values(rows, c[which + "_params"][at // page, :, at % page], c["bits"], W)
        out.append(torch.where(has[:, None, None], x, torch.zeros_like(x)).to(s["type"]))
    return tuple(out)


def _plain_store(s):
    c, slots = s["cache"], s["slots"].long()
    page = c["k"].shape[2]
    # rows without a place go where the first one does, with its content
    has = slots >= 0
    first = torch.argmax(has.int())
    row = torch.where(has, torch.arange(slots.numel(), device="cuda"), first)
    at = slots[row]
    for which, x, W in (("k", s["K"], 4), ("v", s["V"], 16)):
        code, scale, offset = _quantize(x, c["bits"], c["group"])
        c[which][at // page, :, at % page] = _pack(code, c["bits"], W)[row]
        c[which + "_params"][at // page, :, at % page] = torch.stack([scale, offset], 2).to(torch.float16)[row]
    return _plain_load(s)


def _plain_attend(s):
    case, c = s["case"], s["cache"]
    heads, H, D, page = case["heads"], case["kv"], case["D"], case["page"]
    R = heads // H
    out = torch.empty_like(s["Q"], memory_format=torch.contiguous_format)
    lse = torch.empty(out.shape[0], heads, device="cuda")
    lens, news = s["lens"], s["news"]
    scale = D ** -0.5
    b0, row = 0, 0
    while b0 < len(lens):
        # sequences with the same number of queries together, as far as the memory of a step goes
        b1, n = b0 + 1, news[b0]
        longest = lens[b0]
        while b1 < len(lens) and news[b1] == n and (b1 + 1 - b0) * max(longest, lens[b1]) * H * D < (1 << 30):
            longest = max(longest, lens[b1])
            b1 += 1
        nb, np = b1 - b0, -(-longest // page)
        L = np * page
        table = s["table"][b0:b1, :np].long()
        kv = []
        for which, W in (("k", 4), ("v", 16)):
            x = _values(c[which][table], c[which + "_params"][table], c["bits"], W)  # [nb, np, H, page, D]
            kv.append(x.transpose(1, 2).reshape(nb, H, L, D))
        q = s["Q"][row:row + nb * n].float().view(nb, n, H, R, D).permute(0, 2, 1, 3, 4).reshape(nb, H, n * R, D)
        score = torch.matmul(q, kv[0].transpose(2, 3).contiguous()) * scale
        length = s["kv_len"][b0:b1, None, None].long()
        at = length - n + torch.arange(n, device="cuda")[None, :, None]  # position of each query
        t = torch.arange(L, device="cuda")[None, None, :]
        seen = (t <= at) & (t < length)
        if case["window"]:
            seen &= t > at - case["window"]
        seen = seen[:, None, :, None, :].expand(nb, H, n, R, L).reshape(nb, H, n * R, L)
        score = score.masked_fill(~seen, -float("inf"))
        top = score.amax(-1, keepdim=True)
        if s["sinks"] is not None:
            sink = s["sinks"].view(1, H, 1, R).expand(nb, H, n, R).reshape(nb, H, n * R, 1)
            top = torch.maximum(top, sink)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        if s["sinks"] is not None:
            total = total + torch.exp(sink - top)
        o = torch.matmul(p, kv[1]) / torch.where(total > 0, total, torch.ones_like(total))
        o = o.view(nb, H, n, R, D).permute(0, 2, 1, 3, 4).reshape(nb * n, heads, D)
        out[row:row + nb * n] = o.to(s["type"])
        lse[row:row + nb * n] = (top + torch.log(total)).view(nb, H, n, R).permute(0, 2, 1, 3).reshape(nb * n, heads)
        b0, row = b1, row + nb * n
    return out, lse


# ---------------------------------------------------------------------------
# the operators through the framework
# ---------------------------------------------------------------------------

def _own(s):
    from gemm_qmm_nbits_amd import qmm as Q

    case = s["case"]
    if case["op"] == "attend":
        one = max(s["news"]) == 1
        return Q.qkv_attention(s["Q"], s["cache"], s["table"], s["kv_len"], cu_q=None if one else s["cu_q"],
                               max_q=max(s["news"]), max_kv=case["L"], window=case["window"], sinks=s["sinks"],
                               need_lse=True)
    if case["op"] == "store":
        Q.qkv_cache_store(s["K"], s["V"], s["slots"], s["cache"])
    return Q.qkv_cache_load(s["cache"], s["slots"], out_dtype=s["type"])


def run(s):
    if own:
        return _own(s)
    return {"attend": _plain_attend, "store": _plain_store, "load": _plain_load}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    H, D = case["kv"], case["D"]
    size = 4 if case["type"] == "f32" else 2
    row = D * case["bits"] / 8 + 4 * D / case["group"]  # bytes of a key or value of one head
    if case["op"] != "attend":
        held = 2 * case["T"] * H * row
        values = 2 * case["T"] * H * D * size
        if case["op"] == "load":
            return {"bytes": held + values + 4 * case["T"], "flops": 4.0 * case["T"] * H * D}
        return {"bytes": 2 * (held + values) + 8 * case["T"], "flops": 14.0 * case["T"] * H * D}
    lens, news = _lengths(case)
    read, pairs = 0, 0
    for n, q in zip(lens, news):
        counts = [max(0, p + 1) for p in range(n - q, n)]
        if case["window"]:
            counts = [min(x, case["window"]) for x in counts]
        pairs += sum(counts)
        first = max(0, n - q + 1 - case["window"]) if case["window"] else 0
        read += n - first
    T = sum(news)
    io = 2 * T * case["heads"] * D * size + 4 * T * case["heads"] + 4 * read // case["page"]
    return {"bytes": 2 * read * H * row + io, "flops": 4.0 * pairs * case["heads"] * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(case, c, which, pages, places):
    """Values in 64 bits [n, H, D] of the rows at these pages and places."""
    D, bits, W = case["D"], case["bits"], 4 if which == "k" else 16
    d = torch.arange(D, device="cuda")
    at = (d % W) * (D // W) + torch.div(d, W, rounding_mode="floor")
    rows = c[which][pages, :, places].to(torch.int64)
    per = 8 // bits
    byte = rows[..., torch.div(at, per, rounding_mode="floor")]
    code = torch.remainder(torch.div(byte, (2 ** bits) ** (at % per), rounding_mode="floor"), 2 ** bits)
    p = c[which + "_params"][pages, :, places].double()
    g = torch.div(d, case["group"], rounding_mode="floor")
    return code.double() * p[..., 0, :][..., g] + p[..., 1, :][..., g]


def exact(case, seed):
    s = prepare(case, seed)
    c, page = s["cache"], case["page"]
    if case["op"] == "attend":
        return _exact_attend(case, s)
    slots = s["slots"].long()
    T, H, D = case["T"], case["kv"], case["D"]
    out = []
    for which in ("k", "v"):
        y = torch.zeros(T, H, D, dtype=torch.float64, device="cuda")
        for i in range(0, T, 4096):
            rows = i + torch.nonzero(slots[i:i + 4096] >= 0)[:, 0]
            if case["op"] == "load":
                y[rows] = _exact_rows(case, c, which, slots[rows] // page, slots[rows] % page)
                continue
            # the parameters are what fp16 (by way of fp32) makes of each group's least value and range; a
            # code is the integer next to the quotient, halves to the even one
            x = s[which.upper()][rows].double().clamp(-LIMIT, LIMIT).unflatten(-1, (-1, case["group"]))
            top = 2 ** case["bits"] - 1
            low = x.min(-1, keepdim=True).values.float().half().double()
            span = (x.max(-1, keepdim=True).values - low).float()
            step = (span / torch.full_like(span, top)).half().double().clamp(min=0)
            n = (x - low) / torch.where(step == 0, torch.ones_like(step), step)
            down = torch.floor(n)
            over = n - down
            up = (over > 0.5) | ((over == 0.5) & (torch.remainder(down, 2) == 1))
            code = torch.minimum(torch.maximum(down + up.double(), torch.zeros_like(n)), torch.full_like(n, top))
            y[rows] = (low + torch.where(step == 0, torch.zeros_like(n), code) * step).flatten(-2)
        out.append(y)
    return tuple(out)


def _exact_attend(case, s):
    heads, H, D, page = case["heads"], case["kv"], case["D"], case["page"]
    R = heads // H
    T = s["Q"].shape[0]
    out = torch.zeros(T, heads, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, heads), -float("inf"), dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, q) in enumerate(zip(s["lens"], s["news"])):
        first = max(0, n - q + 1 - case["window"]) if case["window"] else 0
        t = torch.arange(first, n, device="cuda")
        pages = s["table"][b].long()[torch.div(t, page, rounding_mode="floor")]
        k, v = (_exact_rows(case, s["cache"], which, pages, t % page) for which in ("k", "v"))
        place = torch.arange(n - q, n, device="cuda")
        away = place[:, None] - t[None, :]
        hidden = away < 0
        if case["window"]:
            hidden = hidden | (away >= case["window"])
        for h in range(heads):
            a = (s["Q"][row:row + q, h].double() @ k[:, h // R].T.contiguous()) / math.sqrt(D)
            a = a.masked_fill(hidden, -float("inf"))
            if s["sinks"] is not None:
                a = torch.cat([a, s["sinks"][h].double().expand(q, 1)], 1)
            norm = torch.logsumexp(a, 1)
            w = torch.exp(a - torch.where(torch.isinf(norm), torch.zeros_like(norm), norm)[:, None])
            out[row:row + q, h] = w[:, :t.numel()] @ v[:, h // R].contiguous()
            lse[row:row + q, h] = norm
        row += q
    return out, lse
