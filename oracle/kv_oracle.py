"""Plain fp64 CPU reference of the low-bit key/value cache and of attention over it (test
infrastructure only).

A cache here is a dict of numpy arrays: codes k, v uint8 [pages, heads, page, D * bits / 8], k_params,
v_params fp16 [pages, heads, page, 2, D / group] and the numbers bits, group, as the library holds it."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

LIMIT = 57344.0
WIDTH = {"k": 4, "v": 16}


def position(D, which):
    """Position of every dimension's code in a row."""
    W = WIDTH[which]
    return np.array([(d % W) * (D // W) + d // W for d in range(D)])


def quantize_group(x, bits):
    """(codes, scale, offset) of one group of values (python floats), in exact arithmetic but for the fp32 and
    fp16 roundings that the definition names."""
    x = [float(v) for v in x]
    if not all(np.isfinite(v) for v in x):
        return [0] * len(x), np.float16(0.0), np.float16(np.nan)
    x = [min(max(v, -LIMIT), LIMIT) for v in x]
    top = 2 ** bits - 1
    o = np.float16(np.float32(min(x)))
    span = np.float32(float(max(x)) - float(o))     # a difference of an fp32 and an fp16 value: fp64 holds it
    s = np.float16(np.float32(max(span, np.float32(0.0))) / np.float32(top))
    if s == 0:
        return [0] * len(x), np.float16(0.0), o
    codes = []
    for v in x:
        q = (Fraction(v) - Fraction(float(o))) / Fraction(float(s))
        codes.append(min(max(round(q), 0), top))    # Fraction rounds halves to the even integer
    return codes, s, o


def quantize_row(x, bits, group):
    """Codes [D], scales and offsets fp16 [D / group] of one row."""
    codes, scales, offsets = [], [], []
    for i in range(0, len(x), group):
        c, s, o = quantize_group(x[i:i + group], bits)
        codes += c
        scales.append(s)
        offsets.append(o)
    return np.array(codes), np.array(scales, np.float16), np.array(offsets, np.float16)


def pack(codes, bits, which):
    """Bytes of a row of codes [D]."""
    D = len(codes)
    row = np.zeros(D, np.uint8)
    row[position(D, which)] = codes
    return row if bits == 8 else (row[0::2] | (row[1::2] << 4)).astype(np.uint8)


def store(K, V, slots, cache):
    """Writes the rows [T, heads, D] of every token into its slot, in order."""
    pages, heads, page = cache["k"].shape[:3]
    bits, group = cache["bits"], cache["group"]
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if not 0 <= slot < pages * page:
            continue
        p, i = divmod(slot, page)
        for which, x in (("k", K), ("v", V)):
            for h in range(heads):
                c, s, o = quantize_row(x[t, h], bits, group)
                cache[which][p, h, i] = pack(c, bits, which)
                cache[which + "_params"][p, h, i, 0] = s
                cache[which + "_params"][p, h, i, 1] = o


def values(cache, which, pages, places):
    """fp64 values [n, heads, D] of the rows at (page, place)."""
    bits, group = cache["bits"], cache["group"]
    rows = cache[which][pages, :, places]
    if bits == 4:
        rows = np.stack([rows & 15, rows >> 4], -1).reshape(*rows.shape[:-1], 2 * rows.shape[-1])
    D = rows.shape[-1]
    codes = rows[..., position(D, which)].astype(np.float64)
    p = cache[which + "_params"][pages, :, places].astype(np.float64)
    g = np.arange(D) // group
    return codes * p[..., 0, :][..., g] + p[..., 1, :][..., g]


def load(cache, slots):
    """fp64 (K, V) [T, heads, D]; zeros for slots outside the pool."""
    pages, heads, page = cache["k"].shape[:3]
    slots = np.asarray(slots, np.int64)
    has = (slots >= 0) & (slots < pages * page)
    out = []
    for which in ("k", "v"):
        x = values(cache, which, slots[has] // page, slots[has] % page)
        y = np.zeros((len(slots), heads, x.shape[-1]))
        y[has] = x
        out.append(y)
    return tuple(out)


def attention(Q, cache, table, kv_len, cu_q=None, scale=None, causal=True, window=0, sinks=None, max_q=None):
    """fp64 out [T, q_heads, D], lse [T, q_heads] and, for error bounds, a dict of
      qk   largest scale * sum |q| (|c s| + |o|) over the seen tokens, per row
      pv   sum_t w_t (|c s| + |o|) per element, w the weights of the softmax
      seen number of tokens seen, per row (-1: row of no sequence).
    A row that sees nothing: zeros."""
    Q = np.asarray(Q, np.float64)
    T, A, D = Q.shape
    pages, heads, page = cache["k"].shape[:3]
    table, kv_len = np.asarray(table), np.asarray(kv_len)
    B = len(kv_len)
    cu = np.arange(B + 1) if cu_q is None else np.asarray(cu_q)
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((T, A, D)), np.full((T, A), -np.inf)
    mag = dict(qk=np.zeros((T, A)), pv=np.zeros((T, A, D)), seen=np.full(T, -1))
    absolute = dict(cache)
    for which in ("k", "v"):
        absolute[which + "_params"] = np.abs(cache[which + "_params"])
    for b in range(B):
        q0 = min(max(int(cu[b]), 0), T)
        q1 = min(max(int(cu[b + 1]), q0), T)
        n = q1 - q0
        length = min(max(int(kv_len[b]), 0), table.shape[1] * page)
        t = np.arange(length)
        pg = table[b][t // page] if length else np.zeros(0, int)
        ok = (pg >= 0) & (pg < pages)
        t, pg = t[ok], pg[ok]
        k, v = (values(cache, which, pg, t % page) for which in ("k", "v"))
        ka, va = (values(absolute, which, pg, t % page) for which in ("k", "v"))
        for i in range(n if max_q is None else min(n, max_q)):
            pos = length - n + i
            see = np.ones(len(t), bool)
            if causal:
                see &= t <= pos
            if window:
                see &= t > pos - window
            mag["seen"][q0 + i] = see.sum()
            for a in range(A):
                h = a // (A // heads)
                s = scale * (k[see, h] @ Q[q0 + i, a])
                if sinks is not None:
                    s = np.append(s, float(sinks[a]))
                if len(s) == 0:
                    continue
                top = s.max()
                w = np.exp(s - top)
                total = w.sum()
                w = w[:see.sum()] / total
                out[q0 + i, a] = w @ v[see, h]
                lse[q0 + i, a] = top + np.log(total)
                mag["qk"][q0 + i, a] = abs(scale) * (ka[see, h] @ np.abs(Q[q0 + i, a])).max(initial=0.0)
                mag["pv"][q0 + i, a] = w @ va[see, h]
    return out, lse, mag
