"""GPU parity of attention over the low-bit cache (qkv_attention) against the fp64 oracle.

Bounds, with u = 2^-24 and everything taken from the oracle's magnitudes: a score is a sum of D products
of exact operands, the scales' and the offsets' products (fp32 throughout), so it is off by dS <=
gamma(D + 16) qk + 8 u qk + 100 u, qk the largest scale sum |q| (|c s| + |o|); the last terms are the score's
roundings in units of log2 and its distance from the reference exponent (which lies within 40 of a score).
A weight is off by 2 dS (its own and the sum's), the sums by gamma(seen + 64).  For bf16 results either
e^S s is rounded to fp16 once, half a step, 2^-11 of each term, or e^S and c s + o are, twice that (with their
product 2^-10 + 2^-22); for fp16 ones e^S s is held by two fp16 values, 2^-22; for terms
below 2^-20 of the largest 2^-25 against a largest of at least 2^5 (2^-30), times the largest code and scale."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q
from oracle import kv_oracle as KO

from gpu_util import U32, assert_elementwise, dev, gamma, host_bits, host_f64, say, torch

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def tt(name):
    return getattr(torch(), DT[name])


class Problem:
    """Sequences with `lens` tokens in the cache, the last `news` of each as queries."""

    def __init__(self, lens, news, heads=8, kv=2, D=64, bits=4, group=32, page=16, ty="bf16", seed=0, spare=2,
                 q_std=1.0, v_std=1.0, extra=0):
        t = torch()
        rng = np.random.default_rng(seed)
        self.lens, self.news, self.ty, self.bits = list(lens), list(news), ty, bits
        self.heads, self.kv, self.D, self.page = heads, kv, D, page
        B = len(lens)
        need = [max(1, -(-n // page)) for n in lens]
        pages = sum(need) + spare
        self.cache = Q.qkv_cache_new(pages, kv, D, bits=bits, group=group, page=page)
        # every slot filled (those past a sequence's end too) in one call
        n = pages * page
        x = rng.standard_normal((2, n, kv, D)) * np.array([1.0, v_std]).reshape(2, 1, 1, 1)
        x[0] += rng.standard_normal((1, kv, D))
        K, V = (t.from_numpy(a.astype(np.float32)).cuda() for a in x)
        Q.qkv_cache_store(K, V, dev(np.arange(n, dtype=np.int32)), self.cache)
        order = rng.permutation(pages)
        self.table_h = np.full((B, max(need)), -1, np.int32)
        i = 0
        for b, c in enumerate(need):
            self.table_h[b, :c] = order[i:i + c]
            i += c
        self.table, self.kv_len = dev(self.table_h), dev(np.array(lens, np.int32))
        self.cu_h = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.cu = dev(self.cu_h)
        self.T = int(self.cu_h[-1]) + extra
        self.Q = t.from_numpy(rng.standard_normal((self.T, heads, D)) * q_std).to(tt(ty)).cuda()

    def host_cache(self):
        c = dict(bits=self.cache["bits"], group=self.cache["group"])
        for w in ("k", "v"):
            c[w] = self.cache[w].cpu().numpy()
            c[w + "_params"] = self.cache[w + "_params"].cpu().numpy()
        return c

    def call(self, **kw):
        one = all(n == 1 for n in self.news) and self.T == len(self.news) and not kw.pop("force_cu", False)
        a = dict(cu_q=None if one else self.cu, need_lse=True)
        if not one:
            a["max_q"] = max(self.news)
        a.update(kw)
        return Q.qkv_attention(self.Q, self.cache, self.table, self.kv_len, **a)


def worst_share(y, ref, bound, ty):
    """Of the excess over the result's own rounding, the part of the bound that it takes."""
    u = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[ty]
    over = np.abs(y - ref) - u * np.abs(ref) - {"f16": 2.0 ** -24, "bf16": 2.0 ** -133}[ty]
    return float(np.max(np.where(bound > 0, over / np.maximum(bound, 1e-300), 0.0), initial=0.0))


def check(p, label="", oracle=None, **kw):
    """One call against the oracle; returns (out, lse)."""
    say(f"  {label} lens={p.lens[:6]} news={p.news[:6]} heads={p.heads}/{p.kv} D={p.D} bits={p.bits} "
        f"group={p.cache['group']} page={p.page} {p.ty} {sorted(kw)}")
    out, lse = p.call(**kw)
    ref, rl, mag = KO.attention(host_f64(p.Q), p.host_cache(), p.table_h, p.lens, cu_q=p.cu_h,
                                scale=kw.get("scale"), causal=kw.get("causal", True), window=kw.get("window", 0),
                                sinks=None if kw.get("sinks") is None else host_f64(kw["sinks"]))
    own = mag["seen"] >= 0
    n = np.maximum(mag["seen"], 0)[:, None]
    dS = gamma(p.D + 16) * mag["qk"] + U32 * (8 * mag["qk"] + 100)
    step = float(p.cache["v_params"][:, :, :, 0].float().nan_to_num().max())
    weights = 2.0 ** -22 if p.ty == "f16" else 2.0 ** -10 + 2.0 ** -22
    bound = mag["pv"] * (weights + 2 * dS + gamma(n + 64.0))[..., None] + (n * 2.0 ** (p.bits - 30) * step)[..., None]
    assert_elementwise(host_f64(out)[own], ref[own], bound[own], p.ty, label + " out")
    seen = np.isfinite(rl) & own[:, None]
    got = host_f64(lse)
    assert np.array_equal(np.isneginf(got[own]), np.isneginf(rl[own]))
    lim = 2 * dS + gamma(n + 64.0) + 2.0 ** -22 * (np.abs(np.where(np.isfinite(rl), rl, 0.0)) + 40)
    say(f"    largest share of the bound: out {worst_share(host_f64(out)[own], ref[own], bound[own], p.ty):.3f}")
    worst = np.abs(got[seen] - rl[seen]) / np.broadcast_to(lim, got.shape)[seen]
    assert worst.size == 0 or worst.max() <= 1.0, (label, "lse", worst.max())
    return out, lse


FORMATS = [(4, 64, 32), (4, 64, 64), (4, 128, 32), (4, 128, 64), (4, 128, 128), (4, 256, 32), (4, 256, 64),
           (4, 256, 128), (8, 64, 32), (8, 64, 64), (8, 128, 32), (8, 128, 64), (8, 128, 128), (8, 256, 32),
           (8, 256, 64), (8, 256, 128)]


@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_single_tokens(bits, D, group, ty):
    """One query per sequence: lengths of one, on and off the tiles (32) and pages, none."""
    p = Problem([1, 15, 16, 17, 0, 33, 100, 257, 640], [1] * 9, heads=8, kv=2, D=D, bits=bits, group=group, ty=ty,
                seed=D + bits)
    check(p, "single")


# Past 64 rows of one cache head, calls that expect much work take another kernel: with MUCH tokens expected
# these small ones do too.
MUCH = 1 << 30
KERNELS = pytest.mark.parametrize("kv", [None, MUCH], ids=["few", "many"])


# queries per sequence, with four heads per cache head: up to 16 rows, 32, two row tiles and many
@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("news", [[4, 3, 1], [8, 5, 2], [16, 9, 13], [70, 33, 1]])
def test_several_tokens(bits, D, group, news):
    p = Problem([90, 41, 13], news, heads=4, kv=1, D=D, bits=bits, group=group, seed=sum(news) + D)
    check(p, "several")


@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_many_rows(bits, D, group, ty):
    """Row tiles of 128 with rows missing, in parts that join."""
    p = Problem([90, 41, 13], [70, 33, 1], heads=4, kv=1, D=D, bits=bits, group=group, seed=D + group, ty=ty)
    check(p, "many", max_kv=MUCH)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_many_rows_in_one_part(D, page):
    """Work-groups enough that none is split: the results are written directly."""
    p = Problem([150, 100, 70, 333], [70, 65, 70, 1], heads=72, kv=72, D=D, group=64, page=page, seed=D)
    check(p, "one part", max_kv=MUCH)


def test_many_work_groups_and_some_left_over():
    """More than one round of work-groups, of which the rest is split."""
    p = Problem([140, 130, 129, 131, 70], [130, 66, 129, 66, 67], heads=60, kv=60, D=64, group=64, seed=3)
    check(p, "left over", max_kv=MUCH)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (5, 1), (10, 2), (40, 10), (16, 1), (17, 1), (64, 8), (72, 1)])
@pytest.mark.parametrize("new", [1, 3])
def test_head_layouts(heads, kv, new):
    p = Problem([70, 35], [new, new], heads=heads, kv=kv, seed=heads)
    check(p, "heads")


@pytest.mark.parametrize("page", [16, 32, 64, 128, 512])
@pytest.mark.parametrize("new", [1, 40])
@KERNELS
def test_pages(page, new, kv):
    """Pages that end inside a tile and tables with more pages than tokens."""
    p = Problem([16, 200, 531, 49], [new if n >= new else n for n in (16, 200, 531, 49)], page=page, seed=page)
    check(p, "pages", max_kv=kv)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 100, 10 ** 6, 2 ** 40])
@pytest.mark.parametrize("new", [1, 5, 90])
@KERNELS
def test_windows(window, new, kv):
    t = torch()
    p = Problem([300, 95, 4], [new, new, min(new, 4)], seed=new)
    check(p, "window", window=window, max_kv=kv)
    check(p, "window, sinks", window=window, sinks=t.linspace(-3, 3, p.heads, device="cuda"), max_kv=kv)


@pytest.mark.parametrize("new", [1, 20, 100])
@KERNELS
def test_not_causal(new, kv):
    p = Problem([130, 101, 300], [new] * 3, seed=new)
    check(p, "all tokens", causal=False, max_kv=kv)


@pytest.mark.parametrize("news", [[5, 5, 5], [30, 40, 9]])
@KERNELS
def test_queries_that_see_nothing(news, kv):
    """More queries than tokens: the first ones stand before the sequence."""
    t = torch()
    p = Problem([3, 0, 1], news, seed=2)
    out, lse = check(p, "nothing", max_kv=kv)
    assert not bool(out[news[0]:news[0] + news[1]].any())
    sinks = t.randn(p.heads, device="cuda")
    out, lse = check(p, "nothing, sinks", sinks=sinks, max_kv=kv)
    assert bool((lse[news[0]] == sinks).all())


@pytest.mark.parametrize("sink", [-200.0, 0.0, 5.0, 300.0, float("-inf")])
def test_sinks(sink):
    t = torch()
    p = Problem([200, 1000, 1], [1, 1, 1], seed=5)
    sinks = t.full((p.heads,), sink, device="cuda")
    check(p, "sinks", sinks=sinks)
    check(p, "sinks, parts", sinks=sinks, max_kv=100000)
    p = Problem([200, 77], [50, 77], seed=6)
    check(p, "sinks, many rows", sinks=sinks)
    check(p, "sinks, many rows, parts", sinks=sinks, max_kv=MUCH)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 1e-3])
def test_scales(scale):
    check(Problem([130, 64], [1, 1], seed=7), "scale", scale=scale)
    check(Problem([130, 64], [33, 20], seed=7), "scale", scale=scale)
    check(Problem([130, 64], [33, 20], seed=7), "scale", scale=scale, max_kv=MUCH)


@pytest.mark.parametrize("max_kv", [1, 300, 2000, 20000, 10 ** 9])
@pytest.mark.parametrize("news", [[1, 1, 1], [6, 2, 1], [100, 50, 1]])
def test_parts(max_kv, news):
    """The tokens in one part to many (more than there are tiles among them), whatever the lengths are."""
    p = Problem([1500, 70, 1], news, heads=4, kv=1, seed=8)
    check(p, "parts", max_kv=max_kv)


def test_long():
    for ty in ("bf16", "f16"):
        p = Problem([20011, 5], [1, 1], heads=4, kv=1, D=128, group=64, seed=9, ty=ty)
        check(p, "long")
        p = Problem([20011, 5], [1, 1], heads=4, kv=1, D=256, group=32, seed=9, ty=ty)
        check(p, "long")
    p = Problem([9000], [3], heads=4, kv=1, D=128, bits=8, group=128, seed=10, ty="f16")
    check(p, "long")


@pytest.mark.parametrize("std,v_std", [(30.0, 1.0), (1e-3, 1e-3), (5.0, 100.0), (1.0, 3e-4)])
@pytest.mark.parametrize("new", [1, 70])
@KERNELS
def test_ranges(std, v_std, new, kv):
    """Peaked and flat softmax, large and small values (scales down to fp16's subnormals)."""
    check(Problem([300, 90], [new, new], q_std=std, v_std=v_std, seed=11), "ranges", max_kv=kv)


@pytest.mark.parametrize("new", [1, 90])
@KERNELS
def test_value_scales_that_grow(new, kv):
    """Later tokens with scales a million times the first ones', in one group of several: the reference exponent
    follows, whatever the scores do."""
    t = torch()
    p = Problem([400], [new], D=128, group=32, seed=12, page=16)
    pages = p.table_h[0]
    for i, pg in enumerate(pages):
        p.cache["v_params"][int(pg), :, :, :, 1] *= float(2.0 ** (i % 13 - 6))
    check(p, "growing", max_kv=kv)
    for i, pg in enumerate(pages):
        p.cache["k_params"][int(pg)] *= float(2.0 ** ((i % 5) - 2))
    check(p, "growing scores", max_kv=kv)
    t.cuda.synchronize()


@pytest.mark.parametrize("new", [1, 6, 70])
@KERNELS
def test_hidden_tokens_do_not_leak(new, kv):
    """NaN in tokens behind the sequence, before the window, after a query's position, on pages that are not in the
    table, and any bits there: the results of rows that do not see them keep every bit."""
    t = torch()
    p = Problem([100, 77], [new, new], page=16, seed=13)
    window = 30
    clean = [host_bits(x).copy() for x in p.call(window=window, max_kv=kv)]
    # all slots of no sequence, and those behind each sequence's end
    used = np.zeros((p.cache["k"].shape[0], 16), bool)
    for b, n in enumerate(p.lens):
        for tok in range(n):
            used[p.table_h[b, tok // 16], tok % 16] = True
    hide = t.from_numpy(~used).cuda()
    for w in ("k", "v"):
        p.cache[w].permute(0, 2, 1, 3)[hide] = 255
        p.cache[w + "_params"].permute(0, 2, 1, 3, 4)[hide] = float("nan")
    got = [host_bits(x) for x in p.call(window=window, max_kv=kv)]
    assert all(np.array_equal(a, b) for a, b in zip(got, clean))
    # a token in the middle: rows whose window misses it, and rows before it, keep their bits
    tok = p.lens[0] - max(1, new // 2)
    pg = int(p.table_h[0, tok // 16])
    for w in ("k", "v"):
        p.cache[w + "_params"][pg, :, tok % 16, 1] = float("nan")
        p.cache[w + "_params"][pg, :, tok % 16, 0] = float("inf")
    out, lse = p.call(window=window, max_kv=kv)
    first = p.lens[0] - new
    for i in range(p.T):
        sees = i < new and tok <= first + i and tok > first + i - window
        if sees:
            assert bool(t.isnan(out[i]).all()) and bool(t.isnan(lse[i]).all())
        else:
            assert np.array_equal(host_bits(out[i]), clean[0][i]) and np.array_equal(host_bits(lse[i]), clean[1][i]), i
    # the value alone not finite, in one group: that group's dimensions only
    for w in ("k", "v"):
        p.cache[w + "_params"][pg, :, tok % 16] = 1.0
    p.cache["v_params"][pg, :, tok % 16, 1, 1] = float("nan")
    p.cache["v_params"][pg, :, tok % 16, 0, 1] = 0.0
    out, lse = p.call(window=window, max_kv=kv)
    i = tok - first
    assert bool(t.isnan(out[i, :, 32:]).all()) and not bool(t.isnan(out[i, :, :32]).any())
    assert not bool(t.isnan(lse[i]).any())


@pytest.mark.parametrize("bits,D,group", [(4, 64, 32), (8, 128, 32), (4, 256, 32), (4, 128, 64)])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
@KERNELS
def test_hidden_values_beyond_fp16(bits, D, group, ty, kv):
    """Finite parameters whose values pass fp16's range, in slots that no row sees, change no bit; great
    ones that rows see are within the bound."""
    t = torch()
    p = Problem([100, 77], [70, 60], bits=bits, D=D, group=group, page=16, ty=ty, seed=16)
    clean = [host_bits(x).copy() for x in p.call(max_kv=kv)]
    used = np.zeros((p.cache["k"].shape[0], 16), bool)
    for b, n in enumerate(p.lens):
        used[p.table_h[b, np.arange(n) // 16], np.arange(n) % 16] = True
    hide = t.from_numpy(~used).cuda()
    p.cache["v"].permute(0, 2, 1, 3)[hide] = 255
    p.cache["v_params"].permute(0, 2, 1, 3, 4)[hide] = 60000.0
    got = [host_bits(x) for x in p.call(max_kv=kv)]
    assert all(np.array_equal(a, b) for a, b in zip(got, clean))
    # offsets up to 2^15 and scales up to 2^15 / 2^bits: a value stays below 2^16 - 2^15 / 2^bits
    p.cache["v_params"][:, :, :, 0] = 2.0 ** (15 - bits)
    p.cache["v_params"][:, :, :, 1] = -(2.0 ** 15)
    p.cache["v_params"][:, :, ::2, 1] = 2.0 ** 14
    if ty == "bf16":  # (fp16 results would hold them too, but a sum's bound passes their range)
        check(p, "great values", max_kv=kv)
    t.cuda.synchronize()


def test_pages_outside_the_pool():
    """Tokens of such pages are not seen; a negative one, one past the pool, the greatest integer."""
    t = torch()
    for new in (1, 50):
        p = Problem([100, 60, 64], [new] * 3, page=16, seed=14)
        p.table_h[0, 2], p.table_h[0, 6], p.table_h[1, 0] = -1, p.cache["k"].shape[0], 2 ** 31 - 1
        p.table_h[2, :] = -5
        p.table.copy_(dev(p.table_h))
        check(p, "pages outside")
        check(p, "pages outside", causal=False)
        check(p, "pages outside", max_kv=MUCH)
    t.cuda.synchronize()


def test_lengths_outside_the_table():
    t = torch()
    p = Problem([64, 32], [1, 1], page=16, seed=15)
    want = [host_bits(x).copy() for x in p.call()]
    width = p.table_h.shape[1]
    p.lens = [64, -3]
    p.kv_len.copy_(dev(np.array([2 ** 31 - 1, -3], np.int32)))
    out, lse = p.call()
    assert width * 16 == 64
    assert np.array_equal(host_bits(out[0]), want[0][0]) and not bool(out[1].any())
    assert bool(t.isneginf(lse[1]).all())


@pytest.mark.parametrize("many", [False, True])
def test_rows_of_no_sequence(many):
    """Rows before the first sequence, behind the last and past max_q are left as they were; offsets outside [0, T]
    are clamped."""
    t = torch()
    for max_kv in (None, 50000, MUCH):
        # (many: 32 heads of one cache head, 192 rows and more)
        p = Problem([50, 90, 20], [4, 6, 2], heads=32 if many else 8, kv=1 if many else 2, seed=16, extra=5)
        cu = np.array([2, 6, 12, 14], np.int32)
        p.cu_h = cu
        p.cu.copy_(dev(cu))
        out = t.full((p.T, p.heads, p.D), 7.0, dtype=t.bfloat16, device="cuda")
        lse = t.full((p.T, p.heads), 7.0, device="cuda")
        check(p, "rows", out=out, lse=lse, max_kv=max_kv)
        assert bool((out[:2] == 7.0).all()) and bool((out[14:] == 7.0).all()) and bool((lse[14:] == 7.0).all())
        out.fill_(7.0)
        p.call(out=out, max_q=3, max_kv=max_kv)
        assert bool((out[5] == 7.0).all()) and bool((out[9:12] == 7.0).all()) and not bool((out[12:14] == 7.0).any())
        p.cu_h = np.array([-4, 6, 12, 1000], np.int32)
        p.cu.copy_(dev(p.cu_h))
        check(p, "clamped", max_kv=max_kv, max_q=p.T)


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@KERNELS
def test_strided_queries(ty, kv):
    """Queries as a slice of a fused projection, at any element offset, heads first, and shared rows."""
    t = torch()
    p = Problem([60, 45], [5, 30], ty=ty, seed=17)
    want = [host_bits(x).copy() for x in p.call(max_kv=kv)]
    wide = t.zeros(p.T, p.heads + 3, p.D + 1, dtype=tt(ty), device="cuda")
    base = p.Q
    for view in (wide[:, 1:p.heads + 1, 1:], wide[:, 3:, :p.D],
                 t.zeros(p.heads, p.T, p.D, dtype=tt(ty), device="cuda").transpose(0, 1)):
        view.copy_(base)
        p.Q = view
        got = [host_bits(x) for x in p.call(max_kv=kv)]
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
    p.Q = base[:1].expand(p.T, p.heads, p.D)
    check(p, "shared rows", max_kv=kv)


@KERNELS
def test_queries_not_finite(kv):
    t = torch()
    for new in (1, 40):
        p = Problem([60, 45], [new, new], seed=18)
        clean = host_bits(p.call(max_kv=kv)[0]).copy()
        p.Q[0, 1, 5], p.Q[0, 2, 0], p.Q[new, 3, 63] = float("nan"), float("inf"), -float("inf")
        out, lse = p.call(max_kv=kv)
        bad = [(0, 1), (0, 2), (new, 3)]
        for r, a in bad:
            assert bool(t.isnan(out[r, a]).all()) and bool(t.isnan(lse[r, a]))
        keep = np.ones((p.T, p.heads), bool)
        for r, a in bad:
            keep[r, a] = False
        assert np.array_equal(host_bits(out)[keep], clean[keep])


def test_queries_of_a_wide_range():
    """bf16 rows of 1e30 and of 1e-30 (scores scaled back), with elements 2^-20 of the largest: all are kept."""
    t = torch()
    for s, new in ((2.0 ** 90, 1), (2.0 ** -100, 1), (2.0 ** 90, 40)):
        p = Problem([60, 45], [new, new], seed=19)
        p.Q[:, :, ::2] *= 2.0 ** -20
        p.Q *= s
        check(p, "range", scale=0.1 / s, max_kv=MUCH)
    t.cuda.synchronize()


def test_repeats_streams_and_graph():
    """Store, then attention over what was stored, as a decode step: repeated calls give the same bits; on another
    stream; captured, with the tables, lengths and inputs changed between replays, two graphs in turn."""
    t = torch()
    p = Problem([500, 301, 64], [1, 1, 1], heads=8, kv=2, D=128, group=64, page=32, seed=20)
    new = t.randn(3, 2, 2, 128, device="cuda", dtype=t.bfloat16)
    slots = t.zeros(3, dtype=t.int32, device="cuda")
    out = t.empty(3, 8, 128, dtype=t.bfloat16, device="cuda")
    lse = t.empty(3, 8, device="cuda")
    ws = t.empty(Q.lib().qkv_attention_workspace_bytes(3, 8, 2, 128, 3, 1, 512, 0), dtype=t.uint8, device="cuda")
    assert ws.numel() > 0

    def place():
        n = p.kv_len.cpu().numpy() - 1
        tab = p.table.cpu().numpy()
        slots.copy_(dev(np.array([tab[b, n[b] // 32] * 32 + n[b] % 32 for b in range(3)], np.int32)))

    def step(o=out, e=lse):
        Q.qkv_cache_store(new[:, 0], new[:, 1], slots, p.cache)
        return Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, max_kv=512, out=o, lse=e, workspace=ws)

    place()
    ref = [host_bits(x).copy() for x in step()]
    for _ in range(3):
        assert all(np.array_equal(host_bits(a), b) for a, b in zip(step(), ref))
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(np.array_equal(host_bits(a), b) for a, b in zip(got, ref))
    o2, e2 = t.empty_like(out), t.empty_like(lse)
    g, g2 = t.cuda.CUDAGraph(), t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step()
    with t.cuda.graph(g2):                  # shares the workspace: replayed one after the other
        step(o2, e2)
    for k, lens in enumerate(([500, 301, 64], [499, 1, 65], [512, 480, 33], [2, 400, 96])):
        p.kv_len.copy_(dev(np.array(lens, np.int32)))
        new.copy_(t.randn(3, 2, 2, 128, device="cuda"))
        p.Q.copy_(t.randn(3, 8, 128, device="cuda"))
        # sequences 1 and 2 have fewer pages than the longest: their table is filled up with sequence 0's
        tab = p.table_h.copy()
        for b in (1, 2):
            tab[b, tab[b] < 0] = p.table_h[0][tab[b] < 0]
        tab = np.roll(tab, k, axis=1)
        p.table.copy_(dev(tab))
        place()
        g.replay()
        g2.replay()
        t.cuda.synchronize()
        got = [host_bits(x).copy() for x in (out, lse, o2, e2)]
        want = [host_bits(x) for x in step()]
        for a, b in zip(got, want + want):
            assert np.array_equal(a, b), k


@pytest.mark.parametrize("kv", [400, MUCH])
def test_prompt_chunk_in_a_graph(kv):
    """Storing a chunk of a prompt and attention over it, captured; offsets, lengths and inputs change between
    replays, with eager calls and other allocations between them."""
    t = torch()
    p = Problem([200, 150], [90, 60], heads=8, kv=2, D=128, group=64, page=32, seed=23)
    new = t.randn(2, 150, 2, 128, device="cuda", dtype=t.bfloat16)
    slots = t.zeros(150, dtype=t.int32, device="cuda")
    out, lse = t.empty(150, 8, 128, dtype=t.bfloat16, device="cuda"), t.empty(150, 8, device="cuda")

    def place(cu, lens):
        at = []
        for b in range(2):
            n = cu[b + 1] - cu[b]
            at += [p.table_h[b, i // 32] * 32 + i % 32 for i in range(lens[b] - n, lens[b])]
        slots.copy_(dev(np.array(at, np.int32)))

    def step(o=out, e=lse):
        Q.qkv_cache_store(new[0], new[1], slots, p.cache)
        return Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, cu_q=p.cu, max_q=100, max_kv=kv, out=o, lse=e)

    place(p.cu_h, p.lens)
    ref = [host_bits(x).copy() for x in step()]
    assert all(np.array_equal(host_bits(a), b) for a, b in zip(step(), ref))
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step()
    for k, (cu, lens) in enumerate((([0, 90, 150], [200, 150]), ([0, 60, 150], [60, 160]), ([0, 100, 150], [101, 50]),
                                    ([0, 90, 150], [200, 150]))):
        p.cu.copy_(dev(np.array(cu, np.int32)))
        p.kv_len.copy_(dev(np.array(lens, np.int32)))
        place(cu, lens)
        new.copy_(t.randn(2, 150, 2, 128, device="cuda"))
        g.replay()
        t.cuda.synchronize()
        got = [host_bits(x).copy() for x in (out, lse)]
        p.cu_h, p.lens, p.news = np.array(cu), lens, [cu[1], cu[2] - cu[1]]
        for a, b in zip(got, check(p, "graph", max_q=100, max_kv=kv)):
            assert np.array_equal(a, host_bits(b)), k


def test_batch_gives_the_rows_of_single_calls():
    """Sequences of one batch do not influence each other (the same split of the tokens)."""
    p = Problem([200, 33, 1, 90], [3, 1, 1, 2], seed=21)
    t = torch()
    kv = 100                                  # one part in the batch and alone
    out, lse = p.call(max_kv=kv)
    for b in range(4):
        r = slice(int(p.cu_h[b]), int(p.cu_h[b + 1]))
        o, e = Q.qkv_attention(p.Q[r], p.cache, p.table[b:b + 1], p.kv_len[b:b + 1], cu_q=dev(np.array(
            [0, p.news[b]], np.int32)), max_q=3, max_kv=kv, need_lse=True)
        assert np.array_equal(host_bits(o), host_bits(out[r])) and np.array_equal(host_bits(e), host_bits(lse[r]))
    t.cuda.synchronize()


def test_nothing_to_do():
    t = torch()
    cache = Q.qkv_cache_new(1, 2, 64, page=16)
    i32 = dict(dtype=t.int32, device="cuda")
    out = Q.qkv_attention(t.empty(0, 4, 64, dtype=t.float16, device="cuda"), cache, t.zeros(0, 3, **i32),
                          t.zeros(0, **i32))
    assert out.shape == (0, 4, 64)
    q = t.ones(2, 4, 64, dtype=t.float16, device="cuda")
    out, lse = Q.qkv_attention(q, cache, t.zeros(2, 0, **i32), t.full((2,), 5, **i32), need_lse=True)  # no pages
    assert not bool(out.any()) and bool(t.isneginf(lse).all())


def test_refusals():
    t = torch()
    p = Problem([20, 20], [1, 1], seed=22)
    with pytest.raises(TypeError):
        Q.qkv_attention(p.Q.float(), p.cache, p.table, p.kv_len)
    with pytest.raises(ValueError):
        Q.qkv_attention(p.Q[:1], p.cache, p.table, p.kv_len)
    with pytest.raises(ValueError):
        Q.qkv_attention(p.Q[:, :7], p.cache, p.table, p.kv_len)
    with pytest.raises(ValueError):
        Q.qkv_attention(p.Q[..., :32], p.cache, p.table, p.kv_len)
    with pytest.raises(ValueError):
        Q.qkv_attention(p.Q.transpose(1, 2).contiguous().transpose(1, 2), p.cache, p.table, p.kv_len)
    with pytest.raises(TypeError):
        Q.qkv_attention(p.Q, p.cache, p.table.long(), p.kv_len)
    with pytest.raises(ValueError):
        Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len[:1])
    with pytest.raises(ValueError):
        Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, cu_q=p.cu[:2])
    with pytest.raises(TypeError):
        Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, sinks=t.zeros(8, device="cuda", dtype=t.float16))
    with pytest.raises(TypeError):
        Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, out=t.empty(2, 8, 64, device="cuda"))
    with pytest.raises(Q.QmmError):
        Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, causal=False, window=4)
    with pytest.raises(Q.QmmError):
        Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, scale=float("nan"))
    with pytest.raises(Q.QmmError):
        Q.qkv_attention(p.Q, p.cache, p.table, p.kv_len, max_kv=100000, workspace=t.empty(
            64, dtype=t.uint8, device="cuda"))
    t.cuda.synchronize()
