"""GPU parity of attention over the low-bit cache at its edges: scales of either sign, hidden tokens next to great
values, queries of a wide range, rows that are NaN, the widest windows; against the fp64 oracle.

Bounds as in test_gpu_kv_attention.py: with u = 2^-24 a score is off by dS <= gamma(D + 16) qk + 8 u qk + 100 u, a
weight by 2 dS, the sums by gamma(seen + 64).  Roundings to fp16, half a step each, 2^-11: none for fp16 results (two
fp16 values hold a weight, 2^-22), one for bf16 ones (e^S s), two where many rows meet groups of 32 (e^S and c s + o,
with their product 2^-10 + 2^-22); for terms below 2^-20 of the largest weight times the largest scale 2^-30 of that,
times the largest code."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q
from oracle import kv_oracle as KO

from gpu_util import U32, assert_elementwise, gamma, host_bits, host_f64, say, torch
from test_gpu_kv_attention import MUCH, Problem

pytestmark = pytest.mark.gpu

# queries per sequence, tokens expected, whether the call takes the kernel for many rows
CALLS = pytest.mark.parametrize("new,kv,many", [(1, None, False), (70, None, False), (70, MUCH, True)],
                                ids=["one", "few", "many"])


def check(p, many, label="", **kw):
    """One call against the oracle; returns (out, lse).  many: it takes the kernel for many rows."""
    group = p.cache["group"]
    say(f"  {label} lens={p.lens} news={p.news} heads={p.heads}/{p.kv} D={p.D} bits={p.bits} group={group} {p.ty} "
        f"many={many} {sorted(kw)}")
    out, lse = p.call(**kw)
    ref, rl, mag = KO.attention(host_f64(p.Q), p.host_cache(), p.table_h, p.lens, cu_q=p.cu_h,
                                scale=kw.get("scale"), window=kw.get("window", 0),
                                sinks=None if kw.get("sinks") is None else host_f64(kw["sinks"]))
    own = mag["seen"] >= 0
    n = np.maximum(mag["seen"], 0)[:, None]
    dS = gamma(p.D + 16) * mag["qk"] + U32 * (8 * mag["qk"] + 100)
    step = float(p.cache["v_params"][:, :, :, 0].float().abs().nan_to_num().max())
    weights = 2.0 ** -22 if p.ty == "f16" else 2.0 ** -10 + 2.0 ** -22 if many and group == 32 else 2.0 ** -11
    bound = mag["pv"] * (weights + 2 * dS + gamma(n + 64.0))[..., None] + (n * 2.0 ** (p.bits - 30) * step)[..., None]
    assert_elementwise(host_f64(out)[own], ref[own], bound[own], p.ty, label + " out")
    seen = np.isfinite(rl) & own[:, None]
    got = host_f64(lse)
    assert np.array_equal(np.isneginf(got[own]), np.isneginf(rl[own]))
    lim = 2 * dS + gamma(n + 64.0) + 2.0 ** -22 * (np.abs(np.where(np.isfinite(rl), rl, 0.0)) + 40)
    worst = np.abs(got[seen] - rl[seen]) / np.broadcast_to(lim, got.shape)[seen]
    assert worst.size == 0 or worst.max() <= 1.0, (label, "lse", worst.max())
    return out, lse


@pytest.mark.parametrize("bits,D,group", [(4, 64, 32), (8, 64, 64), (4, 128, 32), (4, 128, 64), (8, 128, 128),
                                          (4, 256, 64), (8, 256, 32)])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
@CALLS
def test_scales_of_either_sign(bits, D, group, ty, new, kv, many):
    """A code stands for c s + o whatever the sign of s: small negative scales (and -0.0) beside large positive ones
    and the reverse, in one token and in one tile."""
    t = torch()
    p = Problem([100, 77], [new, new], D=D, bits=bits, group=group, ty=ty, seed=D + bits + new)
    rng = np.random.default_rng(D + group)
    shape = p.cache["v_params"][:, :, :, 0].shape
    for choice in ([1.0, -0.001], [-1.0, 0.001], [1.0, -0.0], [-1.0, 0.001, -0.001, 1.0, -0.0, 0.0]):
        p.cache["v_params"][:, :, :, 0] = t.from_numpy(rng.choice(choice, shape)).half().cuda()
        p.cache["k_params"][:, :, :, 0] *= t.from_numpy(rng.choice([1.0, -1.0], shape)).half().cuda()
        check(p, many, f"scales {choice}", max_kv=kv)


@pytest.mark.parametrize("bits,D", [(4, 64), (4, 128), (8, 128), (4, 256)])
@CALLS
def test_hidden_tokens_next_to_great_values(bits, D, new, kv, many):
    """Tokens that read as up to 57344 or 65024 and whose parameters allow for more than fp16 holds: NaN in a token
    of their tile that a row does not see, behind the sequence or after the query, changes no bit of it."""
    t = torch()
    p = Problem([100, 77], [new, new], bits=bits, D=D, group=32, page=16, seed=D + bits)
    # 4 bits: codes up to 14, 14 * 8192 - 57344; 8 bits: up to 239, 239 * 512 - 57344
    p.cache["v"].bitwise_and_(0xee if bits == 4 else 0xef)
    p.cache["v_params"][:, :, ::3, 0] = 8192.0 if bits == 4 else 512.0
    p.cache["v_params"][:, :, ::3, 1] = -57344.0
    clean = [host_bits(x).copy() for x in check(p, many, "great values", max_kv=kv)]
    assert bool(t.isfinite(p.call(max_kv=kv)[0]).all())
    for b, n in enumerate(p.lens):                      # places behind the sequences' ends
        page = int(p.table_h[b, n // 16])
        p.cache["v_params"][page, :, n % 16:] = float("nan")
    got = [host_bits(x) for x in p.call(max_kv=kv)]
    assert all(np.array_equal(a, b) for a, b in zip(got, clean))
    tok = p.lens[0] - 1                                 # the last query's own token
    p.cache["v_params"][int(p.table_h[0, tok // 16]), :, tok % 16, :, -1] = float("nan")
    out, lse = p.call(max_kv=kv)
    assert bool(t.isnan(out[new - 1, :, -32:]).all()) and bool(t.isfinite(out[new - 1, :, :-32]).all())
    keep = np.arange(p.T) != new - 1
    assert np.array_equal(host_bits(out)[keep], clean[0][keep])
    assert np.array_equal(host_bits(lse)[keep], clean[1][keep]) and bool(t.isfinite(lse).all())


@pytest.mark.parametrize("bits,D,group", [(4, 64, 32), (4, 128, 64), (4, 256, 128), (8, 64, 32), (8, 128, 64)])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
@CALLS
def test_small_elements_of_queries(bits, D, group, ty, new, kv, many):
    """Elements that are multiples of 2^-30 of the row's largest enter exactly: the bound has no term for them.  The
    largest ones meet keys that are zero, a group of scale and offset 0, so that the small ones make the scores."""
    t = torch()
    p = Problem([100, 77], [new, new], D=D, bits=bits, group=group, ty=ty, seed=D + bits)
    p.cache["k_params"][..., 0] = 0.0
    rng = np.random.default_rng(D)
    unit = 2.0 ** -24 if ty == "f16" else 2.0 ** -30
    x = rng.integers(-16, 17, (p.T, p.heads, D)) * unit
    x[..., :group] = rng.standard_normal((p.T, p.heads, group)) * 0.1 * unit * 2.0 ** 30
    x[..., 5] = unit * 2.0 ** 30
    x[..., :group] = x[..., :group].clip(-unit * 2.0 ** 30, unit * 2.0 ** 30)
    p.Q.copy_(t.from_numpy(x))
    check(p, many, "small elements", scale=0.02 / unit, max_kv=kv)


@pytest.mark.parametrize("ty", ["f16", "bf16"])
@CALLS
@pytest.mark.parametrize("parts", [False, True])
def test_rows_that_are_nan_with_sinks(ty, new, kv, many, parts):
    """A query, a key or a sink that is not a number: result and lse of the rows that meet it are NaN, with sinks as
    without; the other rows keep their bits."""
    t = torch()
    p = Problem([60, 45], [min(new, 60), min(new, 45)], ty=ty, seed=new)
    if parts:
        kv = MUCH if many else 100000
    n0 = p.news[0]
    sinks = t.linspace(-3, 3, p.heads, device="cuda")
    sinks[6] = -float("inf")
    args = dict(sinks=sinks, max_kv=kv)
    clean = [host_bits(x).copy() for x in check(p, many, "sinks", **args)]

    def rest(out, lse, bad):
        assert bool(t.isnan(out[bad]).all()) and bool(t.isnan(lse[bad]).all())
        keep = ~bad.cpu().numpy()
        assert np.array_equal(host_bits(out)[keep], clean[0][keep])
        assert np.array_equal(host_bits(lse)[keep], clean[1][keep])

    bad = t.zeros(p.T, p.heads, dtype=t.bool, device="cuda")
    q = p.Q.clone()
    for r, a, x in ((0, 1, float("nan")), (0, 6, float("nan")), (n0, 3, float("inf"))):
        p.Q[r, a, 7] = x
        bad[r, a] = True
    rest(*p.call(**args), bad)
    p.Q.copy_(q)
    sinks[2] = float("nan")                 # (every row sees a token: see Problem's lens and news)
    bad = t.zeros_like(bad)
    bad[:, 2] = True
    rest(*p.call(**args), bad)
    sinks[2] = 0.0
    clean = [host_bits(x).copy() for x in p.call(**args)]
    p.cache["k_params"][int(p.table_h[1, 0]), 1, 0, 1] = float("nan")  # sequence 1, token 0, heads 4 to 7
    bad = t.zeros_like(bad)
    bad[n0:, 4:] = True
    rest(*p.call(**args), bad)


def test_sinks_and_rows_that_see_nothing():
    """out = 0 and lse = the sink, whatever it is."""
    t = torch()
    p = Problem([0, 2], [1, 2], seed=3)
    sinks = t.tensor([0.0, -float("inf"), float("inf"), float("nan"), -5.0, 200.0, 1e-30, -300.0], device="cuda")
    for kv in (None, 100000):
        out, lse = p.call(sinks=sinks, max_kv=kv)
        assert not bool(out[0].any())
        assert bool(((lse[0] == sinks) | (t.isnan(lse[0]) & t.isnan(sinks))).all())
        assert not bool(out[1:, 2].any()) and bool((lse[:, 2] == float("inf")).all())
        assert bool(t.isnan(out[1:, 3]).all()) and bool(t.isnan(lse[:, 3]).all())


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 1])
@pytest.mark.parametrize("news", [[49, 2, 5], [140, 70, 3]])
@pytest.mark.parametrize("kv", [None, MUCH])
def test_widest_windows(window, news, kv):
    """A window that covers every sequence is none, up to the largest integer, also where queries stand before
    their sequence's first token."""
    p = Problem([40, 50, 0], news, seed=4)
    many = kv == MUCH and max(news) * 4 > 64
    want = [host_bits(x).copy() for x in check(p, many, "no window", max_kv=kv)]
    got = [host_bits(x) for x in check(p, many, "window", window=window, max_kv=kv)]
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
