"""CPU pins of the key/value cache's oracle: hand-computed groups, the order of the codes, and attention
against the definition written out."""
import math

import numpy as np
import pytest

from oracle import kv_oracle as KO


def empty(pages, heads, page, D, bits, group):
    c = dict(bits=bits, group=group)
    for w in ("k", "v"):
        c[w] = np.zeros((pages, heads, page, D * bits // 8), np.uint8)
        c[w + "_params"] = np.zeros((pages, heads, page, 2, D // group), np.float16)
    return c


def test_quantize_group_by_hand():
    # 0 .. 15 in steps of one: every code is its value
    codes, s, o = KO.quantize_group(list(range(16)) * 2, 4)
    assert s == 1.0 and o == 0.0 and codes == list(range(16)) * 2
    # halves go to the even code: range 0 .. 15, values k + 0.5
    codes, s, o = KO.quantize_group([0.0, 15.0, 0.5, 1.5, 2.5, 13.5] + [0.0] * 26, 4)
    assert s == 1.0 and codes[:6] == [0, 15, 0, 2, 2, 14]
    # one value: scale 0, the offset holds it
    codes, s, o = KO.quantize_group([-2.5] * 32, 8)
    assert s == 0.0 and o == -2.5 and not any(codes)
    # 8 bits, offset below zero
    codes, s, o = KO.quantize_group([-1.0, 254.0, 0.0] + [3.0] * 29, 8)
    assert s == 1.0 and o == -1.0 and codes[:4] == [0, 255, 1, 4]
    # not finite
    for bad in (math.nan, math.inf, -math.inf):
        codes, s, o = KO.quantize_group([1.0, bad] + [2.0] * 30, 4)
        assert s == 0.0 and math.isnan(o) and not any(codes)
    # beyond the limit
    codes, s, o = KO.quantize_group([1e30, -1e30] + [0.0] * 30, 4)
    assert o == -KO.LIMIT and codes[0] == 15 and codes[1] == 0
    assert abs(15 * float(s) + float(o)) < 65504


@pytest.mark.parametrize("D", [64, 128, 256])
def test_positions(D):
    for which, W in (("k", 4), ("v", 16)):
        pos = KO.position(D, which)
        assert sorted(pos) == list(range(D))
        assert pos[1] == D // W and pos[W] == 1


@pytest.mark.parametrize("bits,D,group", [(4, 64, 32), (8, 128, 128), (4, 256, 64)])
def test_store_and_load(bits, D, group):
    rng = np.random.default_rng(bits + D)
    K, V = rng.standard_normal((2, 5, 3, D))
    c = empty(2, 3, 16, D, bits, group)
    KO.store(K, V, [3, -1, 31, 32, 3], c)      # slot 3 twice: the last; -1 and 32 are not stored
    k, v = KO.load(c, [3, 31, 32, -1, 0])
    step = (np.abs(K).max() * 2) / (2 ** bits - 1)
    assert np.abs(k[0] - K[4]).max() <= 0.51 * step and np.abs(v[1] - V[2]).max() <= 0.51 * step * 1.5
    assert not k[2:].any() and not v[2:].any()


def test_attention_definition():
    rng = np.random.default_rng(3)
    D, H, A = 64, 2, 4
    c = empty(4, H, 16, D, 8, 64)
    K, V = rng.standard_normal((2, 64, H, D))
    KO.store(K, V, list(range(64)), c)
    table = np.array([[2, 0, 99], [1, 3, 0]])
    Q = rng.standard_normal((5, A, D))
    out, lse, mag = KO.attention(Q, c, table, [40, 2], cu_q=[0, 2, 5], window=20)
    kk, vv = KO.load(c, list(range(64)))
    # second query of sequence 0: position 39 sees 20 .. 39, of which 32 .. 39 lie on a page that is not there
    toks = [0 * 16 + i - 16 for i in range(20, 32)]
    s = np.array([Q[1, 3] @ kk[t, 1] for t in toks]) / 8.0
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[1, 3], sum(wi * vv[t, 1] for wi, t in zip(w, toks)), atol=1e-12)
    assert np.isclose(lse[1, 3], np.log(np.exp(s).sum())) and mag["seen"][1] == 12
    # three queries, two tokens: the first sees nothing, the second one token
    assert not out[2].any() and np.isneginf(lse[2]).all()
    assert np.allclose(out[3, 0], vv[16, 0])
    out, lse, _ = KO.attention(Q, c, table, [40, 2], cu_q=[0, 2, 5], sinks=np.arange(4.0))
    assert np.allclose(lse[2], np.arange(4.0)) and not out[2].any()
    s0 = Q[3, 1] @ kk[16, 0] / 8.0
    assert np.allclose(out[3, 1], vv[16, 0] * np.exp(s0) / (np.exp(s0) + np.e))
