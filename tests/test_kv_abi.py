"""CPU tests of the key/value cache's entry points: host-only refusals and workspace sizes."""
import ctypes
import math

import pytest

from gemm_qmm_nbits_amd import qmm as Q

FAKE = 0x1000


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_params=FAKE, v_params=FAKE, pages=100, heads=8, page=16, D=128, bits=4, group=64)
    a.update(kw)
    return ctypes.byref(Q.qkv_cache(*a.values()))


def store(cache_kw=None, **kw):
    a = dict(K=FAKE, krs=1024, khs=128, V=FAKE, vrs=1024, vhs=128, type=Q.QMM_BF16, T=7, slots=FAKE)
    a.update(kw)
    return Q.lib().qmm_validate_kv_store(*a.values(), kw["c"] if "c" in kw else cache(**(cache_kw or {})))


def load(cache_kw=None, **kw):
    a = dict(slots=FAKE, T=7, K=FAKE, V=FAKE, type=Q.QMM_F32)
    a.update(kw)
    return Q.lib().qmm_validate_kv_load(cache(**(cache_kw or {})), *a.values())


def attn(cache_kw=None, **kw):
    a = dict(Q=FAKE, rs=4096, hs=128, type=Q.QMM_BF16, T=5, q_heads=32, B=5, cu_q=None, kv_len=FAKE, table=FAKE,
             width=64, max_q=1, max_kv=1, scale=0.1, causal=1, window=0, sinks=None)
    tail = dict(out=FAKE, lse=None, ws=None, wsb=0)
    for k, v in kw.items():
        (a if k in a else tail)[k] = v
    return Q.lib().qmm_validate_kv_attention(*a.values(), cache(**(cache_kw or {})), *tail.values())


@pytest.mark.parametrize("f", [store, load, attn])
def test_cache_refusals(f):
    assert f() == 0
    for b in (2, 3, 0, 16):
        assert f(dict(bits=b)) == -3
    for d in (0, 32, 96, 512, -128):
        assert f(dict(D=d)) == -5
    for g in (0, 16, 48, 256, -64):
        assert f(dict(group=g)) == -4
    assert f(dict(D=64, group=128)) == -4
    for p in (0, 8, 24, 131072, -16):
        assert f(dict(page=p)) == -5
    assert f(dict(heads=0)) == -5 and f(dict(heads=4097)) == -5
    assert f(dict(pages=0)) == -5 and f(dict(pages=1 << 27)) == -5 and f(dict(pages=(1 << 62))) == -5
    assert f(dict(pages=(1 << 27) - 1)) == 0
    for name in ("k", "v", "k_params", "v_params"):
        assert f({name: None}) == -1 and f({name: FAKE + 8}) == -6


@pytest.mark.parametrize("f", [store, load])
def test_token_refusals(f):
    assert f(T=-1) == -5 and f(T=(1 << 24) + 1) == -5
    assert f(dict(heads=64), T=(1 << 20) + 1) == -5     # more rows than one launch has
    assert f(type=3) == -2 and f(type=-1) == -2
    assert f(slots=None) == -1 and f(slots=FAKE + 2) == -6
    assert f(T=0, slots=None, K=None, V=None) == 0


def test_store_refusals():
    assert store(T=1 << 20) == 0 and store(T=(1 << 20) + 1) == -5 and load(T=(1 << 20) + 1) == 0
    assert store(K=None) == -1 and store(V=None) == -1
    assert store(K=FAKE + 1) == -6 and store(K=FAKE + 2) == 0 and store(V=FAKE + 2, type=Q.QMM_F32) == -6
    for k in ("krs", "khs", "vrs", "vhs"):
        assert store(**{k: -1}) == -5 and store(**{k: 0}) == 0 and store(**{k: (1 << 40) + 1}) == -5
    a = (FAKE, 1024, 128, FAKE, 1024, 128, Q.QMM_F16, 7, FAKE, None)
    assert Q.lib().qmm_validate_kv_store(*a) == -1      # no descriptor


def test_load_refusals():
    assert load(K=None) == 0 and load(V=None) == 0 and load(K=None, V=None, slots=None) == 0
    assert load(K=FAKE + 2) == -6 and load(V=FAKE + 2, type=Q.QMM_F16) == 0


def test_attention_refusals():
    assert attn(type=Q.QMM_F32) == -2 and attn(type=5) == -2
    assert attn(T=-1, B=-1) == -5 and attn(T=(1 << 24) + 1, cu_q=FAKE) == -5 and attn(B=65536, cu_q=FAKE) == -5
    assert attn(q_heads=33) == -5 and attn(q_heads=4) == -5 and attn(q_heads=0) == -5 and attn(q_heads=4104) == -5
    assert attn(dict(heads=1), q_heads=513) == -5
    assert attn(rs=-1) == -5 and attn(hs=-1) == -5
    assert attn(width=-1) == -5 and attn(width=(1 << 26) + 1) == -5
    assert attn(max_q=0, cu_q=FAKE) == -5 and attn(max_kv=-1) == -5 and attn(max_kv=1 << 31) == -5
    assert attn(T=6) == -5 and attn(max_q=2) == -5      # without cu_q: one query per sequence
    assert attn(T=6, max_q=2, cu_q=FAKE) == 0
    assert attn(causal=2) == -8 and attn(causal=0) == 0 and attn(window=-1) == -8
    assert attn(causal=0, window=5) == -8 and attn(window=5) == 0
    for s in (math.nan, math.inf, -math.inf):
        assert attn(scale=s) == -10
    assert attn(scale=-1.0) == 0 and attn(scale=0.0) == 0
    for k in ("Q", "kv_len", "table", "out"):
        assert attn(**{k: None}) == -1
    assert attn(width=0, table=None) == 0
    assert attn(Q=FAKE + 1) == -6 and attn(Q=FAKE + 2) == 0 and attn(out=FAKE + 4) == -6
    assert attn(cu_q=FAKE + 2) == -6 and attn(kv_len=FAKE + 2) == -6 and attn(table=FAKE + 2) == -6
    assert attn(sinks=FAKE + 2) == -6 and attn(lse=FAKE + 2) == -6
    assert attn(T=0, B=0, Q=None, kv_len=None, table=None, out=None) == 0
    # more work-groups than one launch has: 65535 sequences of 2^20 queries
    assert attn(T=1 << 20, B=65535, cu_q=FAKE, max_q=1 << 20) == -5


def test_attention_workspace():
    need = Q.lib().qkv_attention_workspace_bytes(5, 32, 8, 128, 5, 1, 30000, 0)
    assert need > 0
    assert attn(max_kv=30000) == -7 and attn(max_kv=30000, ws=FAKE, wsb=need - 1) == -7
    assert attn(max_kv=30000, ws=FAKE, wsb=need) == 0
    assert attn(max_kv=30000, ws=FAKE + 128, wsb=need) == -6
    # max_kv 0 takes the table's width
    assert attn(max_kv=0, width=1875) == -7 and attn(max_kv=0, width=1875, ws=FAKE, wsb=need) == 0
    # the sums and their two numbers of every row, for some number of parts
    rows = 5 * 32
    assert any(need == -(-s * rows * 128 * 4 // 256) * 256 + s * rows * 8 for s in range(2, 200))
    # one part: nothing to join
    assert Q.lib().qkv_attention_workspace_bytes(5, 32, 8, 128, 5, 1, 100, 0) == 0
    assert Q.lib().qkv_attention_workspace_bytes(0, 32, 8, 128, 0, 1, 30000, 0) == 0
    assert Q.lib().qkv_attention_workspace_bytes(5, 33, 8, 128, 5, 1, 30000, 0) == 0


def test_a_window_needs_no_more_parts_than_its_tokens():
    q = Q.lib().qkv_attention_workspace_bytes
    assert q(5, 32, 8, 128, 5, 1, 30000, 128) == 0
    assert q(5, 32, 8, 128, 5, 1, 30000, 29000) <= q(5, 32, 8, 128, 5, 1, 30000, 0)
    assert q(5, 32, 8, 128, 5, 1, 30000, 1 << 40) == q(5, 32, 8, 128, 5, 1, 30000, 0)
    assert q(5, 32, 8, 128, 5, 1, 30000, -1) == 0
    assert attn(max_kv=30000, window=128) == 0 and attn(max_kv=30000, window=29000) == -7
