"""GPU parity of attention over the low-bit cache in each form of its launch, which the size of the workspace tells:
whole work-groups write their results, parts are joined, and a call of many rows may hold both."""
import numpy as np
import pytest

from gemm_qmm_nbits_amd import qmm as Q

from gpu_util import host_bits, torch
from test_gpu_kv_attention import FORMATS, MUCH, Problem
from test_gpu_kv_edges import check

pytestmark = pytest.mark.gpu

# cache heads that make one whole round of work-groups, with four sequences of two row tiles of 128 rows each
ROUND = {64: 96, 128: 64, 256: 32}


def part_rows(p, max_kv, kv=None):
    """Rows of the parts that a call joins (0: none): each takes D sums and two numbers of 4 bytes, all sums rounded
    up to 256."""
    kv = p.kv if kv is None else kv
    need = Q.lib().qkv_attention_workspace_bytes(p.T, p.heads // p.kv * kv, kv, p.D, len(p.lens), max(p.news), max_kv, 0)
    return need // (4 * p.D + 8)


def problem(bits, D, group, ty, more):
    """Two heads per cache head, 130 rows of the longest sequence's queries."""
    kv = ROUND[D] + more
    return Problem([40, 100, 5, 70], [2, 65, 1, 9], heads=2 * kv, kv=kv, D=D, bits=bits, group=group, ty=ty,
                   seed=D + bits + group)


@pytest.mark.parametrize("bits,D,group", [(4, 64, 32), (8, 64, 64), (4, 128, 64), (8, 128, 32), (4, 256, 128),
                                          (8, 256, 32)])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_many_rows_whole(bits, D, group, ty):
    """One round of work-groups, none split."""
    p = problem(bits, D, group, ty, 0)
    assert part_rows(p, MUCH) == 0
    left = part_rows(p, MUCH, p.kv + 1)     # (one head more does not fit: parts of row tiles of 128 rows)
    assert left > 0 and left % 128 == 0
    check(p, True, "whole", max_kv=MUCH)


@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
def test_many_rows_whole_and_in_parts(bits, D, group, ty):
    """More than one round of work-groups: whole ones, and those left over in parts."""
    p = problem(bits, D, group, ty, 2)
    groups = 2 * p.kv * 4
    parts = part_rows(p, MUCH)
    # fewer parts than all groups would have in two each, and more than one of a group
    assert parts % 128 == 0 and 0 < parts // 128 < 2 * groups
    check(p, True, "whole and in parts", max_kv=MUCH)


def test_forms_agree():
    """The heads that both launches have get the same results but for the order of the sums: within the bounds of
    each; where neither splits them, the same bits."""
    t = torch()
    a = problem(4, 128, 64, "bf16", 2)
    out, lse = check(a, True, "whole and in parts", max_kv=MUCH)
    n = ROUND[128]
    cache = {k: v[:, :n].contiguous() if t.is_tensor(v) else v for k, v in a.cache.items()}
    o, e = Q.qkv_attention(a.Q[:, :2 * n], cache, a.table, a.kv_len, cu_q=a.cu, max_q=65, max_kv=MUCH, need_lse=True)
    # rows of the second row tile (the last queries of sequence 1) come first in the launch: whole in both
    last = int(a.cu_h[2]) - 1
    assert np.array_equal(host_bits(out[last, :2 * n]), host_bits(o[last]))
    assert np.array_equal(host_bits(lse[last, :2 * n]), host_bits(e[last]))


@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 7])
def test_few_rows_whole_and_in_parts(bits, D, group, ty, new):
    """Up to 16 rows of a cache head and more, in one part (no workspace) and in several: bf16 results to one
    rounding of a weight, 2^-11, whatever the groups."""
    p = Problem([90, 400, 7], [new] * 3, D=D, bits=bits, group=group, ty=ty, seed=D + group + new)
    assert part_rows(p, 256) == 0
    check(p, False, "in one part", max_kv=256)
    assert part_rows(p, MUCH) > 0
    check(p, False, "in parts", max_kv=MUCH)


@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("std", [0.1, 1.0, 4.0])
def test_many_rows_to_one_rounding(bits, D, group, std):
    """bf16 results of many rows, flat softmax to peaked: one rounding of a weight where groups are of 64 or 128, two
    with groups of 32 (and one again where few rows are asked for)."""
    p = Problem([200, 61], [90, 40], heads=4, kv=1, D=D, bits=bits, group=group, seed=D + bits, q_std=std)
    check(p, True, "many", max_kv=MUCH)
    check(p, False, "few", max_kv=256)
