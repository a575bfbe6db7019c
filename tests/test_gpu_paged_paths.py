"""tree_verify_attn_paged on paths that ordinary shapes do not take: trees of
more than 2048 nodes in bf16, faults and values that are not finite where rows
are copied one by one (page sizes off 8) and in trees of several key tiles."""

import numpy as np
import pytest
import torch

from oracle import paged as op
from paged_util import AttnCase, check_attn
from test_gpu_paged_attn import _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_verify_b200 import build
    build.build()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [2048, 2049, 2500])
def test_trees_of_thousands_of_nodes(T, dtype):
    _check(AttnCase(1, T, 2, 1, 64, 16, [70], dtype, tree="random", seed=T))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [1, 5, 12])
@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1, "past the pool"])
def test_bad_pages_where_rows_are_copied_one_by_one(entry, P, d):
    """The sequence's rows are NaN, its neighbours' are right."""
    T = 6
    c = AttnCase(4, T, 8, 2, d, P, [40, 170, 33, 300], "bf16")
    N = c.k.shape[0]
    c.table[1, 31 // P] = N if entry == "past the pool" else entry
    c.table[3, 299 // P] = N if entry == "past the pool" else entry
    ref = c_oracle(c)
    out, lse, st = _run(c)
    assert st == op.ST_BAD_PAGE
    assert ref["valid"].all(1).tolist() == [True, False, True, False]
    check_attn(out, lse, ref, poison=7.0)


def c_oracle(c):
    """AttnCase.oracle with the bad sequences' lengths taken as 0 for the bound's largest products."""
    lens, table = c.lens, c.table.copy()
    N = c.k.shape[0]
    fine = [all(0 <= table[b, i] < N for i in range(-(-n // c.P))) for b, n in enumerate(lens)]
    c.lens = [n if ok else 0 for n, ok in zip(lens, fine)]
    ref = c.oracle()
    c.lens = lens
    for b, ok in enumerate(fine):
        if not ok:
            ref["valid"][b] = False
    return ref


def _paths(c):
    """[B][T][T]: node j is on node i's root path."""
    B, T = c.parent.shape
    on = np.zeros((B, T, T), bool)
    for b in range(B):
        for i in range(T):
            j = i
            while j >= 0:
                on[b, i, j] = True
                j = int(c.parent[b, j])
    return on


def _spoil(c, ref, nodes, what):
    """Puts `what` into one column of V at the nodes (b, j, kv head); returns which outputs see one."""
    B, T, Hq, d = c.q.shape
    G = Hq // c.kt.shape[2]
    on, hit = _paths(c), np.zeros((B, T, Hq, d), bool)
    for k, (b, j, h) in enumerate(nodes):
        col = (7 + 19 * k) % d
        c.vt[b, j, h, col] = what
        hit[b, on[b, :, j], h * G:(h + 1) * G, col] = True
    return hit & ref["written"][..., None, None]


@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("P,d", [(1, 64), (5, 64), (5, 128), (12, 128)])
def test_values_that_are_not_finite_where_rows_are_copied_one_by_one(P, d, what):
    c = AttnCase(2, 9, 8, 2, d, P, [40, 140], "bf16", tree="random", n_nodes=[6, 9])
    ref = c.oracle()
    c.kt[0, 6:] = c.vt[0, 6:] = what                        # nodes that are not there
    hit = _spoil(c, ref, [(0, 3, 0), (1, 0, 1), (1, 8, 0)], what)
    _not_finite(c, ref, hit, what)


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,L,P,Hq,tree", [(300, 100, 16, 4, "chain"), (300, 5, 5, 4, "random"), (200, 700, 64, 8, "random"),
                                           (600, 3000, 16, 2, "chain")])
def test_values_that_are_not_finite_in_trees_of_several_tiles(T, L, P, Hq, tree, dtype, what):
    c = AttnCase(1, T, Hq, 1, 64, P, [L], dtype, tree=tree, n_nodes=[T - 3], seed=T)
    ref = c.oracle()
    c.kt[0, T - 3:] = c.vt[0, T - 3:] = what
    hit = _spoil(c, ref, [(0, j, 0) for j in (60, 127, 128, 131, T - 60, T - 4)], what)
    _not_finite(c, ref, hit, what)


def _not_finite(c, ref, hit, what):
    out, _, st = _run(c)
    assert st == 0
    o = out.double().cpu().numpy()
    fine = ref["written"][..., None, None] & ~hit
    assert np.all(np.abs(o - ref["out"])[fine] <= ref["bound"][fine])
    assert hit.any() and not np.isfinite(o[hit]).any()
    assert (o[~ref["written"]] == 7).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [40, 9001])
def test_a_value_that_is_not_finite_shows_however_small_its_weight(L, dtype, what):
    """Weights of e^-400 are 0 in fp32; the value is a key's that the row sees, in one piece of work or in many."""
    d, col = 64, 9
    c = AttnCase(1, 3, 4, 1, d, 16, [L], dtype, tree="chain", poison=False)
    c.q.fill_(1)                                            # scores are sums of K over 8
    c.k.fill_(25)                                           # prefix 200
    c.kt.fill_(-25)                                         # tree -200
    c.vt[0, 1, 0, col] = what
    out, lse, st = _run(c)
    assert st == 0
    o = out.double().cpu().numpy()
    hit = np.zeros(o.shape, bool)
    hit[0, 1:, :, col] = True
    assert np.isfinite(o[~hit]).all() and not np.isfinite(o[hit]).any()
    # a prefix key
    c.vt[0, 1, 0, col] = 0
    c.k.fill_(-25)
    c.kt.fill_(25)
    j = L // 2
    c.v[c.table[0, j // 16], j % 16, 0, col] = what
    out, lse, st = _run(c)
    o = out.double().cpu().numpy()
    hit[0, :, :, col] = True
    assert np.isfinite(o[~hit]).all() and not np.isfinite(o[hit]).any()
