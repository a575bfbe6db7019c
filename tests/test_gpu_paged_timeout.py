"""A wait of the tensor-core kernel of tree_verify_attn_paged that runs out
(test hook: pieces of work or products that never come, nothing in flight is
lost): every row is NaN, none is left from an earlier call, the status says
so, and the next call is as ever."""

import numpy as np
import pytest
import torch

from paged_util import AttnCase, check_attn
from test_gpu_paged_attn import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_verify_b200 import build
    build.build()


# B, T, Hq, Hkv, d, P, lens, n_nodes: pieces of one unit in many CTAs, whole
# units, row tiles on a team of three, rows copied one by one
CASES = [
    (2, 3, 8, 2, 128, 16, [9001, 4], None),
    (40, 5, 16, 4, 64, 16, [(97 * i) % 500 + 1 for i in range(40)], [i % 6 for i in range(40)]),
    (30, 40, 64, 8, 128, 64, [300 + i for i in range(30)], None),
    (12, 4, 16, 4, 128, 5, [200 + 31 * i for i in range(12)], None),
]


@pytest.mark.parametrize("lost", [1, 2])
@pytest.mark.parametrize("s", CASES, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_a_wait_that_runs_out(s, lost):
    import tree_verification_verify_b200 as tv
    B, T, Hq, Hkv, d, P, lens, nn = s
    c = AttnCase(B, T, Hq, Hkv, d, P, lens, "bf16", n_nodes=nn, seed=B)
    ref = c.oracle()
    want, want_lse, st = _run(c)                            # (leaves finite partial rows in the workspace)
    assert st == 0
    check_attn(want, want_lse, ref, poison=7.0)
    tv.paged.attn_set_lost(lost)
    try:
        out, lse, st = _run(c)
    finally:
        tv.paged.attn_set_lost(0)
    assert st == 32                                         # TV_DEV_TIMEOUT
    w = torch.from_numpy(np.broadcast_to(ref["written"], out.shape[:2]).copy()).cuda()
    assert out[w].isnan().all() and lse[w].isnan().all()
    assert (out[~w] == 7).all() and (lse[~w] == 7).all()
    out, lse, st = _run(c)
    assert st == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_units_without_keys_are_not_concerned():
    import tree_verification_verify_b200 as tv
    c = AttnCase(3, 2, 8, 2, 128, 16, [0, 0, 0], "bf16", tree="chain")
    for lost in (1, 2):
        tv.paged.attn_set_lost(lost)
        try:
            out, lse, st = _run(c, prefix_only=True)
        finally:
            tv.paged.attn_set_lost(0)
        assert st == 0 and (out == 0).all() and torch.isneginf(lse).all()


def test_the_hook_refuses_what_it_does_not_know():
    import tree_verification_verify_b200 as tv
    for lost in (-1, 3):
        with pytest.raises(tv.TVError):
            tv.paged.attn_set_lost(lost)
