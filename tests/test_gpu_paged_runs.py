"""tree_verify_attn_paged where many pieces of one CTA's stretch have nothing
to load: row tiles that a team of CTAs leaves to some of its members, units
without keys.  Every row must be written and the status stay clear."""

import numpy as np
import pytest
import torch

from paged_util import AttnCase
from test_gpu_paged_attn import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_verify_b200 import build
    build.build()


def _lens(B, lo, hi):
    return [lo + (37 * b) % (hi - lo + 1) for b in range(B)]


# B, T, Hq, Hkv, d, P, lens, n_nodes
TEAMS = [
    (48, 40, 64, 8, 128, 16, _lens(48, 20, 90), None),                          # three row tiles
    (30, 70, 64, 8, 128, 16, _lens(30, 20, 90), None),                          # five: four of a team, then one
    (48, 40, 64, 8, 128, 16, _lens(48, 20, 90), [(40, 16, 30)[b % 3] for b in range(48)]),
    (96, 20, 64, 8, 128, 16, _lens(96, 100, 200), [(20, 12)[b % 2] for b in range(96)]),
    (96, 20, 64, 8, 128, 5, _lens(96, 100, 200), [(20, 12)[b % 2] for b in range(96)]),   # rows copied one by one
    (96, 20, 64, 8, 64, 1, _lens(96, 1, 40), [(20, 12)[b % 2] for b in range(96)]),
    (128, 36, 40, 8, 64, 24, _lens(128, 0, 60), [1 + (7 * b) % 36 for b in range(128)]),
]


@pytest.mark.parametrize("s", TEAMS, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_row_tiles_that_are_not_there(s):
    B, T, Hq, Hkv, d, P, lens, nn = s
    _check(AttnCase(B, T, Hq, Hkv, d, P, lens, "bf16", tree="random", n_nodes=nn, seed=T + P))


@pytest.mark.parametrize("d,P", [(128, 16), (64, 16), (128, 5)])
@pytest.mark.parametrize("T", [1, 20])
def test_units_without_keys(T, d, P):
    """Partials over the prefix alone, most prefixes empty: out 0 and lse -inf there."""
    B = 160
    lens = [(0 if b % 40 else 150 + b) for b in range(B)]
    lens[-1] = 0
    c = AttnCase(B, T, 64, 8, d, P, lens, "bf16", tree="chain", n_nodes=[T if b % 3 else (T + 1) // 2 for b in range(B)])
    out, lse, _ = _check(c, prefix_only=True)
    written = np.arange(T)[None] < c.n_nodes[:, None]
    none = torch.from_numpy(written & (np.asarray(lens) == 0)[:, None]).cuda()
    assert (out[none] == 0).all() and torch.isneginf(lse[none]).all()
