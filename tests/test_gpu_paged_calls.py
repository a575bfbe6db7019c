"""Calls of the paged cache's API that its documentation allows and that go
beyond the plain ones: outputs given in part, device memory that runs out."""

import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_verify_b200 import build
    build.build()


def _accept_case(B=3, T=4, V=50):
    g = torch.Generator().manual_seed(5)
    p = torch.softmax(torch.randn(B, T, V, generator=g) * 2, -1).cuda()
    q = torch.softmax(torch.randn(B, T, V, generator=g) * 2, -1).cuda()
    tok = torch.randint(0, V, (B, T), generator=g).to(torch.int32).cuda()
    parent = torch.tensor([[-1, 0, 0, 1]] * B, dtype=torch.int32).cuda()
    u = torch.rand(2, B, T, generator=g, dtype=torch.float64).cuda()
    return (p, tok, parent, u[0].contiguous(), u[1].contiguous()), dict(draft_probs=q)


def test_acceptance_returns_every_output_whichever_are_given():
    import tree_verification_verify_b200 as tv
    args, kw = _accept_case()
    want = tv.tree_accept_probs(*args, **kw)
    names = list(want)
    for n in range(len(names) + 1):
        for some in itertools.combinations(names, n):
            given = {k: torch.full_like(want[k], -9) for k in some}
            got = tv.tree_accept_probs(*args, **kw, outputs=dict(given))
            assert set(got) == set(names)
            for k in names:
                assert torch.equal(got[k], want[k])
                assert k not in given or got[k] is given[k]
    whole = {k: torch.empty_like(v) for k, v in want.items()}
    assert tv.tree_accept_probs(*args, **kw, outputs=whole) is whole
