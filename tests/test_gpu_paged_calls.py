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


def test_device_memory_that_runs_out_is_torchs_error():
    """An output of 2^40 bytes cannot be made (its inputs are views of little memory); the next call is as ever."""
    import tree_verification_verify_b200 as tv
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    B, T = 2 ** 20, 64
    x = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(1, 16, 1, 128, dtype=torch.bfloat16, device="cuda")
    q, tree = x.expand(B, T, 64, 128), x.expand(B, T, 1, 128)
    with pytest.raises(torch.OutOfMemoryError):
        tv.tree_verify_attn_paged(q, pool, pool, i32(B, 1), i32(B), tree, tree, i32(1, T).expand(B, T))
    out, _ = tv.tree_verify_attn_paged(x, pool, pool, i32(1, 1), i32(1) + 3, x, x, i32(1, 1) - 1)
    assert (out == 0).all()
