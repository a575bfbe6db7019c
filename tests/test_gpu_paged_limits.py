"""The paged cache's row moves at the largest pages and rows that are taken:
two-byte words (an odd number of bf16 a row) whose counts come within a step
of 2^31."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_verify_b200 import build
    build.build()
    yield
    torch.cuda.empty_cache()                                # (tens of GB)


def _random(*shape):
    x = torch.empty(shape, dtype=torch.int16, device="cuda")
    return x.random_(-32768, 32767).view(torch.bfloat16)


def _same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("in_place", [False, True])
def test_compaction_of_the_largest_pages(in_place):
    """Pages of 65534 * 33 * 993 = 2^31 - 2 elements: the one in use moves to the front, whole."""
    import tree_verification_verify_b200 as tv
    P, H, d = 65534, 33, 993
    assert P * H * d == 2 ** 31 - 2
    k, v = _random(2, P, H, d), _random(2, P, H, d)
    table, st = _i32([[1]]), _i32([0])
    out, used = tv.tree_pages_compact(k, v, table, _i32([P]), out=table if in_place else None, dev_status=st)
    torch.cuda.synchronize()
    assert out.tolist() == [[0]] and used.tolist() == [1] and st.item() == 0
    assert _same(k[0], k[1]) and _same(v[0], v[1])


def test_commit_of_the_widest_rows():
    """256 rows of 2^23 two-byte words: 2^31 of them in one path."""
    import tree_verification_verify_b200 as tv
    T, H = 256, 2 ** 23
    kt, vt = _random(1, T, H, 1), _random(1, T, H, 1)
    k, v = (torch.zeros(T, 1, H, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    order = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    acc = torch.cat([torch.arange(1, T, dtype=torch.int32, device="cuda"), _i32([-1])])[None]
    n = tv.tree_commit_kv_paged(k, v, order[None], _i32([0]), kt, vt, _i32([T - 1]), acc)
    torch.cuda.synchronize()
    assert n.tolist() == [T]
    for pool, tree in ((k, kt), (v, vt)):
        for r in range(T):
            assert _same(pool[order[r]], tree[0, r][None])


def test_sizes_past_32_bits_are_refused():
    """Sizes that would wrap in the C ABI's 32-bit fields, as views of little memory where that is possible."""
    import tree_verification_verify_b200 as tv
    big = 2 ** 32
    page = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    pool = page.expand(big + 3, 4, 1, 64)
    layers = page[None].expand(big + 1, 1, 4, 1, 64)
    tree, q = page[:, :1], torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    table, one = _i32([[0]]), _i32([1])
    with pytest.raises(tv.TVError, match="num_pages"):
        tv.tree_verify_attn_paged(q, pool, pool, table, one, tree, tree, _i32([[-1]]))
    with pytest.raises(tv.TVError, match="num_pages"):
        tv.tree_commit_kv_paged(pool, pool, table, one, tree, tree, _i32([0]), _i32([[-1]]))
    with pytest.raises(tv.TVError, match="layers"):
        tv.tree_pages_update(layers, layers, table, _i32([0]), one, one)
    with pytest.raises(tv.TVError, match="layers"):
        tv.tree_pages_compact(layers, layers, table, one)
    p = torch.zeros(1, 1, big + 5, device="cuda")
    u = torch.zeros(1, 1, dtype=torch.float64, device="cuda")
    with pytest.raises(tv.TVError, match="V must be"):
        tv.tree_accept_probs(p, _i32([[0]]), _i32([[-1]]), u, u)
