"""GPU parity of the paged acceptance, commit, page update and compaction
against the fp64 oracle, and of a run of the paged calls together."""

import numpy as np
import pytest
import torch

from oracle import paged as op
from paged_util import DT, tables, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_verify_b200 import build
    build.build()


def dev(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


# ------------------------------------------------------------------ acceptance

def _probs(B, T, V, seed, noise=0.7, sigma=2.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(B, T, V, generator=g, dtype=torch.float64) * sigma
    zd = z + noise * torch.randn(B, T, V, generator=g, dtype=torch.float64)
    return torch.softmax(z, -1).float(), torch.softmax(zd, -1).float(), g


def _accept_case(B, T, V, mode, tree, seed, **kw):
    p, q, g = _probs(B, T, V, seed, **kw)
    par = trees(tree, B, T, seed)
    tok = np.zeros((B, T), np.int32)
    for b in range(B):
        for j in range(1, T):
            c = par[b, j]
            if mode == "specsample":
                tok[b, j] = int(torch.multinomial(q[b, c], 1, generator=g))
            else:
                k = int(sum(par[b, 1:j] == c))
                tok[b, j] = int(torch.topk(p[b, c], min(V, k + 1)).indices[-1])
    u = torch.rand(2, B, T, generator=g, dtype=torch.float64)
    return p, (q if mode == "specsample" else None), tok, par, u[0], u[1]


def _accept(p, q, tok, par, uc, us, nn=None, **kw):
    import tree_verification_verify_b200 as tv
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B, T, _ = p.shape
    outs = dict(n_accepted=torch.full((B,), -9, dtype=torch.int32, device="cuda"),
                accepted_nodes=torch.full((B, T), -9, dtype=torch.int32, device="cuda"),
                out_tokens=torch.full((B, T + 1), -9, dtype=torch.int32, device="cuda"))
    c = lambda x: None if x is None else x.cuda()
    tv.tree_accept_probs(c(p), dev(tok), dev(par), c(uc), c(us), draft_probs=c(q),
                         n_nodes=None if nn is None else dev(nn), dev_status=st, outputs=outs, **kw)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in outs.items()}, int(st.item())


def _accept_check(p, q, tok, par, uc, us, nn=None, **kw):
    ref = op.tree_accept_probs(p, q, tok, par, uc, us, n_nodes=nn)
    # both sides sum at most V fp64 terms, so decisions nearer than V 2^-52 could fall either way: there are none
    assert ref["min_margin"].min() > p.shape[2] * 2.0 ** -48
    got, st = _accept(p, q, tok, par, uc, us, nn, **kw)
    for k in got:
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    assert st == ref["status"]
    return ref


@pytest.mark.parametrize("mode", ["specsample", "specexec"])
@pytest.mark.parametrize("B,T,V,tree", [(1, 1, 1, "chain"), (3, 2, 5, "chain"), (4, 5, 257, "chain"),
                                         (5, 9, 1000, "star"), (2, 40, 4099, "random"), (6, 16, 32000, "bfs"),
                                         (150, 6, 130, "random"), (1, 8, 151936, "bfs"), (80, 4, 9000, "star")])
def test_accept_parity(mode, B, T, V, tree):
    if mode == "specexec" and V < T:
        T = V
    case = _accept_case(B, T, V, mode, tree, seed=B + T + V)
    nn = [T - (b % 3 == 1) * (T // 2) for b in range(B)]
    _accept_check(*case, nn=nn)


@pytest.mark.parametrize("mode", ["specsample", "specexec"])
@pytest.mark.parametrize("B,T,V,tree", [(1, 3, 500001, "star"), (200, 3, 40000, "star"), (1, 4096, 300, "random")])
def test_accept_rows_that_shared_memory_does_not_hold(mode, B, T, V, tree):
    """Rows in pieces: a large vocabulary, many sequences (one CTA each), a tree that fills shared memory."""
    if T > 1000:                                             # (a random tree's nodes have few children)
        g = torch.Generator().manual_seed(9)
        p, q, _ = _probs(B, T, V, 9)
        par = trees(tree, B, T, 9)
        tok = torch.randint(0, V, (B, T), generator=g).numpy()
        if mode == "specexec":
            for c in range(T):
                kids = [j for j in range(1, T) if par[0, j] == c]
                tok[0, kids] = np.random.default_rng(c).permutation(V)[:len(kids)]
        u = torch.rand(2, B, T, generator=g, dtype=torch.float64)
        case = p, (q if mode == "specsample" else None), tok, par, u[0], u[1]
    else:
        case = _accept_case(B, T, V, mode, tree, seed=B + T)
    _accept_check(*case)


def test_accept_many_rejections():
    """A star of drafts from an unrelated distribution: residual after residual at one node."""
    p, _, g = _probs(8, 30, 600, 3)
    q = torch.softmax(torch.randn(8, 30, 600, generator=g, dtype=torch.float64), -1).float()
    par = trees("star", 8, 30)
    tok = np.stack([[0] + torch.multinomial(q[b, 0], 29, replacement=True, generator=g).tolist() for b in range(8)])
    u = torch.rand(2, 8, 30, generator=g, dtype=torch.float64)
    _accept_check(p, q, tok, par, u[0] * 0.5 + 0.5 - 2.0 ** -30, u[1])


def test_accept_equal_distributions_keep_everything():
    p, _, g = _probs(3, 10, 300, 4)
    par = trees("chain", 3, 10)
    tok = np.stack([[0] + [int(torch.multinomial(p[b, j - 1], 1, generator=g)) for j in range(1, 10)] for b in range(3)])
    u = torch.full((3, 10), 1 - 2.0 ** -53, dtype=torch.float64)
    got, st = _accept(p, p.clone(), tok, par, u, torch.rand(3, 10, generator=g, dtype=torch.float64))
    assert st == 0 and got["n_accepted"].tolist() == [9, 9, 9]


@pytest.mark.parametrize("V", [7, 1300, 40001])
def test_accept_samples_at_the_ends(V):
    """u = 0 takes the first token with weight, the largest u the last one; zeros are never drawn."""
    p, _, _ = _probs(4, 1, V, V)
    p[:, :, 0] = 0
    p[:, :, -2:] = 0
    us = torch.tensor([[0.0], [1 - 2.0 ** -53], [2.0 ** -60], [0.5]], dtype=torch.float64)
    got, st = _accept(p, None, np.zeros((4, 1)), trees("chain", 4, 1), None, us)
    assert st == 0 and got["n_accepted"].tolist() == [0] * 4
    assert got["out_tokens"][:3, 0].tolist() == [1, V - 3, 1]
    cum = torch.cumsum(p[3, 0].double(), 0)
    assert got["out_tokens"][3, 0] == int((cum <= 0.5 * cum[-1]).sum())


def test_accept_zero_residual_and_zero_draft():
    """p = q: after a rejection the residual's sum is 0 and p stays; q(x) = 0 with p(x) > 0 is accepted."""
    V = 64
    p = torch.full((3, 3, V), 1.0 / V)
    q = p.clone()
    # sequence 1: the first child's token has q = 0
    q[1, 0, 5] = 0
    # sequence 2: q is larger everywhere, so the residual is empty and the second child is tested against p
    q[2, 0] = 2.0 / V
    tok = np.array([[0, 3, 4], [0, 5, 4], [0, 3, 4]])
    uc = torch.tensor([[0, .9, .9], [0, .999, .9], [0, .75, .25]], dtype=torch.float64)
    us = torch.full((3, 3), 0.5, dtype=torch.float64)
    par = trees("star", 3, 3)
    ref = op.tree_accept_probs(p, q, tok, par, uc, us)
    got, st = _accept(p, q, tok, par, uc, us)
    assert st == ref["status"] == 0
    assert got["accepted_nodes"][:, 0].tolist() == [1, 1, 2] == ref["accepted_nodes"][:, 0].tolist()


def test_accept_faults():
    p, q, tok, par, uc, us = _accept_case(12, 6, 500, "specsample", "star", 11)
    uc[:] = 0.999999                                       # the children are tested one after the other
    nan = float("nan")
    p[0, 0, 77] = nan
    p[1, 0, 3] = -0.5
    q[2, 0, 9] = float("inf")
    uc[3, 1] = nan
    uc[4, 1] = 1.0
    us[5] = -0.1
    p[6, 0] = 0.0
    tok[7, 2] = 500
    tok[8, 1] = -1
    par[9, 3] = 3
    par[10, 0] = 0
    nn = [6] * 11 + [7]
    ref = op.tree_accept_probs(p, q, tok, par, uc, us, n_nodes=nn)
    got, st = _accept(p, q, tok, par, uc, us, nn)
    for k in got:
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
    assert st == ref["status"] == op.ST_NONFINITE | op.ST_BAD_TOKEN | op.ST_BAD_PARENT | op.ST_BAD_LEN
    assert (got["out_tokens"][[0, 1, 2, 3, 4, 5, 6]][:, 0] == -1).sum() >= 6


def test_accept_reads_only_what_it_needs():
    """A row that no test and no sample of the walk reads may hold NaN."""
    p, q, tok, par, uc, us = _accept_case(1, 3, 300, "specsample", "chain", 2)
    uc[:] = 0.0
    p[0, 0, :] = nan = float("nan")
    p[0, 0, tok[0, 1]], q[0, 0, tok[0, 1]] = 0.5, 0.5
    q[0, 2] = nan
    got, st = _accept(p, q, tok, par, uc, us)
    assert st == 0 and got["n_accepted"].tolist() == [2] and 0 <= got["out_tokens"][0, 2] < 300


def test_accept_strides_and_modes():
    p, q, tok, par, uc, us = _accept_case(3, 5, 333, "specsample", "random", 8)
    wide = torch.full((3, 5, 401), float("nan"))
    wide[:, :, 1:334] = p
    ref = op.tree_accept_probs(p, q, tok, par, uc, us)
    import tree_verification_verify_b200 as tv
    w = wide.cuda()[:, :, 1:334]                            # rows that start off 16 bytes, 401 elements apart
    o = tv.tree_accept_probs(w, dev(tok), dev(par), uc.cuda(), us.cuda(), draft_probs=q.cuda())
    np.testing.assert_array_equal(o["out_tokens"].cpu().numpy(), ref["out_tokens"])
    o = tv.tree_accept_probs(w, dev(tok), dev(par), None, us.cuda())
    ref = op.tree_accept_probs(p, None, tok, par, None, us)
    np.testing.assert_array_equal(o["out_tokens"].cpu().numpy(), ref["out_tokens"])
    for bad in (dict(mode="greedy"), dict(mode="specsample")):
        with pytest.raises(tv.TVError):
            tv.tree_accept_probs(w, dev(tok), dev(par), uc.cuda(), us.cuda(), **bad)
    with pytest.raises(tv.TVError):
        tv.tree_accept_probs(w, dev(tok), dev(par), uc.cuda().float(), us.cuda(), draft_probs=q.cuda())


def test_accept_agrees_with_the_philox_walk():
    """Philox's own numbers handed in, and the softmax of the logits: tree_accept's walk."""
    import tree_verification_verify_b200 as tv
    from synth import accept_case, tree_random_recursive
    par = tree_random_recursive(20, torch.Generator().manual_seed(5))
    c = accept_case(40, 20, 3000, par, 0.8, sigma=2.0, seed=6, correlated=True, noise=0.4, device="cuda")
    ref = tv.tree_accept(c.target_logits, c.draft_tokens, c.parent, draft_probs=c.draft_probs, temperature=0.8, seed=3)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    B, T = c.parent.shape
    P = c.parent.cpu().tolist()
    at = [(b, j) for b in range(B) for j in range(T)]
    kid = [sum(P[b][i] == P[b][j] for i in range(1, j)) if j else 0 for b, j in at]
    bs, js = i32([b for b, _ in at]), i32([j for _, j in at])
    uc = tv.philox_uniforms(3, 0, bs, i32([max(P[b][j], 0) for b, j in at]), i32(kid), i32([1] * len(at))).view(B, T)
    us = tv.philox_uniforms(3, 0, bs, js, i32([0] * len(at)), i32([2] * len(at))).view(B, T)
    p = torch.softmax(c.target_logits.double() / float(np.float32(0.8)), -1).float()
    got = tv.tree_accept_probs(p, c.draft_tokens, c.parent, uc, us, draft_probs=c.draft_probs)
    # p is rounded to fp32 here: sequences that met a decision within that rounding are left out
    far = ref["min_margin"] > 1e-5
    assert int(far.sum()) > 30 and int(ref["n_accepted"].sum()) > 20
    for k in got:
        assert torch.equal(got[k][far], ref[k][far]), k


# ------------------------------------------------------------------ commit

def _pool(layers, N, P, H, d, dtype, seed, layout="dense"):
    g = torch.Generator().manual_seed(seed)
    if layout == "heads":                                   # [layers][pages][heads][rows][d] viewed as rows, heads
        return tuple(torch.randn(layers, N, H, P, d, generator=g).to(DT[dtype]).cuda().transpose(2, 3) for _ in range(2))
    pad = 3 if layout == "padded" else 0
    return tuple(torch.randn(layers, N, P, H, d + pad, generator=g).to(DT[dtype]).cuda()[..., :d] for _ in range(2))


def _paths(B, T, rng):
    acc, n = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n[b] = rng.integers(0, T)
        acc[b, :n[b]] = np.sort(rng.permutation(np.arange(1, T))[:n[b]])
    return n, acc


def _same(k, v, ref):
    np.testing.assert_array_equal(k.double().cpu().numpy(), ref["k_pages"])
    np.testing.assert_array_equal(v.double().cpu().numpy(), ref["v_pages"])


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("layers,B,T,H,d,P,dtype,layout", [
    (1, 1, 1, 1, 64, 16, "bf16", "dense"), (3, 4, 9, 2, 128, 16, "bf16", "dense"), (2, 5, 6, 3, 33, 5, "bf16", "dense"),
    (2, 3, 300, 1, 64, 7, "fp32", "heads"), (1, 3, 8, 2, 80, 24, "fp32", "padded"), (33, 2, 4, 8, 16, 1, "bf16", "heads")])
def test_commit_parity(layers, B, T, H, d, P, dtype, layout, inplace):
    import tree_verification_verify_b200 as tv
    rng = np.random.default_rng(T + d)
    lens = rng.integers(0, 40, B)
    room = lens + T
    N = int(sum(-(-r // P) for r in room)) + 1
    table = tables(room, P, int(max(-(-r // P) for r in room)), N, T)
    k, v = _pool(layers, N, P, H, d, dtype, 1, layout)
    kt, vt = _pool(layers, B, T, H, d, dtype, 2)
    n, acc = _paths(B, T, rng)
    ref = op.tree_commit_kv_paged(k, v, table, lens, kt, vt, n, acc)
    L = dev(lens)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = None if inplace else torch.full_like(L, -5)
    got = tv.tree_commit_kv_paged(k, v, dev(table), L, kt, vt, dev(n), dev(acc), prefix_len_out=out, dev_status=st)
    torch.cuda.synchronize()
    _same(k, v, ref)
    assert got.cpu().tolist() == ref["prefix_len"].tolist() and int(st.item()) == ref["status"] == 0
    if not inplace:
        assert L.cpu().tolist() == lens.tolist()


def test_commit_one_layer_without_the_layer_dimension():
    import tree_verification_verify_b200 as tv
    rng = np.random.default_rng(1)
    k, v = _pool(1, 12, 4, 2, 64, "bf16", 5)
    kt, vt = _pool(1, 2, 5, 2, 64, "bf16", 6)
    table = tables([20, 20], 4, 5, 12, 3)
    n, acc = _paths(2, 5, rng)
    ref = op.tree_commit_kv_paged(k, v, table, [3, 0], kt, vt, n, acc)
    L = dev([3, 0])
    tv.tree_commit_kv_paged(k[0], v[0], dev(table), L, kt[0], vt[0], dev(n), dev(acc))
    torch.cuda.synchronize()
    _same(k, v, ref)
    assert L.cpu().tolist() == ref["prefix_len"].tolist()


def test_commit_faults_leave_a_sequence_alone():
    import tree_verification_verify_b200 as tv
    B, T, P, W = 8, 5, 4, 4
    k, v = _pool(2, 40, P, 1, 16, "fp32", 7)
    kt, vt = _pool(2, B, T, 1, 16, "fp32", 8)
    table = tables([W * P] * B, P, W, 40, 4)
    lens = np.array([3, -1, 14, 3, 3, 3, 7, 3])
    n = np.array([2, 1, 2, 5, 2, 2, 2, -1])
    acc = np.tile(np.array([1, 3, -1, -1, -1]), (B, 1))
    acc[4, 0] = 5
    acc[5, 1] = 1
    table[6, 2] = 40
    ref = op.tree_commit_kv_paged(k, v, table, lens, kt, vt, n, acc)
    L, st = dev(lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.tree_commit_kv_paged(k, v, dev(table), L, kt, vt, dev(n), dev(acc), dev_status=st)
    torch.cuda.synchronize()
    _same(k, v, ref)
    assert L.cpu().tolist() == ref["prefix_len"].tolist() == [6] + lens[1:].tolist()
    assert int(st.item()) == ref["status"] == op.ST_BAD_LEN | op.ST_BAD_ROW | op.ST_BAD_PAGE


def test_commit_at_the_longest_length():
    """A length is an int32: 2^31 - 2 rows take one more, 2^31 - 1 take none."""
    import tree_verification_verify_b200 as tv
    P = 65536
    k = torch.zeros(2, P, 1, 4, device="cuda")
    v = torch.zeros_like(k)
    table = torch.zeros(2, 32768, dtype=torch.int32, device="cuda")
    table[1] = 1
    tree = torch.ones(2, 1, 1, 4, device="cuda")
    L, st = dev([2 ** 31 - 2, 2 ** 31 - 1]), dev([0])
    tv.tree_commit_kv_paged(k, v, table, L, tree, tree, dev([0, 0]), dev([[-1], [-1]]), dev_status=st)
    torch.cuda.synchronize()
    assert L.tolist() == [2 ** 31 - 1] * 2 and int(st.item()) == op.ST_BAD_LEN
    assert k[0, P - 2].eq(1).all() and float(k.sum()) == 4 and float(v.sum()) == 4


# ------------------------------------------------------------------ page tables

def _update(k, v, table, src, keep, grow, W, pinned=None):
    import tree_verification_verify_b200 as tv
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((len(src), W), -9, dtype=torch.int32, device="cuda")
    got, n_free = tv.tree_pages_update(k, v, dev(table), dev(src), dev(keep), dev(grow),
                                       pinned=None if pinned is None else dev(pinned), out=out, dev_status=st)
    torch.cuda.synchronize()
    return got.cpu().numpy(), int(n_free.item()), int(st.item())


@pytest.mark.parametrize("layout", ["dense", "heads", "padded"])
@pytest.mark.parametrize("seed", range(12))
def test_update_parity(seed, layout):
    rng = np.random.default_rng(seed)
    P, d = int(rng.choice([1, 3, 8, 16, 64])), int(rng.choice([16, 33, 128]))
    B_in, B = int(rng.integers(1, 9)), int(rng.integers(1, 40))
    lens = rng.integers(0, 120, B_in)
    W = int(-(-(lens.max() + 20) // P) + rng.integers(0, 3))
    N = int(sum(-(-n // P) for n in lens)) + B * (20 // P + 2) + 5
    table = tables(lens, P, W, N, seed)
    src = rng.integers(-1, B_in, B)
    keep = np.array([0 if s < 0 else (lens[s] if rng.random() < 0.7 else rng.integers(0, lens[s] + 1)) for s in src])
    grow = rng.integers(0, 20, B) * (rng.random(B) < 0.8)
    pinned = (rng.random(N) < 0.05).astype(np.int32) * 3 if seed % 2 else None
    k, v = _pool(2, N, P, 2, d, "bf16" if seed % 3 else "fp32", seed, layout)
    ref = op.tree_pages_update(k, v, table, src, keep, grow, W, pinned)
    got, n_free, st = _update(k, v, table, src, keep, grow, W, pinned)
    np.testing.assert_array_equal(got, ref["page_table"])
    assert n_free == ref["n_free"] and st == ref["status"]
    _same(k, v, ref)


def test_update_of_large_tables():
    """More sequences than the plan has warps, more pages than a CTA scans at a time."""
    rng = np.random.default_rng(0)
    B, P, W, N = 3000, 2, 40, 300001
    lens = rng.integers(0, 60, B)
    table = tables(lens, P, W, N, 1)
    src = rng.integers(-1, B, B)
    keep = np.where(src < 0, 0, lens[np.maximum(src, 0)])
    grow = rng.integers(0, 20, B)
    pinned = (rng.random(N) < 0.4).astype(np.int32)
    k, v = _pool(1, N, P, 1, 2, "bf16", 0)
    ref = op.tree_pages_update(k, v, table, src, keep, grow, W, pinned)
    got, n_free, st = _update(k, v, table, src, keep, grow, W, pinned)
    np.testing.assert_array_equal(got, ref["page_table"])
    assert n_free == ref["n_free"] and st == 0
    _same(k, v, ref)


def test_update_without_room_changes_nothing():
    k, v = _pool(1, 6, 4, 1, 16, "bf16", 3)
    before = k.clone(), v.clone()
    table = tables([10, 9], 4, 4, 6, 2)
    src, keep, grow = [0, 0, 1], [10, 10, 9], [4, 4, 4]
    ref = op.tree_pages_update(k, v, table, src, keep, grow, 4)
    got, n_free, st = _update(k, v, table, src, keep, grow, 4)
    assert n_free == ref["n_free"] < 0 and st == op.ST_NO_PAGES == ref["status"] and (got == -1).all()
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    # exactly enough
    keep, grow = [10, 0, 9], [2, 0, 3]
    ref = op.tree_pages_update(k, v, table, [0, -1, 1], keep, grow, 4)
    got, n_free, st = _update(k, v, table, [0, -1, 1], keep, grow, 4)
    np.testing.assert_array_equal(got, ref["page_table"])
    assert st == 0 and n_free == ref["n_free"]


def test_update_faults_and_empty_batches():
    k, v = _pool(1, 30, 4, 1, 16, "bf16", 3)
    lens = [10, 9, 16]
    table = tables(lens, 4, 4, 30, 2)
    table[2, 3] = 30
    src = [0, 3, -2, 1, 1, 2, 2, 0, -1]
    keep = [10, 1, 1, 17, -1, 16, 12, 10, 5]
    grow = [1, 1, 1, 0, 1, 0, 2, -1, 3]
    ref = op.tree_pages_update(k, v, table, src, keep, grow, 4)
    got, n_free, st = _update(k, v, table, src, keep, grow, 4)
    np.testing.assert_array_equal(got, ref["page_table"])
    assert n_free == ref["n_free"] and st == ref["status"] == op.ST_BAD_ROW | op.ST_BAD_LEN | op.ST_BAD_PAGE
    _same(k, v, ref)
    got, n_free, st = _update(k, v, table, [], [], [], 4, np.arange(30) < 4)
    assert got.shape == (0, 4) and n_free == 26 and st == 0
    got, n_free, st = _update(k, v, np.zeros((0, 4)), [-1, -1], [0, 0], [5, 0], 4)
    assert got.tolist() == [[0, 1, -1, -1], [-1] * 4] and n_free == 28 and st == 0


def test_update_refuses_its_own_table():
    import tree_verification_verify_b200 as tv
    k, v = _pool(1, 6, 4, 1, 16, "bf16", 3)
    t = dev(tables([10, 9], 4, 4, 6, 2))
    z = dev([0, 1])
    with pytest.raises(tv.TVError):
        tv.tree_pages_update(k, v, t, z, dev([10, 9]), z, out=t)
    with pytest.raises(tv.TVError):
        tv.tree_pages_update(k, v, t, z, dev([10, 9]), z.long())
    with pytest.raises(tv.TVError):
        tv.tree_pages_compact(k, v, t, dev([10, 9]), out=t[:, :3])


@pytest.mark.parametrize("layout", ["dense", "heads", "padded"])
@pytest.mark.parametrize("seed", range(12))
def test_compact_parity(seed, layout):
    import tree_verification_verify_b200 as tv
    rng = np.random.default_rng(100 + seed)
    P, d, B = int(rng.choice([1, 3, 8, 16, 64])), int(rng.choice([16, 33, 128])), int(rng.integers(1, 30))
    lens = rng.integers(0, 150, B)
    W = int(-(-lens.max() // P) + rng.integers(1, 3))
    need = int(sum(-(-n // P) for n in lens))
    N = need + int(rng.integers(0, need + 40))
    table = tables(lens, P, W, N, seed)
    if B > 2:                                               # a shared prefix
        table[1], lens[1] = table[0], lens[0] // 2
    pinned = (rng.random(N) < 0.1).astype(np.int32) if seed % 2 else None
    k, v = _pool(2, N, P, 2, d, "bf16" if seed % 3 else "fp32", seed, layout)
    ref = op.tree_pages_compact(k, v, table, lens, pinned)
    t, st = dev(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, n_used = tv.tree_pages_compact(k, v, t, dev(lens), pinned=None if pinned is None else dev(pinned),
                                        out=t if seed % 4 < 2 else None, dev_status=st)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out.cpu().numpy(), ref["page_table"])
    assert int(n_used.item()) == ref["n_used"] and int(st.item()) == 0
    _same(k, v, ref)


def test_compact_faults_and_ends():
    import tree_verification_verify_b200 as tv
    k, v = _pool(1, 40, 4, 1, 16, "bf16", 3)
    lens = [10, 17, -3, 8, 0]
    table = tables([10, 16, 4, 8, 0], 4, 4, 40, 9)
    table[3, 1] = -2
    ref = op.tree_pages_compact(k, v, table, lens)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, n_used = tv.tree_pages_compact(k, v, dev(table), dev(lens), dev_status=st)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out.cpu().numpy(), ref["page_table"])
    assert int(n_used.item()) == ref["n_used"] and int(st.item()) == ref["status"] == op.ST_BAD_LEN | op.ST_BAD_PAGE
    _same(k, v, ref)
    out, n_used = tv.tree_pages_compact(k, v, dev(np.zeros((0, 4))), dev([]))
    assert out.shape == (0, 4) and int(n_used.item()) == 0
    # a full pool and a large one
    for N, B in ((64, 16), (70001, 900)):
        k, v = _pool(1, N, 1, 1, 8, "bf16", 3)
        lens = np.full(B, N // B if B == 16 else 40)
        table = tables(lens, 1, int(lens.max()), N, 5)
        ref = op.tree_pages_compact(k, v, table, lens)
        out, n_used = tv.tree_pages_compact(k, v, dev(table), dev(lens))
        np.testing.assert_array_equal(out.cpu().numpy(), ref["page_table"])
        assert int(n_used.item()) == ref["n_used"]
        _same(k, v, ref)


# ------------------------------------------------------------------ together

def test_a_server_over_pages_equals_contiguous_caches():
    """Steps of a small server: fork and grow, attention, acceptance, commit, compaction, captured into one graph, against
    the contiguous calls on caches that are copied row by row."""
    import tree_verification_verify_b200 as tv
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    B, T, Hq, H, d, P, W, N, V = 4, 6, 8, 2, 64, 16, 20, 90, 200
    k, v = r(1, N, P, H, d), r(1, N, P, H, d)
    lens = dev([30, 17, 0, 64])
    table = dev(tables([30, 17, 0, 64], P, W, N, 3))
    parent = dev(trees("random", B, T, 1))
    flat = torch.zeros(2, B, W * P, H, d, dtype=torch.bfloat16, device="cuda")
    for b, n in enumerate(lens.tolist()):
        for j in range(n):
            flat[0, b, j], flat[1, b, j] = k[0, table[b, j // P], j % P], v[0, table[b, j // P], j % P]
    io = dict(q=r(B, T, Hq, d), kt=r(1, B, T, H, d), vt=r(1, B, T, H, d), p=torch.full((B, T, V), 1 / V, device="cuda"),
              dq=torch.full((B, T, V), 1 / V, device="cuda"), tok=dev(np.zeros((B, T))), u=torch.zeros(2, B, T, device="cuda",
                                                                                              dtype=torch.float64),
              src=dev(range(B)), grow=dev([T] * B))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        keep = lens[io["src"].long()]
        new, n_free = tv.tree_pages_update(k, v, table, io["src"], keep, io["grow"], dev_status=st)
        out, lse = tv.tree_verify_attn_paged(io["q"], k[0], v[0], new, keep, io["kt"][0], io["vt"][0], parent, dev_status=st)
        o = tv.tree_accept_probs(io["p"], io["tok"], parent, io["u"][0], io["u"][1], draft_probs=io["dq"], dev_status=st)
        tv.tree_commit_kv_paged(k, v, new, keep, io["kt"], io["vt"], o["n_accepted"], o["accepted_nodes"], dev_status=st)
        tv.tree_pages_compact(k, v, new, keep, out=new, dev_status=st)
        table.copy_(new)
        lens.copy_(keep)
        return out, lse, o, n_free

    keepsake = [x.clone() for x in (k, v, table, lens)]
    step()                                                  # before the capture
    for x, y in zip((k, v, table, lens), keepsake):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i, src in enumerate(([0, 1, 2, 3], [3, 1, 3, 3], [0, 0, 2, 2], [1, 1, 1, 1], [0, 1, 2, 3])):
        p, q, gen = _probs(B, T, V, 50 + i, noise=0.3)
        io["p"].copy_(p)
        io["dq"].copy_(q)
        io["tok"].copy_(torch.stack([torch.multinomial(q[b, parent[b].cpu().clamp(min=0).long()], 1, generator=gen)[:, 0]
                                     for b in range(B)]))
        io["u"].copy_(torch.rand(2, B, T, generator=gen, dtype=torch.float64))
        io["src"].copy_(dev(src))
        for x in ("q", "kt", "vt"):
            io[x].copy_(r(*io[x].shape))
        s = io["src"].long()
        flat = flat[:, s].clone()
        flen = lens[s].clone()
        ref, rlse, _ = tv.tree_verify_attn(io["q"], flat[0], flat[1], flen, io["kt"][0], io["vt"][0], parent)
        want = op.tree_accept_probs(p, q, io["tok"].cpu(), parent.cpu(), io["u"][0].cpu(), io["u"][1].cpu())
        graph.replay()
        torch.cuda.synchronize()
        out, lse, o, n_free = outs
        # each side rounds its weights (2^-8 of sum p |v|) and its output (2^-8 of |o|) to bf16, and both sums are at
        # most the largest |v|, which passes 4 here: 4 * 2^-8 of it in all (1/64 alone is one step of a value in [2, 4))
        vmax = max(flat[1].abs().max().item(), io["vt"].abs().max().item())
        assert (out.float() - ref.float()).abs().max() <= 2.0 ** -6 * vmax and (lse - rlse).abs().max() < 1e-4
        np.testing.assert_array_equal(o["out_tokens"].cpu().numpy(), want["out_tokens"])
        tv.tree_commit_kv(flat[0], flat[1], flen, io["kt"][0], io["vt"][0], o["n_accepted"], o["accepted_nodes"])
        assert torch.equal(lens, flen) and int(st.item()) == 0
        used = set()
        for b, n in enumerate(lens.tolist()):
            rows = torch.arange(n, device="cuda")
            pg = table[b, rows // P].long()
            assert torch.equal(k[0, pg, rows % P], flat[0, b, :n]) and torch.equal(v[0, pg, rows % P], flat[1, b, :n])
            used |= set(pg.tolist())
        assert not used or max(used) < len(used)
