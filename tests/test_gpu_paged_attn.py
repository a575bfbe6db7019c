"""GPU parity of tree_verify_attn_paged against the fp64 oracle, by an
element-wise error bound (tests/paged_util.py)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as op
from paged_util import AttnCase, check_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_verify_b200 import build
    build.build()


def _run(c, **kw):
    import tree_verification_verify_b200 as tv
    a = c.cuda()
    out = torch.full_like(a["q"], 7.0)
    lse = torch.full(a["q"].shape[:3], 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.tree_verify_attn_paged(**a, out=out, lse=lse, dev_status=st, **kw)
    torch.cuda.synchronize()
    return out, lse, int(st.item())


def _check(c, **kw):
    ref = c.oracle(**kw)
    out, lse, st = _run(c, **kw)
    check_attn(out, lse, ref, poison=7.0)
    assert st == ref["status"]
    return out, lse, ref


# single tokens and trees, short and long, page sizes that do and do not
# divide a key tile, head groups of every kind
SHAPES = [
    # B, T, Hq, Hkv, d, P, lens, tree, n_nodes
    (1, 1, 8, 2, 64, 16, [1], "chain", None),
    (2, 1, 8, 8, 128, 16, [0, 5], "chain", None),
    (3, 1, 32, 8, 128, 16, [700, 129, 128], "chain", None),
    (4, 5, 16, 2, 128, 64, [127, 0, 300, 1], "random", [5, 1, 3, 0]),
    (2, 16, 28, 4, 128, 24, [1000, 333], "bfs", None),
    (2, 33, 8, 2, 64, 5, [97, 210], "random", [33, 20]),
    (1, 64, 16, 4, 128, 128, [513], "bfs", None),
    (2, 40, 10, 2, 64, 1, [64, 65], "star", [40, 7]),
    (1, 130, 4, 2, 64, 8, [260], "random", [129]),
    (1, 300, 4, 1, 128, 32, [100], "chain", None),
    (1, 3, 64, 1, 128, 256, [511], "star", None),
    (3, 7, 6, 2, 128, 48, [47, 48, 49], "random", None),
    (2, 4, 4, 1, 32, 16, [130, 63], "random", None),
    (40, 2, 4, 2, 64, 16, [(37 * i) % 90 for i in range(40)], "chain", [i % 3 for i in range(40)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("s", SHAPES, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_parity(s, dtype):
    B, T, Hq, Hkv, d, P, lens, tree, nn = s
    _check(AttnCase(B, T, Hq, Hkv, d, P, lens, dtype, tree=tree, n_nodes=nn, seed=T + d))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_long_sequence_is_split_over_the_gpu_and_merged(dtype):
    c = AttnCase(2, 3, 8, 2, 128, 16, [9001, 4], dtype, tree="chain")
    out, lse, _ = _check(c)
    again, lse2, _ = _run(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


# more rows than one row tile: two, three and seven tiles of 128 rows, read by
# teams of two and four; trees of several key tiles; sequences of few nodes
# next to those of many
TEAMS = [
    (2, 40, 16, 2, 128, 16, [600, 77], "random", [40, 17]),
    (3, 200, 8, 2, 64, 16, [700, 0, 129], "random", [200, 3, 130]),
    (2, 50, 12, 2, 128, 32, [300, 1], "bfs", [43, 42]),
    (2, 600, 2, 2, 128, 64, [40, 200], "random", [600, 513]),
    (1, 150, 20, 4, 128, 5, [333], "bfs", None),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("s", TEAMS, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_row_tiles_of_wide_trees(s, dtype):
    B, T, Hq, Hkv, d, P, lens, tree, nn = s
    _check(AttnCase(B, T, Hq, Hkv, d, P, lens, dtype, tree=tree, n_nodes=nn, seed=T + d))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
@pytest.mark.parametrize("prefix_only", [False, True])
def test_many_sequences_of_any_length(dtype, d, prefix_only):
    """More tiles than four per CTA, so that borders of units count in the split; empty sequences among them."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 5000, 24)]
    lens[3] = lens[4] = lens[23] = 0
    nn = [int(x) for x in rng.integers(0, 3, 24)]
    c = AttnCase(24, 2, 8, 8, d, 16, lens, dtype, tree="chain", n_nodes=nn)
    _check(c, prefix_only=prefix_only)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["nphd", "nhpd"])
def test_strided_pools_and_outputs(dtype, layout):
    import tree_verification_verify_b200 as tv
    c = AttnCase(2, 6, 8, 2, 64, 16, [75, 33], dtype, layout=layout)
    ref = c.oracle()
    a = c.cuda()
    big = torch.zeros(2, 6, 12, 64, dtype=c.dt, device="cuda")
    big[:, :, 2:10] = a["q"]
    a["q"] = big[:, :, 2:10]                               # heads inside a wider projection
    wide = torch.full((2, 6, 8, 80), 7.0, dtype=c.dt, device="cuda")
    out, lse = tv.tree_verify_attn_paged(**a, out=wide[..., 8:72])
    torch.cuda.synchronize()
    check_attn(out, lse, ref)
    assert (wide[..., :8] == 7).all() and (wide[..., 72:] == 7).all()


def test_unaligned_pool_takes_the_cuda_core_kernel():
    import tree_verification_verify_b200 as tv
    c = AttnCase(2, 6, 8, 2, 64, 16, [75, 33], "bf16")
    ref = c.oracle()
    a = c.cuda()
    for k in ("k_pages", "v_pages"):
        x = torch.empty(a[k].numel() + 1, dtype=c.dt, device="cuda")[1:].view(a[k].shape)
        a[k] = x.copy_(a[k])
    out, lse = tv.tree_verify_attn_paged(**a)
    torch.cuda.synchronize()
    check_attn(out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefix_only_partials_merge_to_the_whole(dtype):
    import tree_verification_verify_b200 as tv
    lens = [0, 150, 31]
    c = AttnCase(3, 5, 8, 2, 128, 16, lens, dtype, n_nodes=[5, 4, 5])
    _check(c, prefix_only=True)
    # the tree alone (an empty prefix) and the prefix alone are two partials of the whole
    a = c.cuda()
    o1, l1 = tv.tree_verify_attn_paged(**a, prefix_only=True)
    o2, l2 = tv.tree_verify_attn_paged(**dict(a, prefix_len=torch.zeros_like(a["prefix_len"])))
    out, lse = tv.tree_verify_attn_merge(torch.stack([o1, o2]), torch.stack([l1, l2]))
    torch.cuda.synchronize()
    ref = c.oracle()
    extra = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -22)   # the partials and the merged row are rounded once more each
    ok = ref["valid"] & ref["written"]
    d = np.abs(out.double().cpu().numpy() - ref["out"])[ok]
    assert np.all(d <= 2 * ref["bound"][ok] + extra * np.abs(ref["out"][ok]) + extra * ref["bound"][ok].max() * 256)


def test_scale_and_defaults():
    c = AttnCase(1, 4, 4, 1, 64, 16, [40], "fp32")
    _check(c, scale=0.37)
    import tree_verification_verify_b200 as tv
    out, lse = tv.tree_verify_attn_paged(**c.cuda(), want_lse=False)
    torch.cuda.synchronize()
    assert lse is None
    check_attn(out, None, c.oracle())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_faults_are_contained(dtype):
    T, lens = 6, [40, 70, 33, 20]
    c = AttnCase(4, T, 8, 2, 64, 16, lens, dtype)
    c.table[1, 2] = -3                                      # a page in use out of range
    c.lens[2] = c.table.shape[1] * 16 + 1                   # longer than the table
    c.parent[3, 2] = 4                                      # a malformed parent: node 2 and what hangs off it
    c.parent[3, 3:] = [0, 2, 3]
    ref = op.tree_verify_attn_paged(c.q, torch.nan_to_num(c.k.float()), torch.nan_to_num(c.v.float()), c.table, c.lens,
                                    c.kt, c.vt, c.parent)
    out, lse, st = _run(c)
    assert st == ref["status"] == op.ST_BAD_PAGE | op.ST_BAD_LEN | op.ST_BAD_PARENT
    o = out.double().cpu().numpy()
    assert ref["valid"].tolist() == [[True] * 6, [False] * 6, [False] * 6, [True, True, False, True, False, True]]
    assert np.isnan(o[~ref["valid"]]).all() and np.isnan(lse.cpu().numpy()[~ref["valid"]]).all()
    assert np.abs(o - ref["out"])[ref["valid"]].max() < 2.0 ** -5
    c = AttnCase(2, T, 8, 2, 64, 16, [40, 3], dtype, n_nodes=[T + 1, 2])
    out, _, st = _run(c)
    assert st == op.ST_BAD_LEN and (out[0] == 7).all() and not out[1, :2].isnan().any() and (out[1, 2:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_masked_values_do_not_reach_other_rows(dtype, what):
    """K/V of nodes past n_nodes and of nodes on other branches may hold anything; the rows that see such a node show it."""
    c = AttnCase(2, 9, 8, 2, 64, 16, [40, 140], dtype, tree="star", n_nodes=[6, 9])
    ref = c.oracle()
    for t in (c.kt, c.vt):
        t[0, 6:] = what
        t[0, 3] = what
    c.vt[1, 5, 1, 7] = what                                 # (in K an infinity may give the key no weight at all)
    out, lse, st = _run(c)
    assert st == 0
    o = out.double().cpu().numpy()
    hit = np.zeros((2, 9, 8, 64), bool)
    hit[0, 3] = True
    hit[1, 5, 4:] = True                                    # kv head 1 serves query heads 4 .. 7
    ok = ref["written"][..., None, None] & ~hit
    assert np.all(np.abs(o - ref["out"])[ok] <= ref["bound"][ok])
    assert not np.isfinite(o[0, 3]).any() and not np.isfinite(o[1, 5, 4:, 7]).any()


def test_nonfinite_tree_values_alone_in_v():
    """A visible V value that is not finite shows in its column only."""
    c = AttnCase(1, 5, 4, 1, 64, 16, [30], "bf16", tree="chain")
    ref = c.oracle()
    c.vt[0, 2, 0, 9] = float("inf")
    c.vt[0, 4, 0, 9] = float("-inf")
    out, _, _ = _run(c)
    o = out.double().cpu().numpy()
    assert np.isposinf(o[0, 2:4, :, 9]).all() and np.isnan(o[0, 4, :, 9]).all()
    fine = np.isfinite(o)
    assert fine.sum() == 5 * 4 * 64 - 3 * 4
    assert np.all(np.abs(o - ref["out"])[fine] <= ref["bound"][fine])


def test_shared_pages_and_wide_tables():
    """Two sequences read one prefix from the same pages; the table has far more columns than any sequence uses."""
    c = AttnCase(3, 4, 8, 2, 128, 16, [64, 100, 64], "bf16")
    c.table[2, :4] = c.table[0, :4]
    wide = np.full((3, 5000), 2 ** 31 - 1, np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    _check(c)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 32)])
def test_offsets_past_32_bits(dtype, d):
    """Pages that lie more than 2^31 elements into the pool."""
    import tree_verification_verify_b200 as tv
    c = AttnCase(1, 3, 4, 2, d, 16, [70], dtype, tree="chain")
    ref = c.oracle()
    a = c.cuda()
    row = 16 * 2 * d
    N = 2 ** 31 // row + 9
    k, v = (torch.empty(N, 16, 2, d, dtype=c.dt, device="cuda") for _ in range(2))
    small = c.k.shape[0]
    k[N - small:], v[N - small:] = a["k_pages"], a["v_pages"]
    table = torch.from_numpy(c.table).cuda()
    table[0, :5] += N - small
    out, lse = tv.tree_verify_attn_paged(**dict(a, k_pages=k, v_pages=v, page_table=table))
    torch.cuda.synchronize()
    check_attn(out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_longest_prefix(dtype):
    """2^31 - 1 rows, all of one page: q = 0 gives every key the weight 1, V = 1 the output 1.  A CTA's sums are
    integers below 2^24, hence exact; the merge rounds each of at most 592 pieces a few times (2^-24 each)."""
    import tree_verification_verify_b200 as tv
    from paged_util import DT
    P, d = 65536, 64
    k = torch.randn(1, P, 1, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    v = torch.ones_like(k)
    one = torch.ones(1, 1, 1, d, dtype=DT[dtype], device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st = i32([0])
    out, lse = tv.tree_verify_attn_paged(one * 0, k, v, torch.zeros(1, 32768, dtype=torch.int32, device="cuda"),
                                         i32([2 ** 31 - 1]), one, one, i32([[-1]]), dev_status=st)
    assert int(st.item()) == 0
    assert (out.double() - 1).abs().max().item() <= 600 * 4 * 2.0 ** -24
    assert abs(lse.double().item() - np.log(2.0 ** 31)) <= (600 * 4 + 64) * 2.0 ** -24


def test_streams_and_graphs_have_scratch_of_their_own():
    """Two captured graphs replayed at the same time on two streams, with eager calls between."""
    import tree_verification_verify_b200 as tv
    cases = [AttnCase(1, 2, 8, 2, 128, 16, [n], "bf16", seed=n) for n in (5000, 4100)]
    args = [c.cuda() for c in cases]
    want = [tv.tree_verify_attn_paged(**a)[0].clone() for a in args]
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tv.tree_verify_attn_paged(**a)[0])
        graphs.append(g)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for i in range(2):
            outs[i].zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
        e = tv.tree_verify_attn_paged(**args[0], stream=s[2])[0]
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(e, want[0])


def test_the_shapes_the_tensor_cores_take():
    import tree_verification_verify_b200 as tv
    for kw, path in ((dict(d=128, P=16, dtype="bf16"), 1), (dict(d=64, P=5, dtype="bf16"), 1),
                     (dict(d=128, P=16, dtype="fp32"), 0), (dict(d=32, P=16, dtype="bf16"), 0)):
        c = AttnCase(1, 2, 4, 1, kw["d"], kw["P"], [20], kw["dtype"])
        a = c.cuda()
        p = tv.paged.AttnPagedArgs(dtype=int(kw["dtype"] == "bf16"), B=1, T=2, Hq=4, Hkv=1, d=kw["d"],
                                   num_pages=a["k_pages"].shape[0], page_size=kw["P"], max_pages=2)
        for f, x in (("q", "q"), ("k_pages", "k_pages"), ("v_pages", "v_pages"), ("page_table", "page_table"),
                     ("prefix_len", "prefix_len"), ("k_tree", "k_tree"), ("v_tree", "v_tree"), ("parent", "parent"),
                     ("out", "q")):
            setattr(p, f, a[x].data_ptr())
        d = kw["d"]
        p.q_sb, p.q_st, p.q_sh, p.o_sb, p.o_st, p.o_sh = (8 * d, 4 * d, d) * 2
        p.kv_sp, p.kv_sr, p.kv_sh, p.kt_sb, p.kt_st, p.kt_sh = kw["P"] * d, d, d, 2 * d, d, d
        assert tv.lib().tv_attn_paged_path(ctypes.byref(p)) == path, kw


def test_refusals():
    import tree_verification_verify_b200 as tv
    c = AttnCase(2, 3, 4, 2, 64, 16, [20, 5], "bf16")
    a = c.cuda()
    for bad in (dict(page_table=a["page_table"].long()), dict(page_table=a["page_table"][:1]),
                dict(prefix_len=a["prefix_len"][:1]), dict(k_tree=a["k_tree"][:, :2]), dict(q=a["q"].half()),
                dict(v_pages=a["v_pages"][:, :8]), dict(k_pages=a["k_pages"].float()),
                dict(out=torch.empty(2, 3, 4, 32, dtype=c.dt, device="cuda")),
                dict(lse=torch.empty(2, 3, 4, dtype=torch.float64, device="cuda")),
                dict(parent=a["parent"][:, :2]), dict(scale=float("inf")), dict(prefix_len=a["prefix_len"].cpu())):
        with pytest.raises(tv.TVError):
            tv.tree_verify_attn_paged(**dict(a, **bad))
