"""Pins of the paged oracle by routes that share none of its code, and the
paged calls' refusals (host-side checks; nothing is launched)."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged as op
from oracle.accept import tree_accept, softmax_t
from oracle.attention import tree_verify_attn
from oracle.commit import tree_commit_kv
from oracle.philox import uniform, TAG_CHILD, TAG_RESIDUAL, TAG_SPECEXEC
from synth import accept_case, tree_random_recursive

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _tables(rows, P, N, W, rng):
    order = rng.permutation(N)
    t, at = np.full((len(rows), W), -1), 0
    for b, n in enumerate(rows):
        k = -(-n // P)
        t[b, :k] = order[at:at + k]
        at += k
    return t


@pytest.mark.parametrize("P", [1, 3, 8])
def test_attention_through_pages_is_attention_over_the_same_rows(P):
    rng = np.random.default_rng(P)
    B, T, Hq, Hkv, d = 3, 6, 4, 2, 8
    lens = [0, 7, 19]
    W = 22 // P + 1
    table = _tables(lens, P, 40, W, rng)
    kp, vp = rng.normal(size=(2, 40, P, Hkv, d))
    kc, vc = np.zeros((2, B, 20, Hkv, d))
    for b, n in enumerate(lens):
        for j in range(n):
            kc[b, j], vc[b, j] = kp[table[b, j // P], j % P], vp[table[b, j // P], j % P]
    q = rng.normal(size=(B, T, Hq, d))
    kt, vt = rng.normal(size=(2, B, T, Hkv, d))
    par = np.stack([tree_random_recursive(T, torch.Generator().manual_seed(b)) for b in range(B)])
    for only in (False, True):
        a = op.tree_verify_attn_paged(q, kp, vp, table, lens, kt, vt, par, prefix_only=only)
        e = tree_verify_attn(q, kc, vc, np.array(lens), kt, vt, par, prefix_only=only)
        np.testing.assert_allclose(a["out"], e["out"], rtol=0, atol=1e-14)
        np.testing.assert_allclose(a["lse"], e["lse"], rtol=0, atol=1e-14)
        assert a["status"] == e["status"] == 0
    table[2, 1] = 40                                    # one bad page: that sequence alone is lost
    a = op.tree_verify_attn_paged(q, kp, vp, table, lens, kt, vt, par)
    assert a["status"] == op.ST_BAD_PAGE and not a["valid"][2].any() and a["valid"][:2].all()


@pytest.mark.parametrize("mode", ["specsample", "specexec"])
def test_given_numbers_reproduce_the_philox_walk(mode):
    """With the softmax as probabilities and Philox's numbers as the given ones, the walk is tree_accept's."""
    par = tree_random_recursive(24, torch.Generator().manual_seed(3))
    c = accept_case(6, 24, 60, par, 0.7, sigma=2.0, seed=5, correlated=True, mode=mode,
                    child_rule="sample" if mode == "specsample" else "top", with_q=mode == "specsample")
    ref = tree_accept(c.target_logits, c.draft_probs, c.draft_tokens, c.parent, mode=mode, temperature=0.7, seed=9,
                      step=2)
    tau = float(np.float32(0.7))
    p = np.stack([[softmax_t(c.target_logits[b, t].double().numpy(), tau) for t in range(24)] for b in range(6)])
    parent = c.parent.numpy()
    uc, us = np.zeros((6, 24)), np.zeros((6, 24))
    for b in range(6):
        for j in range(24):
            k = sum(parent[b, i] == parent[b, j] for i in range(1, j)) if j else 0
            uc[b, j] = uniform(9, 2, b, parent[b, j], k, TAG_CHILD) if j else 0.0
            us[b, j] = uniform(9, 2, b, j, 0, TAG_RESIDUAL if mode == "specsample" else TAG_SPECEXEC)
    got = op.tree_accept_probs(p, c.draft_probs if mode == "specsample" else None, c.draft_tokens, c.parent, uc, us)
    assert ref["n_accepted"].sum() > 0
    for k in ("n_accepted", "accepted_nodes", "out_tokens"):
        np.testing.assert_array_equal(got[k], ref[k])


def test_first_token_follows_the_target():
    """Exact over a grid of uniforms: two children drawn from q, their tests and the residual sample together emit
    tokens with the target's probabilities."""
    p, q = np.array([0.5, 0.125, 0.375]), np.array([0.25, 0.5, 0.25])
    par, grid = np.array([[-1, 0, 0]]), 16
    us = (np.arange(grid) + 0.5) / grid
    mass = np.zeros(3)
    for x1 in range(3):
        for x2 in range(3):
            # breakpoints of the tests at 1/16 steps are exact for the first child; the second and the sample
            # are integrated over their exact ratios
            w = q[x1] * q[x2]
            a1 = min(1.0, p[x1] / q[x1])
            mass[x1] += w * a1
            r = np.maximum(p - q, 0)
            r = r / r.sum()
            a2 = min(1.0, r[x2] / q[x2])
            mass[x2] += w * (1 - a1) * a2
            r2 = np.maximum(r - q, 0)
            r2 = r2 / r2.sum() if r2.sum() > 0 else r
            mass += w * (1 - a1) * (1 - a2) * r2
            for u1 in us:
                for u2 in us:
                    got = op.tree_accept_probs(np.tile(p, (1, 3, 1)), np.tile(q, (1, 3, 1)), np.array([[0, x1, x2]]),
                                               par, np.array([[0, u1, u2]]), np.full((1, 3), 0.5))
                    want = [1] if u1 < p[x1] / q[x1] else ([2] if u2 < r[x2] / q[x2] else [])
                    assert list(got["accepted_nodes"][0, :got["n_accepted"][0]]) == want
    np.testing.assert_allclose(mass, p, atol=1e-12)


def test_commit_then_gather_is_the_contiguous_commit():
    rng = np.random.default_rng(0)
    B, T, P, W, N = 3, 5, 4, 6, 20
    lens, n_acc = np.array([0, 3, 14]), np.array([4, 0, 2])
    acc = np.array([[1, 2, 3, 4, -1], [-1] * 5, [2, 4, -1, -1, -1]])
    table = _tables([24, 24, 24], P, N, W, rng)
    kp, vp = rng.normal(size=(2, 2, N, P, 1, 3))
    kt, vt = rng.normal(size=(2, 2, B, T, 1, 3))
    got = op.tree_commit_kv_paged(kp, vp, table, lens, kt, vt, n_acc, acc)
    for l in range(2):
        kc = np.stack([op.gather(kp[l], table[b], 24) for b in range(B)])
        vc = np.stack([op.gather(vp[l], table[b], 24) for b in range(B)])
        ref = tree_commit_kv(kc, vc, lens, kt[l], vt[l], n_acc, acc)
        for b in range(B):
            np.testing.assert_array_equal(op.gather(got["k_pages"][l], table[b], 24), ref["k_cache"][b])
            np.testing.assert_array_equal(op.gather(got["v_pages"][l], table[b], 24), ref["v_cache"][b])
        np.testing.assert_array_equal(got["prefix_len"], ref["prefix_len"])
    assert got["status"] == 0


@pytest.mark.parametrize("seed", range(20))
def test_update_keeps_rows_and_gives_private_room(seed):
    """What an update is for, whatever its rule: every kept row reads as before, every row of room lies in a page that
    no other sequence, no pin and no other row of the sequence holds, and the free pages are counted."""
    rng = np.random.default_rng(seed)
    P, W, N, B_in, B = int(rng.integers(1, 6)), 8, 60, 4, 6
    lens = rng.integers(0, W * P // 2, B_in)
    table = _tables(lens, P, N, W, rng)
    kp, vp = rng.normal(size=(2, 2, N, P, 1, 2))
    src = rng.integers(-1, B_in, B)
    keep = np.array([0 if s < 0 else rng.integers(0, lens[s] + 1) for s in src])
    grow = rng.integers(0, 4, B) * rng.integers(0, 2, B)
    pinned = rng.random(N) < 0.1
    got = op.tree_pages_update(kp, vp, table, src, keep, grow, W, pinned)
    assert got["status"] == 0
    new = got["page_table"]
    holders = {}
    for b in range(B):
        np.testing.assert_array_equal(op.gather(got["k_pages"][0], new[b], keep[b]),
                                      op.gather(kp[0], table[src[b]], keep[b]))
        np.testing.assert_array_equal(op.gather(got["v_pages"][1], new[b], keep[b]),
                                      op.gather(vp[1], table[src[b]], keep[b]))
        k = -(-(keep[b] + grow[b]) // P)
        assert (new[b, :k] >= 0).all() and (new[b, k:] == -1).all()
        for i in range(k):
            holders.setdefault(new[b, i], []).append((b, i))
    for b in range(B):
        for j in range(keep[b], keep[b] + grow[b]):
            page = new[b, j // P]
            assert holders[page] == [(b, j // P)] and not pinned[page]
    assert got["n_free"] == sum(1 for x in range(N) if x not in holders and not pinned[x])


@pytest.mark.parametrize("seed", range(20))
def test_compaction_keeps_rows_and_packs(seed):
    rng = np.random.default_rng(seed)
    P, W, N, B = int(rng.integers(1, 6)), 8, 50, 4
    lens = rng.integers(0, W * P + 1, B)
    table = _tables(lens, P, N, W, rng)
    table[3], lens[3] = table[2], lens[2] // 2           # a shared prefix
    pinned = rng.random(N) < (0.15 if seed % 2 else 0.0)
    kp, vp = rng.normal(size=(2, 1, N, P, 1, 2))
    got = op.tree_pages_compact(kp, vp, table, lens, pinned)
    used = set()
    for b in range(B):
        np.testing.assert_array_equal(op.gather(got["k_pages"][0], got["page_table"][b], lens[b]),
                                      op.gather(kp[0], table[b], lens[b]))
        k = -(-lens[b] // P)
        used |= set(got["page_table"][b, :k])
        assert (got["page_table"][b, k:] == -1).all()
    for x in range(N):
        if pinned[x]:
            np.testing.assert_array_equal(got["k_pages"][0, x], kp[0, x])
    assert all(x < got["n_used"] or pinned[x] for x in used)
    assert got["n_used"] == len(used | {x for x in range(N) if pinned[x]})


# ------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def tv():
    from tree_verification_verify_b200 import build
    build.build()
    import tree_verification_verify_b200 as tv
    return tv


def test_paged_struct_layouts_match_the_header(tv, tmp_path):
    P = tv.paged
    structs = {"tv_attn_paged_args": P.AttnPagedArgs, "tv_accept_probs_args": P.AcceptProbsArgs,
               "tv_commit_paged_args": P.CommitPagedArgs, "tv_pages_update_args": P.PagesUpdateArgs,
               "tv_pages_compact_args": P.PagesCompactArgs}
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "tree_verify.h"', "int main(void){"]
    for c, py in structs.items():
        src.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        src += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    (tmp_path / "a.c").write_text("\n".join(src + ["return 0;}"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")],
                   check=True)
    got = dict(((a, b), int(v)) for a, b, v in
               (x.split() for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True,
                                                  check=True).stdout.splitlines()))
    for c, py in structs.items():
        assert got[c, "size"] == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert got[c, f] == getattr(py, f).offset, (c, f)


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def _attn(tv, **kw):
    a = tv.paged.AttnPagedArgs(dtype=1, B=2, T=3, Hq=8, Hkv=2, d=64, num_pages=4, page_size=16, max_pages=2)
    for f in ("q", "k_pages", "v_pages", "page_table", "prefix_len", "k_tree", "v_tree", "parent", "out"):
        setattr(a, f, 4096)
    for f, v in kw.items():
        setattr(a, f, v)
    return tv.lib().tree_verify_attn_paged(ctypes.byref(a), None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(), WORKSPACE), (dict(B=0), OK), (dict(T=0), OK), (dict(dtype=2), INVALID), (dict(B=-1), INVALID),
    (dict(Hq=9), INVALID), (dict(Hkv=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=65537), UNSUPPORTED),
    (dict(num_pages=-1), INVALID), (dict(num_pages=(1 << 24) + 1), UNSUPPORTED), (dict(max_pages=-1), INVALID),
    (dict(d=48), UNSUPPORTED), (dict(Hq=130), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(scale=-1.0), INVALID), (dict(prefix_only=2), INVALID), (dict(page_table=None), INVALID),
    (dict(k_pages=None), INVALID), (dict(q=None), INVALID), (dict(out=4097), INVALID), (dict(v_tree=4097), INVALID)])
def test_attn_paged_refusals(tv, kw, want):
    assert _attn(tv, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), OK), (dict(B=-1), INVALID), (dict(V=0), INVALID), (dict(mode=1), INVALID), (dict(mode=4), INVALID),
    (dict(T=4097), UNSUPPORTED), (dict(V=(1 << 30) + 1), UNSUPPORTED), (dict(B=16385), UNSUPPORTED),
    (dict(u_sample=None), INVALID), (dict(u_child=None), INVALID), (dict(draft_probs=None, mode=2), INVALID),
    (dict(tp_st=99), INVALID), (dict(dp_st=99), INVALID), (dict(out_tokens=None), INVALID),
    (dict(target_probs=4098), INVALID)])
def test_accept_probs_refusals(tv, kw, want):
    a = tv.paged.AcceptProbsArgs(B=2, T=3, V=100, tp_st=100, dp_st=100)
    for f in ("target_probs", "draft_probs", "draft_tokens", "parent", "u_child", "u_sample", "n_accepted",
              "accepted_nodes", "out_tokens"):
        setattr(a, f, 4096)
    for f, v in kw.items():
        setattr(a, f, v)
    assert tv.lib().tree_accept_probs(ctypes.byref(a), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), WORKSPACE), (dict(B=0), OK), (dict(T=0), INVALID), (dict(layers=0), INVALID), (dict(d=1025), UNSUPPORTED),
    (dict(B=16385), UNSUPPORTED), (dict(prefix_len_out=None), INVALID), (dict(accepted_nodes=None), INVALID),
    (dict(page_table=None), INVALID), (dict(k_tree=4098), INVALID), (dict(page_size=0), INVALID)])
def test_commit_paged_refusals(tv, kw, want):
    a = tv.paged.CommitPagedArgs(dtype=0, layers=1, B=2, T=3, Hkv=2, d=64, num_pages=4, page_size=16, max_pages=2)
    for f in ("k_pages", "v_pages", "page_table", "prefix_len", "prefix_len_out", "k_tree", "v_tree", "n_accepted",
              "accepted_nodes"):
        setattr(a, f, 4096)
    for f, v in kw.items():
        setattr(a, f, v)
    assert tv.lib().tree_commit_kv_paged(ctypes.byref(a), None, 0, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), WORKSPACE), (dict(B=-1), INVALID), (dict(source=None), INVALID), (dict(page_table_out=None), INVALID),
    (dict(page_table_out=8192), INVALID), (dict(page_table_out=8192 + 4 * 7), INVALID), (dict(po_sb=3), INVALID),
    (dict(pt_sb=3), INVALID), (dict(num_pages=(1 << 24) + 1), UNSUPPORTED), (dict(B_in=16385), UNSUPPORTED),
    (dict(k_pages=None), INVALID), (dict(layers=-1), INVALID),
    (dict(B=16384, max_pages=1 << 17, po_sb=1 << 17), UNSUPPORTED),
    (dict(page_size=65536, Hkv=64, d=512), UNSUPPORTED), (dict(page_size=65535, Hkv=32, d=1024), WORKSPACE)])
def test_pages_update_refusals(tv, kw, want):
    a = tv.paged.PagesUpdateArgs(dtype=0, layers=1, B_in=2, B=2, Hkv=2, d=64, num_pages=8, page_size=16, max_pages_in=4,
                                 max_pages=4, page_table=8192, pt_sb=4, page_table_out=16384, po_sb=4)
    for f in ("k_pages", "v_pages", "source", "keep", "grow"):
        setattr(a, f, 4096)
    for f, v in kw.items():
        setattr(a, f, v)
    assert tv.lib().tree_pages_update(ctypes.byref(a), None, 0, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(), WORKSPACE), (dict(page_table_out=8192), WORKSPACE), (dict(page_table_out=8192 + 4), INVALID),
    (dict(page_table_out=8192, po_sb=5), INVALID), (dict(length=None), INVALID), (dict(dtype=7), INVALID),
    (dict(d=0), INVALID), (dict(d=1025), UNSUPPORTED)])
def test_pages_compact_refusals(tv, kw, want):
    a = tv.paged.PagesCompactArgs(dtype=0, layers=1, B=2, Hkv=2, d=64, num_pages=8, page_size=16, max_pages=4,
                                  page_table=8192, pt_sb=4, page_table_out=16384, po_sb=4)
    for f in ("k_pages", "v_pages", "length"):
        setattr(a, f, 4096)
    for f, v in kw.items():
        setattr(a, f, v)
    assert tv.lib().tree_pages_compact(ctypes.byref(a), None, 0, None) == want


def test_paged_calls_refuse_host_tensors(tv):
    k = torch.zeros(4, 16, 1, 64)
    t = torch.zeros(1, 2, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    q, kt, par = torch.zeros(1, 2, 4, 64), torch.zeros(1, 2, 1, 64), torch.tensor([[-1, 0]], dtype=torch.int32)
    u = torch.zeros(1, 2, dtype=torch.float64)
    for call in (lambda: tv.tree_verify_attn_paged(q, k, k, t, n, kt, kt, par),
                 lambda: tv.tree_accept_probs(torch.ones(1, 2, 8), t, par, u, u),
                 lambda: tv.tree_commit_kv_paged(k, k, t, n, kt, kt, n, t),
                 lambda: tv.tree_pages_update(k, k, t, n, n, n),
                 lambda: tv.tree_pages_compact(k, k, t, n)):
        with pytest.raises(tv.TVError):
            call()
