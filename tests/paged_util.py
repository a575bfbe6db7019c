"""Inputs of the paged parity tests, and the error bound of the attention.

The bound, element by element.  With u = 2^-24 (half a step of fp32,
relative) and p the exact weights of a row:
* a score is a d-term fp32 dot product times the scale: its error is at most
  e_s = (d + 2) u scale sum_i |q_i k_i|, largest over the row's keys; a weight
  is exp of it, so its relative error is at most e_s plus e_x, the error of
  the exponential and of its argument's rounding: the kernels' ex2.approx /
  expf are within 2^-21 relative, and the argument, at most |s| + |max| in
  log2 units, is rounded once (2 u |s|_max); numerator and denominator both
  carry it: 2 (e_s + e_x);
* the sums over n keys and the merges of at most n pieces round each term at
  most n + 8 times: (n + 8) u;
* with bf16 the weights that meet V are rounded once more, 2^-8;
* all of these act on terms p_j v_j, so they are relative to
  A = sum_j p_j |v_j|; the output's own rounding is relative to |o|.
lse: e_s + e_x + (n + 8) u, plus u |lse| and one rounding of log2 / ln 2.
"""

import numpy as np
import torch

from oracle import paged as op
from synth import tree_bfs_fanout, tree_chain, tree_random_recursive, tree_star

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def trees(kind, B, T, seed=0):
    g = torch.Generator().manual_seed(seed)
    f = dict(chain=lambda: tree_chain(T), star=lambda: tree_star(T), random=lambda: tree_random_recursive(T, g),
             bfs=lambda: tree_bfs_fanout(T, (4, 3, 2)))[kind]
    return np.stack([f() for _ in range(B)]).astype(np.int32)


def tables(rows, P, W, N, seed=0):
    """Distinct pages in random order; entries past a sequence's rows hold out-of-range values."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(N)
    t = rng.choice([-1, -7, N, 2 ** 30], size=(len(rows), W)).astype(np.int32)
    at = 0
    for b, n in enumerate(rows):
        k = -(-n // P)
        t[b, :k] = order[at:at + k]
        at += k
    return t


class AttnCase:
    def __init__(self, B, T, Hq, Hkv, d, P, lens, dtype, tree="random", n_nodes=None, seed=0, spare=2, layout="nphd",
                 poison=True):
        self.lens = list(lens)
        N = sum(-(-n // P) for n in lens) + spare
        W = max(-(-n // P) for n in lens) + 1
        g = torch.Generator().manual_seed(1000 + seed)
        dt = DT[dtype]
        r = lambda *s: torch.randn(*s, generator=g).to(dt)
        self.dt, self.P = dt, P
        self.q, self.kt, self.vt = r(B, T, Hq, d), r(B, T, Hkv, d), r(B, T, Hkv, d)
        shape, perm = dict(nphd=((N, P, Hkv, d), (0, 1, 2, 3)), nhpd=((N, Hkv, P, d), (0, 2, 1, 3)))[layout]
        self.k, self.v = (r(*shape).permute(*perm) for _ in range(2))
        self.table = tables(lens, P, W, N, seed)
        self.parent = trees(tree, B, T, seed)
        self.n_nodes = None if n_nodes is None else np.asarray(n_nodes, np.int32)
        if poison:
            # rows that belong to no sequence hold NaN
            live = torch.zeros(N, P, dtype=torch.bool)
            for b, n in enumerate(lens):
                for j in range(n):
                    live[self.table[b, j // P], j % P] = True
            self.k[~live] = float("nan")
            self.v[~live] = float("nan")

    def oracle(self, **kw):
        clean = lambda x: torch.nan_to_num(x.float(), nan=0.0).to(x.dtype)
        nn = self.n_nodes
        ref = op.tree_verify_attn_paged(self.q, clean(self.k), clean(self.v), self.table, self.lens, self.kt, self.vt,
                                        self.parent, n_nodes=nn, **kw)
        mag = op.tree_verify_attn_paged(self.q, clean(self.k), clean(self.v).abs(), self.table, self.lens, self.kt,
                                        self.vt.abs(), self.parent, n_nodes=nn, **kw)
        # the largest sum_i |q_i k_i| of a row, over all keys of its sequence
        B, T, Hq, d = self.q.shape
        Hkv = self.kt.shape[2]
        dots = np.zeros((B, T, Hq))
        q = self.q.double().abs().numpy()
        for b in range(B):
            keys = np.concatenate([op.gather(clean(self.k).double().numpy(), self.table[b], self.lens[b]),
                                   self.kt[b].double().numpy()])
            for h in range(Hq):
                dots[b, :, h] = (q[b, :, h] @ np.abs(keys[:, h // (Hq // Hkv)]).T).max(-1)
        scale = kw.get("scale") or d ** -0.5
        n = np.array([x + T for x in self.lens])[:, None, None]
        e_s = (d + 2) * U * scale * dots
        e_x = 2.0 ** -21 + 2 * U * 1.45 * scale * dots
        sums = (n + 8) * U
        bf = self.dt == torch.bfloat16
        rel = 2 * (e_s + e_x) + sums + (2.0 ** -8 if bf else 0.0)
        ref["bound"] = rel[..., None] * mag["out"] + (2.0 ** -8 if bf else U) * (1 + rel[..., None]) * mag["out"]
        ref["lse_bound"] = e_s + e_x + sums + 4 * U * (1 + np.abs(ref["lse"]))
        return ref

    def cuda(self):
        c = lambda x: x.cuda() if isinstance(x, torch.Tensor) else torch.from_numpy(np.asarray(x, np.int32)).cuda()
        strided = lambda x: x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) if not x.is_contiguous() \
            else x.cuda()
        return dict(q=c(self.q), k_pages=strided(self.k), v_pages=strided(self.v), page_table=c(self.table),
                    prefix_len=c(self.lens), k_tree=c(self.kt), v_tree=c(self.vt), parent=c(self.parent),
                    n_nodes=None if self.n_nodes is None else c(self.n_nodes))


def check_attn(out, lse, ref, poison=None):
    o, z = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
    ok = ref["valid"] & ref["written"]
    assert np.all(np.abs(o - ref["out"])[ok] <= ref["bound"][ok]), \
        float(np.nanmax((np.abs(o - ref["out"])[ok] / np.maximum(ref["bound"][ok], 1e-300))))
    bad = ref["written"] & ~ref["valid"]
    assert np.all(np.isnan(o[bad]))
    if z is not None:
        empty = np.isneginf(ref["lse"]) & ok[..., None]
        assert np.all(np.isneginf(z[empty]))
        full = ok[..., None] & ~empty
        assert np.all(np.abs(z - ref["lse"])[full] <= ref["lse_bound"][full])
        assert np.all(np.isnan(z[bad]))
    if poison is not None:
        assert np.all(o[~ref["written"]] == poison)
