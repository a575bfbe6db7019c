"""Verification over a paged cache, fp64 oracle -- TEST INFRASTRUCTURE ONLY.

The cache is a pool of pages [num_pages][P][Hkv][d]; row j of sequence b is
row j % P of page table[b][j // P].  Written from that definition: every
call gathers or scatters rows one by one, in plain loops.

tree_verify_attn_paged   the rows gathered into a contiguous cache, then the
                         contiguous oracle.
tree_accept_probs        the walk of accept.tree_accept from given
                         probabilities and uniforms, residual after residual.
tree_commit_kv_paged     the accepted rows written one by one.
tree_pages_update        pages shared, kept, or copied by the rule that a
                         sequence may write only where no other new sequence
                         and no pin holds the page; fresh pages are the
                         lowest free ones in (sequence, position) order.
tree_pages_compact       the k-th used unpinned page at or past n_used moves
                         to the k-th free page below it.
"""

from __future__ import annotations

import numpy as np

from .accept import inverse_cdf
from .attention import _f64, _i64, tree_verify_attn

ST_BAD_PARENT = 1
ST_BAD_TOKEN = 2
ST_NONFINITE = 4
ST_BAD_ROW = 8
ST_BAD_LEN = 16
ST_BAD_PAGE = 64
ST_NO_PAGES = 128


def gather(pages, table, n):
    """Rows 0 .. n-1 of the sequence with page-table row `table`."""
    P = pages.shape[1]
    return np.array([pages[int(table[j // P]), j % P] for j in range(n)]).reshape(n, *pages.shape[2:])


def tree_verify_attn_paged(q, k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, parent, n_nodes=None,
                           scale=0.0, prefix_only=False, rows=None):
    """The dict of attention.tree_verify_attn; a sequence with a bad page in use has no valid rows."""
    K, V = _f64(k_pages), _f64(v_pages)
    table, L = _i64(page_table), _i64(prefix_len)
    N, P, Hkv, d = K.shape
    B, W = table.shape
    T = _i64(parent).shape[1]
    nn = _i64(n_nodes) if n_nodes is not None else np.full(B, T, dtype=np.int64)
    cap = W * P
    good = [int(x) if 0 <= x <= cap else 0 for x in L]
    bad_page = [any(not 0 <= table[b, i] < N for i in range(-(-good[b] // P))) for b in range(B)]
    # the contiguous oracle's bound on prefix_len is the width of its cache
    Lmax = max(good, default=0)
    kc, vc = np.zeros((B, Lmax, Hkv, d)), np.zeros((B, Lmax, Hkv, d))
    lens = np.array([x if 0 <= x <= cap else -1 for x in L])
    for b in range(B):
        if bad_page[b]:
            lens[b] = 0
        elif good[b]:
            kc[b, :good[b]], vc[b, :good[b]] = gather(K, table[b], good[b]), gather(V, table[b], good[b])
    ref = tree_verify_attn(q, kc, vc, lens, k_tree, v_tree, parent, n_nodes=nn, scale=scale, prefix_only=prefix_only,
                           rows=rows)
    for b in range(B):
        if bad_page[b] and 0 < nn[b] <= T:
            ref["status"] |= ST_BAD_PAGE
            ref["valid"][b] = False
            ref["out"][b] = np.nan
            ref["lse"][b] = np.nan
    return ref


def tree_accept_probs(target_probs, draft_probs, draft_tokens, parent, u_child, u_sample, n_nodes=None):
    """SPECSAMPLE with draft_probs, else SPECEXEC.  min_margin as in accept.tree_accept."""
    B, T, V = tuple(target_probs.shape)
    tok, par = _i64(draft_tokens), _i64(parent)
    nn = _i64(n_nodes) if n_nodes is not None else np.full(B, T, dtype=np.int64)
    uc = _f64(u_child) if u_child is not None else None
    us = _f64(u_sample)
    n_acc = np.zeros(B, dtype=np.int64)
    acc = np.full((B, T), -1, dtype=np.int64)
    out = np.full((B, T + 1), -1, dtype=np.int64)
    margin = np.full(B, np.inf)
    status = 0

    def valid(x):
        return np.all(np.isfinite(x)) and np.all(x >= 0)

    for b in range(B):
        n = int(nn[b])
        if n < 0 or n > T:
            status |= ST_BAD_LEN
            continue
        if n == 0:
            continue
        kids = {}
        if par[b, 0] != -1:
            status |= ST_BAD_PARENT
        for j in range(1, n):
            if not 0 <= tok[b, j] < V:
                status |= ST_BAD_TOKEN
            if not 0 <= par[b, j] < j:
                status |= ST_BAD_PARENT
            else:
                kids.setdefault(int(par[b, j]), []).append(j)
        c, path, bonus = 0, [], -1
        while True:
            nxt, fault = None, False
            ch = [j for j in kids.get(c, []) if 0 <= tok[b, j] < V]
            p = _f64(target_probs[b, c])
            r = p.copy()
            whole = False                       # the row has been read as a whole
            if draft_probs is not None and ch:
                q = _f64(draft_probs[b, c])
                for j in ch:
                    x, u = int(tok[b, j]), uc[b, j]
                    if not (valid(p[x]) and valid(q[x]) and 0 <= u < 1):
                        fault = True
                        break
                    ratio = r[x] / q[x] if q[x] > 0 else (np.inf if r[x] > 0 else 0.0)
                    if np.isfinite(ratio):
                        margin[b] = min(margin[b], abs(u - ratio))
                    if u < ratio:
                        nxt = j
                        break
                    if not (valid(p) and valid(q)):
                        fault = True
                        break
                    rest = np.maximum(r - q, 0.0)
                    if rest.sum() > 0:
                        r = rest / rest.sum()
            if fault:
                status |= ST_NONFINITE
                break
            if nxt is None:
                u = us[b, c]
                if not (0 <= u < 1) or not valid(p) or not r.sum() > 0:
                    status |= ST_NONFINITE
                    break
                x, mg = inverse_cdf(r, u)
                margin[b] = min(margin[b], mg)
                if draft_probs is None:
                    nxt = next((j for j in ch if tok[b, j] == x), None)
                if nxt is None:
                    bonus = x
                    break
            path.append(nxt)
            c = nxt
        n_acc[b] = len(path)
        acc[b, :len(path)] = path
        out[b, :len(path)] = [int(tok[b, j]) for j in path]
        out[b, len(path)] = bonus
    return dict(n_accepted=n_acc, accepted_nodes=acc, out_tokens=out, min_margin=margin, status=status)


def tree_commit_kv_paged(k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, n_accepted, accepted_nodes):
    """Pools [layers][num_pages][P][Hkv][d], trees [layers][B][T][Hkv][d]."""
    K, V, KT, VT = (_f64(x).copy() for x in (k_pages, v_pages, k_tree, v_tree))
    table, L, n_acc, acc = _i64(page_table), _i64(prefix_len).copy(), _i64(n_accepted), _i64(accepted_nodes)
    N, P = K.shape[1:3]
    B, T = KT.shape[1:3]
    status = 0
    for b in range(B):
        n, Lb = int(n_acc[b]), int(L[b])
        if n < 0 or n > T - 1 or Lb < 0 or Lb + n + 1 > min(table.shape[1] * P, 2 ** 31 - 1):
            status |= ST_BAD_LEN
            continue
        rows = [0] + [int(acc[b, r]) for r in range(n)]
        places = [(int(table[b, (Lb + r) // P]), (Lb + r) % P) for r in range(n + 1)]
        bad = 0
        if any(x < 1 or x >= T for x in rows[1:]) or any(rows[r] <= rows[r - 1] for r in range(1, n + 1)):
            bad |= ST_BAD_ROW
        if any(not 0 <= page < N for page, _ in places):
            bad |= ST_BAD_PAGE
        if bad:
            status |= bad
            continue
        for x, (page, row) in zip(rows, places):
            K[:, page, row], V[:, page, row] = KT[:, b, x], VT[:, b, x]
        L[b] = Lb + n + 1
    return dict(k_pages=K, v_pages=V, prefix_len=L, status=status)


def tree_pages_update(k_pages, v_pages, page_table, source, keep, grow, max_pages, pinned=None):
    """Pools [layers][num_pages][P][Hkv][d].  Also returns `writable`: per new sequence the (page, row) places of its
    rows from keep[b] on."""
    K, V = _f64(k_pages).copy(), _f64(v_pages).copy()
    table, src, keep, grow = _i64(page_table), _i64(source), _i64(keep).copy(), _i64(grow)
    N, P = K.shape[1:3]
    B_in, W_in = table.shape
    B = len(src)
    held_outside = set() if pinned is None else {i for i, x in enumerate(_i64(pinned)) if x != 0}
    status, live = 0, []
    for b in range(B):
        bits = 0
        if src[b] == -1:
            keep[b] = 0
        elif not 0 <= src[b] < B_in:
            bits |= ST_BAD_ROW
        if keep[b] < 0 or grow[b] < 0 or keep[b] > W_in * P or keep[b] + grow[b] > max_pages * P:
            bits |= ST_BAD_LEN
        if not bits and any(not 0 <= table[src[b], i] < N for i in range(-(-int(keep[b]) // P))):
            bits |= ST_BAD_PAGE
        status |= bits
        if not bits:
            live.append(b)
    readers, writers = set(held_outside), {}
    for b in live:
        for i in range(-(-int(keep[b]) // P)):
            page = int(table[src[b], i])
            if grow[b] > 0 and (i + 1) * P > keep[b]:
                writers.setdefault(page, []).append(b)
            else:
                readers.add(page)
    free = sorted(set(range(N)) - readers - set(writers))
    out = np.full((B, max_pages), -1, dtype=np.int64)
    copies, need = [], 0
    for b in live:
        for i in range(-(-int(keep[b] + grow[b]) // P)):
            fresh = True
            if i * P < keep[b]:
                page = int(table[src[b], i])
                partial = grow[b] > 0 and (i + 1) * P > keep[b]
                fresh = partial and (page in readers or writers[page][0] != b)
                if fresh:
                    copies.append((page, need, int(keep[b]) - i * P))
            if fresh:
                page = free[need] if need < len(free) else -1
                need += 1
            out[b, i] = page
    if need > len(free):
        out[:] = -1
        return dict(page_table=out, n_free=len(free) - need, k_pages=K, v_pages=V, status=status | ST_NO_PAGES)
    for page, k, rows in copies:
        K[:, free[k], :rows], V[:, free[k], :rows] = K[:, page, :rows], V[:, page, :rows]
    return dict(page_table=out, n_free=len(free) - need, k_pages=K, v_pages=V, status=status)


def tree_pages_compact(k_pages, v_pages, page_table, length, pinned=None):
    K, V = _f64(k_pages).copy(), _f64(v_pages).copy()
    table, L = _i64(page_table).copy(), _i64(length)
    N, P = K.shape[1:3]
    B, W = table.shape
    fixed = set() if pinned is None else {i for i, x in enumerate(_i64(pinned)) if x != 0}
    status, used = 0, set()
    held = []
    for b in range(B):
        if not 0 <= L[b] <= W * P:
            status |= ST_BAD_LEN
        held.append(-(-int(np.clip(L[b], 0, W * P)) // P))
        for i in range(held[b]):
            if 0 <= table[b, i] < N:
                used.add(int(table[b, i]))
            else:
                status |= ST_BAD_PAGE
    total = len(used | fixed)
    holes = [x for x in range(total) if x not in used and x not in fixed]
    movers = [x for x in range(total, N) if x in used and x not in fixed]
    to = dict(zip(movers, holes))
    for a, z in to.items():
        K[:, z], V[:, z] = K[:, a], V[:, a]
    for b in range(B):
        for i in range(W):
            table[b, i] = to.get(int(table[b, i]), table[b, i]) if i < held[b] else -1
    return dict(page_table=table, n_used=total, k_pages=K, v_pages=V, status=status)
