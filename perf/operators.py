"""What is measured of verification over a paged K/V cache.

Five operators that make up one verification step of a server whose cache
lives in pages: tree attention through a page table, acceptance from given
probabilities and given random numbers, the commit of the accepted rows
into their pages, the update of the page tables from step to step (fork,
roll back, free, grow, copy on write) and the compaction of the pool.

`own` False computes them in plain torch operations; `own` True makes the
framework's calls on the same inputs.  A case's sequence lengths and tree
shapes follow from the case alone, everything else from the seed.
"""

import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user, plain single-token decoding on a short context: latency alone
        dict(name="attn_one_token", op="attn", B=1, T=1, Hq=32, Hkv=8, d=128, P=16, lo=700, hi=700,
             dtype="bf16", tree="chain", ragged=False),
        # a server's batch: 16-node trees on prefixes from short to long, small pages
        dict(name="attn_serving_trees", op="attn", B=32, T=16, Hq=64, Hkv=8, d=128, P=16, lo=512, hi=16384,
             dtype="bf16", tree="depth", ragged=True),
        # long documents with a wide tree, large pages
        dict(name="attn_long_trees", op="attn", B=2, T=64, Hq=32, Hkv=8, d=128, P=128, lo=65537, hi=131072,
             dtype="bf16", tree="bfs", ragged=False),
        # full precision, small heads, pages that end inside every tile
        dict(name="attn_fp32_odd_pages", op="attn", B=3, T=15, Hq=4, Hkv=1, d=64, P=5, lo=97, hi=1009,
             dtype="fp32", tree="bfs", ragged=True),
        # one user, a chain of four drafted tokens
        dict(name="accept_chain", op="accept", B=1, T=5, V=32000, mode="specsample", tree="chain", ragged=False),
        # a server's batch of sampled trees over a large vocabulary
        dict(name="accept_trees", op="accept", B=32, T=16, V=152064, mode="specsample", tree="depth", ragged=True),
        # one user, one layer, full precision
        dict(name="commit_one", op="commit", B=1, T=15, layers=1, Hkv=1, d=64, P=5, lo=128, hi=128, dtype="fp32"),
        # a server's batch, the layers of a model in one call
        dict(name="commit_layers", op="commit", B=32, T=16, layers=32, Hkv=8, d=128, P=16, lo=20, hi=150,
             dtype="bf16"),
        # four beams over a small pool, every one from another's prefix
        dict(name="update_beams", op="update", B=4, layers=1, pages=64, W=16, P=16, Hkv=8, d=128, dtype="bf16",
             fan=2, lo=30, hi=200, grow=17),
        # a server's turn: some sequences end, some fork, the rest grow by a tree's rows
        dict(name="update_batch", op="update", B=128, layers=2, pages=1200, W=64, P=64, Hkv=8, d=128, dtype="bf16",
             fan=4, lo=17, hi=900, grow=16),
        # a small pool after a few sequences ended
        dict(name="compact_small", op="compact", B=4, layers=1, pages=96, W=24, P=16, Hkv=8, d=128, dtype="bf16",
             lo=30, hi=200, pinned=False),
        # a large pool, with pages that a prefix store holds
        dict(name="compact_pool", op="compact", B=96, layers=2, pages=3500, W=128, P=16, Hkv=8, d=128, dtype="bf16",
             lo=17, hi=900, pinned=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["attn", "attn", "attn", "accept", "accept", "commit", "update", "compact"])
    if op == "attn":
        while True:
            Hq, Hkv = rng.choice([(32, 8), (64, 8), (8, 8), (28, 4), (4, 1), (40, 8), (16, 1)])
            dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
            hi = _log_int(rng, 1, 131072)
            c = dict(op="attn", B=_log_int(rng, 1, 96), T=_log_int(rng, 1, 96), Hq=Hq, Hkv=Hkv,
                     d=rng.choice([64, 128]), P=rng.choice([1, 5, 16, 16, 24, 32, 64, 128, 256]),
                     lo=rng.choice([0, hi // 7, hi]), hi=hi, dtype=dtype,
                     tree=rng.choice(["chain", "star", "depth", "bfs"]), ragged=rng.random() < 0.5)
            w = work(c)
            if w["bytes"] <= 0.9e9 and w["flops"] <= (2e11 if dtype == "bf16" else 2e10):
                return c
    if op == "accept":
        while True:
            c = dict(op="accept", B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 64), V=_log_int(rng, 250, 152064),
                     mode=rng.choice(["specsample", "specsample", "specexec"]),
                     tree=rng.choice(["chain", "star", "depth", "bfs"]), ragged=rng.random() < 0.5)
            if c["B"] * c["T"] * c["V"] <= 32 * 16 * 152064:
                return c
    if op == "commit":
        while True:
            hi = _log_int(rng, 1, 2000)
            c = dict(op="commit", B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 64), layers=_log_int(rng, 1, 32),
                     Hkv=rng.choice([1, 2, 8]), d=rng.choice([64, 80, 128]), P=rng.choice([1, 5, 16, 24, 64]),
                     lo=rng.choice([0, hi // 3, hi]), hi=hi, dtype=rng.choice(["bf16", "fp32"]))
            rows = sum(_lens(c)) + c["B"] * (c["T"] + c["P"])
            if rows * _row_bytes(c) <= 0.6e9 and work(c)["bytes"] <= 60e6:
                return c
    while True:
        hi = _log_int(rng, 2, 1500)
        B, P = _log_int(rng, 1, 160), rng.choice([1, 8, 16, 24, 64])
        c = dict(op=op, B=B, layers=_log_int(rng, 1, 4), P=P, Hkv=rng.choice([1, 2, 8]), d=rng.choice([64, 128]),
                 dtype=rng.choice(["bf16", "fp32"]), lo=rng.choice([0, hi // 3, hi]), hi=hi)
        if op == "update":
            c["fan"], c["grow"] = _log_int(rng, 1, 8), _log_int(rng, 1, 64)
            c["W"] = -(-(hi + c["grow"]) // P) + rng.randrange(3)
            need = sum(-(-(n + c["grow"]) // P) + 1 for n in _lens(c))
        else:
            c["pinned"] = rng.random() < 0.5
            c["W"] = -(-hi // P) + rng.randrange(3)
            need = sum(-(-n // P) for n in _lens(c))
        c["pages"] = 2 * need + rng.randrange(8, 64)
        if c["pages"] <= 8000 and c["pages"] * P * _row_bytes(c) <= 1.2e9:
            return c


# ------------------------------------------------------- what a case implies

def _lens(c):
    """Prefix lengths: spread over [lo, hi], the first at lo, the last at hi."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    if B == 1:
        return [hi]
    out = [lo + int((hi - lo + 1) * ((0.6180339887498949 * b) % 1.0)) for b in range(B)]
    out[0], out[-1] = lo, hi
    return out


def _trees(c):
    """parent[] of every sequence (node 0 the root) and the node counts."""
    B, T, kind = c["B"], c["T"], c["tree"]
    rng = random.Random(1000 * T + B)
    par, n = [], []
    for b in range(B):
        if kind == "chain":
            p = list(range(-1, T - 1))
        elif kind == "star":
            p = [-1] + [0] * (T - 1)
        elif kind == "bfs":                              # 4, then 3, then 2 children, level by level
            p, depth, k = [-1], [0], 0
            while len(p) < T:
                for _ in range((4, 3, 2)[min(depth[k], 2)]):
                    if len(p) < T:
                        p.append(k)
                        depth.append(depth[k] + 1)
                k += 1
        else:                                            # random, depth at most 6
            p, depth = [-1], [0]
            for i in range(1, T):
                q = rng.choice([j for j in range(i) if depth[j] < 6])
                p.append(q)
                depth.append(depth[q] + 1)
        par.append(p)
        n.append(rng.randint((T + 1) // 2, T) if c["ragged"] else T)
    return par, n


def _row_bytes(c):
    """Bytes of one cache row, K and V, all layers."""
    return 2 * c.get("layers", 1) * c["Hkv"] * c["d"] * _SIZE[c["dtype"]]


def work(case):
    c = case
    if c["op"] == "attn":
        par, n = _trees(c)
        e, keys, pairs = _SIZE[c["dtype"]], 0, 0
        for b, L in enumerate(_lens(c)):
            depth = [0] * c["T"]
            for i in range(1, c["T"]):
                depth[i] = depth[par[b][i]] + 1
            keys += L + n[b]
            pairs += sum(L + depth[i] + 1 for i in range(n[b]))
        rows = sum(n) * c["Hq"]
        table = 4 * sum(-(-L // c["P"]) for L in _lens(c))
        return dict(bytes=keys * _row_bytes(c) + rows * (2 * c["d"] * e + 4) + table, flops=4 * c["d"] * c["Hq"] * pairs)
    if c["op"] == "accept":
        # the row at which each walk stops; sampled trees need the draft's row there too
        k = 2 if c["mode"] == "specsample" and c["T"] > 1 else 1
        return dict(bytes=c["B"] * (4 * c["V"] * k + 16 * c["T"]), flops=2 * k * c["B"] * c["V"])
    if c["op"] == "commit":
        return dict(bytes=2 * _accepted(c)[1] * _row_bytes(c), flops=0)
    lens = _lens(c)
    table = 4 * c["B"] * c["W"]
    if c["op"] == "update":
        source, keep, grow = _turn(c)
        moved, writers = 0, set()
        for s, k, g in zip(source, keep, grow):
            if s >= 0 and g > 0 and k % c["P"]:
                page = (s, k // c["P"])
                shared = any(s2 == s and (k2 // c["P"] > page[1] or (g2 == 0 and -(-k2 // c["P"]) > page[1]))
                             for s2, k2, g2 in zip(source, keep, grow))
                if shared or page in writers:
                    moved += k % c["P"]
                else:
                    writers.add(page)
        return dict(bytes=2 * moved * _row_bytes(c) + 2 * table, flops=0)
    used = sum(-(-n // c["P"]) for n in lens)
    share = max(0.0, 1.0 - used / c["pages"])            # of the used pages, those past the packed end
    return dict(bytes=int(2 * used * share * c["P"] * _row_bytes(c)) + 2 * table, flops=0)


def _accepted(c):
    """Accepted nodes of every sequence, and the rows that are committed."""
    rng = random.Random(7 + c["T"] * 31 + c["B"])
    paths = []
    for b in range(c["B"]):
        n = min(c["T"] - 1, rng.choice([0, 1, 2, 3, 3, 4, 6, c["T"] - 1]))
        paths.append(sorted(rng.sample(range(1, c["T"]), n)))
    return paths, sum(len(p) + 1 for p in paths)


def _turn(c):
    """A turn's sources, kept rows and rows to grow by."""
    B, lens = c["B"], _lens(c)
    rng = random.Random(13 + B * 17 + c["W"])
    source, keep, grow = [], [], []
    for b in range(B):
        kind = rng.random()
        s = (b // c["fan"]) * c["fan"] if kind < 0.6 else b
        k = lens[s]
        if kind > 0.9:                                   # rolled back
            k = rng.randint(0, k)
        elif kind > 0.82:                                # ended; a new sequence takes its place
            s, k = -1, 0
        source.append(s)
        keep.append(k)
        grow.append(0 if rng.random() < 0.1 else min(c["grow"], c["W"] * c["P"] - k))
    return source, keep, grow


# ------------------------------------------------------------------ inputs

def _device():
    return torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")


def _randn(shape, dtype, g, dev):
    x = torch.empty(shape, dtype=dtype, device=dev)
    return x.normal_(generator=g)


def _tables(c, rows, pages, W, g, dev):
    """Page tables [B][W] that hold `rows[b]` rows a sequence: distinct pages in random order, -1 past the end."""
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((c["B"], W), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(rows):
        k = -(-n // c["P"])
        table[b, :k] = order[at:at + k]
        at += k
    return table


def prepare(case, seed):
    c, dev = case, _device()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 12345)
    st = dict(case=c)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    if c["op"] == "accept":
        par, n = _trees(c)
        B, T, V = c["B"], c["T"], c["V"]
        p = torch.empty(B, T, V, device=dev)
        q = torch.empty(B, T, V, device=dev) if c["mode"] == "specsample" else None
        tok = torch.zeros(B, T, dtype=torch.int32, device=dev)
        for b in range(B):
            z = torch.randn(T, V, generator=g, device=dev) * 3
            zd = z + 0.6 * torch.randn(T, V, generator=g, device=dev)       # a drafter that often agrees
            p[b] = torch.softmax(z, -1)
            qb = torch.softmax(zd, -1)
            if q is not None:
                q[b] = qb
                kids = torch.multinomial(qb, T, replacement=True, generator=g)
            else:
                kids = torch.topk(zd, min(T, V), -1).indices
            at = [0] * T
            for j in range(1, T):
                c_ = par[b][j]
                tok[b, j] = kids[c_, at[c_] % kids.shape[1]]
                at[c_] += 1
        u = torch.rand(2, B, T, generator=g, device=dev, dtype=torch.float64)
        return dict(st, p=p, q=q, tok=tok, parent=ints(par), n=ints(n), u_child=u[0].contiguous(),
                    u_sample=u[1].contiguous())
    dt, lens = _TYPES[c["dtype"]], _lens(c)
    B, P, H, d = c["B"], c["P"], c["Hkv"], c["d"]
    if c["op"] == "attn":
        par, n = _trees(c)
        T, Hq = c["T"], c["Hq"]
        pages = sum(-(-x // P) for x in lens) + 3
        W = -(-max(lens) // P) + 2
        table = _tables(c, lens, pages, W, g, dev)
        kv = [_randn((pages, P, H, d), dt, g, dev) for _ in range(2)]
        tree = [_randn((B, T, H, d), dt, g, dev) for _ in range(2)]
        q = _randn((B, T, Hq, d), dt, g, dev)
        return dict(st, q=q, k=kv[0], v=kv[1], table=table, lens=ints(lens), kt=tree[0], vt=tree[1], parent=ints(par),
                    n=ints(n), host=(lens, par, n), out=torch.zeros_like(q),
                    lse=torch.zeros(B, T, Hq, device=dev))
    if c["op"] == "commit":
        T, paths = c["T"], _accepted(c)[0]
        room = [x + T for x in lens]
        pages = sum(-(-x // P) for x in room) + 1
        table = _tables(c, room, pages, -(-max(room) // P), g, dev)
        kv = [_randn((c["layers"], pages, P, H, d), dt, g, dev) for _ in range(2)]
        tree = [_randn((c["layers"], B, T, H, d), dt, g, dev) for _ in range(2)]
        acc = ints([p + [-1] * (T - len(p)) for p in paths])
        return dict(st, k=kv[0], v=kv[1], table=table, lens=ints(lens), kt=tree[0], vt=tree[1],
                    n=ints([len(p) for p in paths]), acc=acc, lens_out=torch.zeros_like(ints(lens)))
    kv = [_randn((c["layers"], c["pages"], P, H, d), dt, g, dev) for _ in range(2)]
    table = _tables(c, lens, c["pages"], c["W"], g, dev)
    st.update(k=kv[0], v=kv[1], table=table, table_out=torch.empty_like(table),
              count=torch.zeros(1, dtype=torch.int32, device=dev))
    if c["op"] == "update":
        source, keep, grow = _turn(c)
        return dict(st, source=ints(source), keep=ints(keep), grow=ints(grow))
    pinned = None
    if c["pinned"]:                                      # one page in forty, free ones and used ones
        pinned = (torch.rand(c["pages"], generator=g, device=dev) < 0.025).to(torch.int32)
    return dict(st, lens=ints(lens), pinned=pinned)


# ------------------------------------------------------------------- passes

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import tree_verification_verify_b200 as tv
        if op == "attn":
            out, lse = tv.tree_verify_attn_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["kt"], s["vt"],
                                                 s["parent"], n_nodes=s["n"], out=s["out"], lse=s["lse"])
            return [out, lse]
        if op == "accept":
            o = tv.tree_accept_probs(s["p"], s["tok"], s["parent"], s["u_child"], s["u_sample"],
                                     draft_probs=s["q"], n_nodes=s["n"], mode=s["case"]["mode"])
            return [o["n_accepted"], o["accepted_nodes"], o["out_tokens"]]
        if op == "commit":
            tv.tree_commit_kv_paged(s["k"], s["v"], s["table"], s["lens"], s["kt"], s["vt"], s["n"], s["acc"],
                                    prefix_len_out=s["lens_out"])
            return [s["k"], s["v"], s["lens_out"]]
        if op == "update":
            tv.tree_pages_update(s["k"], s["v"], s["table"], s["source"], s["keep"], s["grow"],
                                 out=s["table_out"], n_free=s["count"])
        else:
            tv.tree_pages_compact(s["k"], s["v"], s["table"], s["lens"], pinned=s["pinned"],
                                  out=s["table_out"], n_used=s["count"])
        return [s["table_out"], s["count"], s["k"], s["v"]]
    return dict(attn=_attn, accept=_accept, commit=_commit, update=_update, compact=_compact)[op](s)


def _attn(s):
    """Sequence by sequence: gather the pages, scores, softmax, products, in 32 bits."""
    c = s["case"]
    lens, _, n = s["host"]
    G, P, d = c["Hq"] // c["Hkv"], c["P"], c["d"]
    for b, L in enumerate(lens):
        m = n[b]
        pages = s["table"][b, :-(-L // P)].long()
        k = torch.cat([s["k"][pages].reshape(-1, c["Hkv"], d)[:L], s["kt"][b, :m]]).float()
        v = torch.cat([s["v"][pages].reshape(-1, c["Hkv"], d)[:L], s["vt"][b, :m]]).float()
        # ancestors: a node's row is its parent's with itself added
        seen = torch.zeros(m, m, dtype=torch.bool, device=k.device)
        node = torch.arange(m, device=k.device)
        at = node
        for _ in range(m if c["tree"] == "chain" else min(m, 8)):
            seen[node, at] = True
            at = torch.maximum(s["parent"][b].long()[at], torch.zeros_like(at))
        q = s["q"][b, :m].float().view(m, c["Hkv"], G, d).permute(1, 0, 2, 3).reshape(c["Hkv"], m * G, d)
        x = torch.matmul(q, k.permute(1, 2, 0)) / math.sqrt(d)
        x.view(c["Hkv"], m, G, L + m)[..., L:].masked_fill_(~seen[None, :, None, :], -math.inf)
        top = x.max(-1, keepdim=True).values
        x = torch.exp(x - top)
        z = x.sum(-1, keepdim=True)
        o = torch.matmul(x, v.permute(1, 0, 2)) / z
        s["out"][b, :m] = o.view(c["Hkv"], m, G, d).permute(1, 0, 2, 3).reshape(m, c["Hq"], d).to(s["out"].dtype)
        lse = (top + torch.log(z)).view(c["Hkv"], m, G)
        s["lse"][b, :m] = lse.permute(1, 0, 2).reshape(m, c["Hq"])
    return [s["out"], s["lse"]]


def _sample(r, u):
    """Smallest t with cum_t > u * sum."""
    cum = torch.cumsum(r, -1)
    return torch.searchsorted(cum, (u * cum[:, -1])[:, None].contiguous(), right=True)[:, 0]


def _accept(s):
    """All sequences at once, node after node (children come after their parents), in 64 bits: sums over
    a vocabulary next to a threshold."""
    p, q, tok, par = s["p"], s["q"], s["tok"].long(), s["parent"].long()
    B, T, V = p.shape
    dev, rows = p.device, torch.arange(B, device=p.device)
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    count = torch.zeros(B, dtype=torch.long, device=dev)
    nodes = torch.full((B, T + 1), -1, dtype=torch.long, device=dev)       # one spare column takes the idle writes
    r = p[:, 0].double()
    x = _sample(r, s["u_sample"][:, 0]) if q is None else None
    for j in range(1, T):
        child = (par[:, j] == cur) & (j < s["n"])
        if q is None:
            ok = child & (tok[:, j] == x)
        else:
            qc = q[rows, cur].double()
            ratio = r.gather(1, tok[:, j:j + 1])[:, 0] / qc.gather(1, tok[:, j:j + 1])[:, 0]
            ok = child & (s["u_child"][:, j] < ratio)
            rest = torch.clamp(r - qc, min=0)
            total = rest.sum(-1)
            r = torch.where((child & ~ok & (total > 0))[:, None], rest / total[:, None], r)
        nodes[rows, torch.where(ok, count, T)] = j
        count = count + ok
        cur = torch.where(ok, j, cur)
        r = torch.where(ok[:, None], p[:, j].double(), r)
        if q is None:
            x = torch.where(ok, _sample(r, s["u_sample"][:, j]), x)
    if q is not None:
        x = _sample(r, s["u_sample"][rows, cur])
    nodes[:, T] = -1
    out = torch.full_like(nodes, -1)
    out[:, :T] = torch.where(nodes[:, :T] >= 0, tok.gather(1, nodes[:, :T].clamp(min=0)), -1)
    out[rows, count] = x
    return [count.int(), nodes[:, :T].int(), out.int()]


def _commit(s):
    """Every row of every path in one scatter; entries past a path repeat its root row."""
    c = s["case"]
    B, T, P = c["B"], c["T"], c["P"]
    dev = s["lens"].device
    r = torch.arange(T, device=dev)[None, :].expand(B, T)
    r = torch.where(r <= s["n"][:, None], r, 0)
    node = torch.cat([torch.zeros(B, 1, dtype=torch.long, device=dev), s["acc"][:, :T - 1].long()], 1).gather(1, r)
    pos = s["lens"].long()[:, None] + r
    page, row = s["table"].long().gather(1, pos // P), pos % P
    b = torch.arange(B, device=dev)[:, None].expand(B, T)
    s["k"][:, page, row] = s["kt"][:, b, node]
    s["v"][:, page, row] = s["vt"][:, b, node]
    s["lens_out"].copy_(s["lens"] + s["n"] + 1)
    return [s["k"], s["v"], s["lens_out"]]


def _update(s):
    c = s["case"]
    P, W, pages, B = c["P"], c["W"], c["pages"], c["B"]
    dev = s["table"].device
    src, keep, grow = s["source"].long(), s["keep"].long(), s["grow"].long()
    keep = torch.where(src >= 0, keep, 0)
    held, want = (keep + P - 1) // P, (keep + grow + P - 1) // P
    col = torch.arange(W, device=dev)[None, :]
    old = s["table"].long()[src.clamp(min=0)]
    has = col < held[:, None]
    partial = (keep % P > 0) & (grow > 0)
    is_part = has & partial[:, None] & (col == held[:, None] - 1)
    # pages that are read on, and the pages that one sequence goes on writing
    reads = torch.zeros(pages + 1, dtype=torch.long, device=dev)
    reads.scatter_(0, torch.where(has & ~is_part, old, pages).flatten(), 1)
    part = torch.where(partial, old.gather(1, (held - 1).clamp(min=0)[:, None])[:, 0], pages)
    first = torch.full((pages + 1,), B, dtype=torch.long, device=dev)
    first.scatter_reduce_(0, part, torch.arange(B, device=dev), "amin")
    stays = partial & (reads[part] == 0) & (first[part] == torch.arange(B, device=dev))
    copy = partial & ~stays
    free = (reads[:pages] == 0) & (first[:pages] == B)
    rank = torch.cumsum(free.long(), 0) - 1
    total = free.sum()
    lists = torch.full((pages + 1,), -1, dtype=torch.long, device=dev)
    lists.scatter_(0, torch.where(free, rank, pages), torch.where(free, torch.arange(pages, device=dev), -1))
    fresh = (is_part & copy[:, None]) | ((col >= held[:, None]) & (col < want[:, None]))
    order = (torch.cumsum(fresh.flatten().long(), 0) - 1).view(B, W)
    new = torch.where(fresh, lists[order.clamp(min=0, max=pages)], torch.where(has, old, -1))
    # copy on write, all sequences in one scatter: an entry that copies nothing writes a row that is in use with itself
    row = torch.arange(P, device=dev)[None, :].expand(B, P)
    some = part.index_select(0, copy.int().argmax()[None]).clamp(max=pages - 1)
    frm = torch.where(copy, part, some)[:, None].expand(B, P)
    to = new.gather(1, (held - 1).clamp(min=0)[:, None]).expand(B, P)
    to = torch.where(copy[:, None] & (row < (keep % P)[:, None]), to, frm)
    for t in (s["k"], s["v"]):
        t[:, to, row] = t[:, frm, row]
    s["table_out"].copy_(new)
    s["count"].copy_(total - fresh.sum())
    return [s["table_out"], s["count"], s["k"], s["v"]]


def _compact(s):
    c = s["case"]
    P, W, pages = c["P"], c["W"], c["pages"]
    dev = s["table"].device
    has = torch.arange(W, device=dev)[None, :] < ((s["lens"].long() + P - 1) // P)[:, None]
    old = s["table"].long()
    used = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    used.scatter_(0, torch.where(has, old, pages).flatten(), True)
    used = used[:pages]
    fixed = s["pinned"] != 0 if s["pinned"] is not None else torch.zeros_like(used)
    total = (used | fixed).sum()
    page = torch.arange(pages, device=dev)
    mover = used & ~fixed & (page >= total)
    hole = ~used & ~fixed & (page < total)
    lists = torch.zeros(pages + 1, dtype=torch.long, device=dev)
    lists.scatter_(0, torch.where(hole, torch.cumsum(hole.long(), 0) - 1, pages), page)
    to = torch.where(mover, lists[torch.cumsum(mover.long(), 0).clamp(min=1) - 1], page)
    s["table_out"].copy_(torch.where(has, to[old.clamp(min=0)], -1))
    s["count"].copy_(total)
    for t in (s["k"], s["v"]):
        # page x takes the page that moves to it, or stays
        come = torch.arange(pages + 1, device=dev)
        come.scatter_(0, torch.where(mover, to, pages), torch.where(mover, page, pages))
        t.copy_(t[:, come[:pages]])
    return [s["table_out"], s["count"], s["k"], s["v"]]


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits, node by node and page by page."""
    c = case
    if c["op"] == "attn":
        return _exact_attn(prepare(c, seed))
    s = prepare(c, seed)
    if c["op"] == "accept":
        return _exact_accept(s)
    if c["op"] == "commit":
        P, k, v = c["P"], s["k"], s["v"]
        lens, n, acc, table = (s[x].tolist() for x in ("lens", "n", "acc", "table"))
        for b in range(c["B"]):
            for r, node in enumerate([0] + acc[b][:n[b]]):
                page, row = table[b][(lens[b] + r) // P], (lens[b] + r) % P
                k[:, page, row], v[:, page, row] = s["kt"][:, b, node], s["vt"][:, b, node]
        out = torch.tensor([a + m + 1 for a, m in zip(lens, n)], dtype=torch.int32)
        return [k.double(), v.double(), out]
    if c["op"] == "update":
        return _exact_update(s)
    return _exact_compact(s)


def _exact_attn(s):
    c = s["case"]
    lens, par, n = s["host"]
    if work(c)["flops"] > 4e11:
        return None
    out, lse = s["out"].double(), s["lse"].double()
    G = c["Hq"] // c["Hkv"]
    for b, L in enumerate(lens):
        rows = torch.arange(L, device=out.device)
        page, row = s["table"][b].long()[rows // c["P"]], rows % c["P"]
        path = torch.zeros(n[b], n[b], dtype=torch.bool)
        for i in range(n[b]):
            j = i
            while j >= 0:
                path[i, j] = True
                j = par[b][j]
        path = path.to(out.device)
        for g in range(c["Hkv"]):
            k, v = (torch.cat([s[x][page, row, g].double(), s[y][b, :n[b], g].double()])
                    for x, y in (("k", "kt"), ("v", "vt")))
            for h in range(g * G, g * G + G):
                x = s["q"][b, :n[b], h].double() @ k.T * c["d"] ** -0.5
                x[:, L:][~path] = -math.inf
                z = torch.logsumexp(x, 1)
                out[b, :n[b], h] = torch.exp(x - z[:, None]) @ v
                lse[b, :n[b], h] = z
    return [out, lse]


def _exact_accept(s):
    c = s["case"]
    B, T = c["B"], c["T"]
    par, n, tok = (s[x].tolist() for x in ("parent", "n", "tok"))
    uc, us = s["u_child"].tolist(), s["u_sample"].tolist()
    count, nodes, out = [], [], []

    def pick(r, u):
        cum = torch.cumsum(r, 0)
        return int((cum <= u * cum[-1]).sum())

    for b in range(B):
        cur, path = 0, []
        while True:
            r, kids = s["p"][b, cur].double(), [j for j in range(cur + 1, n[b]) if par[b][j] == cur]
            nxt = None
            if s["q"] is None:
                x = pick(r, us[b][cur])
                nxt = next((j for j in kids if tok[b][j] == x), None)
            else:
                q = s["q"][b, cur].double()
                for j in kids:
                    if uc[b][j] * float(q[tok[b][j]]) < float(r[tok[b][j]]):
                        nxt = j
                        break
                    rest = torch.relu(r - q)
                    if float(rest.sum()) > 0:
                        r = rest / rest.sum()
                if nxt is None:
                    x = pick(r, us[b][cur])
            if nxt is None:
                break
            path.append(nxt)
            cur = nxt
        count.append(len(path))
        nodes.append(path + [-1] * (T - len(path)))
        out.append([tok[b][j] for j in path] + [x] + [-1] * (T - len(path)))
    return [torch.tensor(x, dtype=torch.int32) for x in (count, nodes, out)]


def _exact_update(s):
    c = s["case"]
    P, W, pages = c["P"], c["W"], c["pages"]
    old, src, keep, grow = (s[x].tolist() for x in ("table", "source", "keep", "grow"))
    read, write = set(), {}
    for b in range(c["B"]):
        if src[b] < 0:
            keep[b] = 0
        for i in range(-(-keep[b] // P)):
            page = old[src[b]][i]
            if grow[b] > 0 and (i + 1) * P > keep[b]:
                write.setdefault(page, b)
            else:
                read.add(page)
    free = [x for x in range(pages) if x not in read and x not in write]
    left, moves, new = list(free), [], []
    for b in range(c["B"]):
        line = []
        for i in range(-(-(keep[b] + grow[b]) // P)):
            if i * P >= keep[b]:
                line.append(left.pop(0))
                continue
            page = old[src[b]][i]
            if grow[b] > 0 and (i + 1) * P > keep[b] and (page in read or write[page] != b):
                moves.append((page, left[0], keep[b] - i * P))
                page = left.pop(0)
            line.append(page)
        new.append(line + [-1] * (W - len(line)))
    for t in (s["k"], s["v"]):
        for a, z, m in moves:
            t[:, z, :m] = t[:, a, :m]
    return [torch.tensor(new, dtype=torch.int32), torch.tensor([len(left)], dtype=torch.int32),
            s["k"].double(), s["v"].double()]


def _exact_compact(s):
    c = s["case"]
    P, W, pages = c["P"], c["W"], c["pages"]
    old, lens = s["table"].tolist(), s["lens"].tolist()
    fixed = set() if s["pinned"] is None else {i for i, x in enumerate(s["pinned"].tolist()) if x}
    held = [line[:-(-n // P)] for line, n in zip(old, lens)]
    used = {x for line in held for x in line}
    total = len(used | fixed)
    holes = [x for x in range(total) if x not in used and x not in fixed]
    moves = dict(zip([x for x in range(total, pages) if x in used and x not in fixed], holes))
    for t in (s["k"], s["v"]):
        for a, z in moves.items():
            t[:, z] = t[:, a]
    new = [[moves.get(x, x) for x in line] + [-1] * (W - len(line)) for line in held]
    return [torch.tensor(new, dtype=torch.int32), torch.tensor([total], dtype=torch.int32),
            s["k"].double(), s["v"].double()]
