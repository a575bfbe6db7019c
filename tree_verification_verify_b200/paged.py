"""Verification over a paged K/V cache: binding of the paged calls of
include/tree_verify.h (argument checks and marshalling only).

    tree_verify_attn_paged   tree attention through a page table
    tree_accept_probs        acceptance walk from given probabilities and
                             given random numbers
    tree_commit_kv_paged     the accepted path's K/V into its pages
    tree_pages_update        next page tables: fork, roll back, free, grow,
                             copy on write
    tree_pages_compact       the pages in use to the front of the pool

A cache is two tensors k_pages, v_pages [num_pages][page_size][Hkv][d] with
equal strides and a contiguous last dimension; where all layers are handled
in one call they may have a leading layer dimension.  Index tensors are
int32.

Every call runs on the device of its tensors, on that device's current
stream unless `stream` is given.  Scratch is kept per device and stream;
calls captured into a CUDA graph get scratch of their own inside the graph,
so graphs may be replayed at the same time.
"""

from __future__ import annotations

import ctypes

import torch

import tree_verification_verify_b200 as _tv

c_i32, c_i64, c_f32, c_vp, c_size = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                                      ctypes.c_size_t)

_POOL = [("k_pages", c_vp), ("v_pages", c_vp)]


class AttnPagedArgs(ctypes.Structure):
    _fields_ = [("dtype", c_i32), ("B", c_i32), ("T", c_i32), ("Hq", c_i32), ("Hkv", c_i32), ("d", c_i32),
                ("num_pages", c_i32), ("page_size", c_i32), ("max_pages", c_i32),
                ("q", c_vp), ("q_sb", c_i64), ("q_st", c_i64), ("q_sh", c_i64),
                *_POOL, ("kv_sp", c_i64), ("kv_sr", c_i64), ("kv_sh", c_i64),
                ("page_table", c_vp), ("pt_sb", c_i64), ("prefix_len", c_vp),
                ("k_tree", c_vp), ("v_tree", c_vp), ("kt_sb", c_i64), ("kt_st", c_i64), ("kt_sh", c_i64),
                ("parent", c_vp), ("parent_sb", c_i64), ("n_nodes", c_vp), ("scale", c_f32),
                ("out", c_vp), ("o_sb", c_i64), ("o_st", c_i64), ("o_sh", c_i64),
                ("lse", c_vp), ("dev_status", c_vp), ("prefix_only", c_i32)]


class AcceptProbsArgs(ctypes.Structure):
    _fields_ = [("B", c_i32), ("T", c_i32), ("V", c_i32),
                ("target_probs", c_vp), ("tp_sb", c_i64), ("tp_st", c_i64),
                ("draft_probs", c_vp), ("dp_sb", c_i64), ("dp_st", c_i64),
                ("draft_tokens", c_vp), ("tok_sb", c_i64), ("parent", c_vp), ("parent_sb", c_i64),
                ("n_nodes", c_vp), ("u_child", c_vp), ("u_sample", c_vp), ("mode", c_i32),
                ("n_accepted", c_vp), ("accepted_nodes", c_vp), ("out_tokens", c_vp), ("dev_status", c_vp)]


class CommitPagedArgs(ctypes.Structure):
    _fields_ = [("dtype", c_i32), ("layers", c_i32), ("B", c_i32), ("T", c_i32), ("Hkv", c_i32), ("d", c_i32),
                ("num_pages", c_i32), ("page_size", c_i32), ("max_pages", c_i32),
                *_POOL, ("kv_sl", c_i64), ("kv_sp", c_i64), ("kv_sr", c_i64), ("kv_sh", c_i64),
                ("page_table", c_vp), ("pt_sb", c_i64), ("prefix_len", c_vp), ("prefix_len_out", c_vp),
                ("k_tree", c_vp), ("v_tree", c_vp), ("kt_sl", c_i64), ("kt_sb", c_i64), ("kt_st", c_i64),
                ("kt_sh", c_i64), ("n_accepted", c_vp), ("accepted_nodes", c_vp), ("acc_sb", c_i64),
                ("dev_status", c_vp)]


class PagesUpdateArgs(ctypes.Structure):
    _fields_ = [("dtype", c_i32), ("layers", c_i32), ("B_in", c_i32), ("B", c_i32), ("Hkv", c_i32), ("d", c_i32),
                ("num_pages", c_i32), ("page_size", c_i32), ("max_pages_in", c_i32), ("max_pages", c_i32),
                *_POOL, ("kv_sl", c_i64), ("kv_sp", c_i64), ("kv_sr", c_i64), ("kv_sh", c_i64),
                ("page_table", c_vp), ("pt_sb", c_i64), ("source", c_vp), ("keep", c_vp), ("grow", c_vp),
                ("pinned", c_vp), ("page_table_out", c_vp), ("po_sb", c_i64), ("n_free", c_vp),
                ("dev_status", c_vp)]


class PagesCompactArgs(ctypes.Structure):
    _fields_ = [("dtype", c_i32), ("layers", c_i32), ("B", c_i32), ("Hkv", c_i32), ("d", c_i32),
                ("num_pages", c_i32), ("page_size", c_i32), ("max_pages", c_i32),
                *_POOL, ("kv_sl", c_i64), ("kv_sp", c_i64), ("kv_sr", c_i64), ("kv_sh", c_i64),
                ("page_table", c_vp), ("pt_sb", c_i64), ("length", c_vp), ("pinned", c_vp),
                ("page_table_out", c_vp), ("po_sb", c_i64), ("n_used", c_vp), ("dev_status", c_vp)]


def bind(L):
    """Declare the calls of this module on the loaded library."""
    for name, args in (("tree_verify_attn_paged", AttnPagedArgs), ("tree_commit_kv_paged", CommitPagedArgs),
                       ("tree_pages_update", PagesUpdateArgs), ("tree_pages_compact", PagesCompactArgs)):
        f = getattr(L, name)
        f.argtypes = [ctypes.POINTER(args), c_vp, c_size, c_vp]
        f.restype = ctypes.c_int
        f = getattr(L, name + "_workspace_size")
        f.argtypes = [ctypes.POINTER(args)]
        f.restype = c_size
    L.tree_accept_probs.argtypes = [ctypes.POINTER(AcceptProbsArgs), c_vp]
    L.tree_accept_probs.restype = ctypes.c_int
    L.tv_attn_paged_path.argtypes = [ctypes.POINTER(AttnPagedArgs)]
    L.tv_attn_paged_path.restype = c_i32


# ------------------------------------------------------------------ checks

_DTYPES = {torch.bfloat16: _tv.TV_BF16, torch.float32: _tv.TV_FP32}


def _dt(t, what):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise _tv.TVError(f"{what} must be bf16 or fp32")
    return dt


def _need(ok, msg):
    if not ok:
        raise _tv.TVError(msg)


def _vec(t, n, name, dtype=torch.int32):
    if t is not None and (t.dtype != dtype or t.shape != (n,) or not t.is_contiguous()):
        raise _tv.TVError(f"{name} must be contiguous {dtype} of shape ({n},)")
    return None if t is None else t.data_ptr()


def _mat(t, rows, cols, name):
    """A [rows][cols] int32 table with contiguous rows."""
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != rows or (cols is not None and t.shape[1] != cols) or \
            (t.stride(1) != 1 and t.shape[1] > 1 and t.numel() > 0):
        raise _tv.TVError(f"{name} must be int32 [{rows}][{'...' if cols is None else cols}] with contiguous rows")
    return t


def _pair(k, v, dims, name):
    if k.dim() not in dims or k.dtype != v.dtype or k.shape != v.shape or k.stride() != v.stride():
        raise _tv.TVError(f"{name} K and V must share shape, strides and dtype")
    if k.stride(-1) != 1:
        raise _tv.TVError(f"{name} K/V must have a contiguous last dimension")


def _layers(t):
    """(layers, layer stride, the other strides) of a tensor with an optional leading layer dimension."""
    st = t.stride()
    return (t.shape[0], st[0], st[1:]) if t.dim() == 5 else (1, 0, st)


def _pool(k_pages, v_pages):
    """Shape and strides of a pool with an optional layer dimension."""
    _pair(k_pages, v_pages, (4, 5), "the pool's")
    layers, sl, st = _layers(k_pages)
    num_pages, P, Hkv, d = k_pages.shape[-4:]
    return layers, num_pages, P, Hkv, d, sl, st


# Scratch per (device, stream): made on that stream, its ticket counters
# zeroed once and left zero by every call.
_scratch = {}


class _Call:
    """The device, stream and scratch of one call.  Its tensors must share one CUDA device."""

    __slots__ = ("dev", "stream", "raw", "guard")

    def __init__(self, stream, *ts):
        dev = _tv._need_cuda(*ts)
        self.dev = dev
        self.stream = stream
        self.raw = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream
        # another device than the current one, or another stream: allocations and launches go there
        self.guard = None
        if stream is not None:
            _need(stream.device == dev, "stream must belong to the tensors' device")
            self.guard = torch.cuda.stream(stream)
        elif torch._C._cuda_getDevice() != dev.index:
            self.guard = torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)
        return False

    def run(self, name, args):
        """Launch a call that takes a workspace."""
        L = _tv.lib()
        p = ctypes.byref(args)
        need = getattr(L, name + "_workspace_size")(p)
        ptr = None
        if need:
            if torch.cuda.is_current_stream_capturing():
                # part of the graph: no other graph or stream can meet it
                buf = torch.empty(need + 256, dtype=torch.uint8, device=self.dev)
                buf[:_TICKET_BYTES + 256].zero_()
            else:
                buf = _scratch.get((self.dev.index, self.raw))
                if buf is None or buf.numel() < need + 256:
                    buf = torch.zeros(need + 256, dtype=torch.uint8, device=self.dev)
                    _scratch[self.dev.index, self.raw] = buf
            ptr = (buf.data_ptr() + 255) & ~255
        _tv._check(getattr(L, name)(p, ptr, need, self.raw), name)


_TICKET_BYTES = 64 * 1024


# --------------------------------------------------------------- attention

def tree_verify_attn_paged(q, k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, parent, n_nodes=None,
                           scale: float = 0.0, out=None, lse=None, want_lse: bool = True, dev_status=None,
                           stream=None, prefix_only: bool = False):
    """Tree attention over a paged prefix (include/tree_verify.h, tree_verify_attn_paged): tree_verify_attn with the
    prefix rows of sequence b found in pages page_table[b] of k_pages, v_pages [num_pages][page_size][Hkv][d].
    q [B][T][Hq][d], tree K/V [B][T][Hkv][d], page_table [B][max_pages], prefix_len [B], parent [B][T], n_nodes [B] or
    None.  T = 1 decodes single tokens.  Returns (out, lse); rows past n_nodes[b] are not written."""
    with _Call(stream, q, k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, parent, n_nodes, out, lse,
               dev_status) as c:
        dt = _dt(q, "q")
        _need(q.dim() == 4 and q.stride(3) == 1, "q must be [B][T][Hq][d] with a contiguous last dimension")
        B, T, Hq, d = q.shape
        _pair(k_pages, v_pages, (4,), "the pool's")
        _pair(k_tree, v_tree, (4,), "tree")
        num_pages, P, Hkv, dk = k_pages.shape
        _need(k_pages.dtype == q.dtype and k_tree.dtype == q.dtype and dk == d, "K/V must share q's dtype and d")
        _need(k_tree.shape == (B, T, Hkv, d), "tree K/V must be [B][T][Hkv][d]")
        _mat(page_table, B, None, "page_table")
        _mat(parent, B, T, "parent")
        if out is None:
            out = torch.empty(B, T, Hq, d, dtype=q.dtype, device=c.dev)
        _need(out.shape == q.shape and out.dtype == q.dtype and out.stride(3) == 1,
              "out must have q's shape and dtype with a contiguous last dimension")
        if lse is None and want_lse:
            lse = torch.empty(B, T, Hq, dtype=torch.float32, device=c.dev)
        _need(lse is None or (lse.shape == (B, T, Hq) and lse.dtype == torch.float32 and lse.is_contiguous()),
              "lse must be contiguous fp32 [B][T][Hq]")
        qs, ks, ts, os = q.stride(), k_pages.stride(), k_tree.stride(), out.stride()
        a = AttnPagedArgs(dt, B, T, Hq, Hkv, d, num_pages, P, page_table.shape[1],
                          q.data_ptr(), qs[0], qs[1], qs[2],
                          k_pages.data_ptr(), v_pages.data_ptr(), ks[0], ks[1], ks[2],
                          page_table.data_ptr(), page_table.stride(0), _vec(prefix_len, B, "prefix_len"),
                          k_tree.data_ptr(), v_tree.data_ptr(), ts[0], ts[1], ts[2],
                          parent.data_ptr(), parent.stride(0), _vec(n_nodes, B, "n_nodes"), scale,
                          out.data_ptr(), os[0], os[1], os[2], None if lse is None else lse.data_ptr(),
                          None if dev_status is None else dev_status.data_ptr(), bool(prefix_only))
        c.run("tree_verify_attn_paged", a)
        return out, lse


# --------------------------------------------------------------- acceptance

_PROB_MODES = {"auto": 0, "specsample": 2, "specexec": 3}


def tree_accept_probs(target_probs, draft_tokens, parent, u_child, u_sample, draft_probs=None, n_nodes=None,
                      mode: str = "auto", dev_status=None, stream=None, outputs=None):
    """Acceptance walk from given probabilities and random numbers (include/tree_verify.h, tree_accept_probs).
    target_probs, draft_probs fp32 [B][T][V] with contiguous rows; draft_tokens, parent int32 [B][T]; u_child (the test
    of each node; None for "specexec") and u_sample (the sample at each node) fp64 [B][T] in [0, 1).  Returns a dict of
    device tensors n_accepted [B], accepted_nodes [B][T], out_tokens [B][T+1]."""
    o = outputs
    with _Call(stream, target_probs, draft_tokens, parent, u_child, u_sample, draft_probs, n_nodes, dev_status,
               *(() if o is None else o.values())) as c:
        _need(mode in _PROB_MODES, f"mode must be one of {sorted(_PROB_MODES)}")
        _need(target_probs.dim() == 3, "target_probs must be [B][T][V]")
        B, T, V = target_probs.shape
        for t, name in ((target_probs, "target_probs"), (draft_probs, "draft_probs")):
            _need(t is None or (t.dtype == torch.float32 and t.shape == (B, T, V) and (V == 1 or t.stride(2) == 1)),
                  f"{name} must be fp32 [B][T][V] with contiguous rows")
        _mat(draft_tokens, B, T, "draft_tokens")
        _mat(parent, B, T, "parent")
        for t, name in ((u_child, "u_child"), (u_sample, "u_sample")):
            _need(t is None or (t.dtype == torch.float64 and t.shape == (B, T) and t.is_contiguous()),
                  f"{name} must be contiguous fp64 [B][T]")
        if o is None:
            o = dict(n_accepted=torch.empty(B, dtype=torch.int32, device=c.dev),
                     accepted_nodes=torch.empty(B, T, dtype=torch.int32, device=c.dev),
                     out_tokens=torch.empty(B, T + 1, dtype=torch.int32, device=c.dev))
        for name, shape in (("n_accepted", (B,)), ("accepted_nodes", (B, T)), ("out_tokens", (B, T + 1))):
            _need(o[name].dtype == torch.int32 and o[name].shape == shape and o[name].is_contiguous(),
                  f"{name} must be contiguous int32 {shape}")
        tp, dp = target_probs.stride(), (0, 0) if draft_probs is None else draft_probs.stride()
        a = AcceptProbsArgs(B, T, V, target_probs.data_ptr(), tp[0], tp[1],
                            None if draft_probs is None else draft_probs.data_ptr(), dp[0], dp[1],
                            draft_tokens.data_ptr(), draft_tokens.stride(0), parent.data_ptr(), parent.stride(0),
                            _vec(n_nodes, B, "n_nodes"), None if u_child is None else u_child.data_ptr(),
                            None if u_sample is None else u_sample.data_ptr(), _PROB_MODES[mode],
                            o["n_accepted"].data_ptr(), o["accepted_nodes"].data_ptr(), o["out_tokens"].data_ptr(),
                            None if dev_status is None else dev_status.data_ptr())
        _tv._check(_tv.lib().tree_accept_probs(ctypes.byref(a), c.raw), "tree_accept_probs")
        return o


# --------------------------------------------------------------- KV commit

def tree_commit_kv_paged(k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, n_accepted, accepted_nodes,
                         prefix_len_out=None, dev_status=None, stream=None):
    """Append each sequence's accepted path (the root, then the accepted nodes) to its pages, all layers in one launch
    (include/tree_verify.h, tree_commit_kv_paged).  k_pages, v_pages [layers][num_pages][page_size][Hkv][d] and tree
    K/V [layers][B][T][Hkv][d], or both without the layer dimension.  prefix_len advances in place unless
    prefix_len_out is given.  Returns the tensor that holds the new lengths."""
    if prefix_len_out is None:
        prefix_len_out = prefix_len
    with _Call(stream, k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, n_accepted, accepted_nodes,
               prefix_len_out, dev_status) as c:
        dt = _dt(k_pages, "K/V")
        layers, num_pages, P, Hkv, d, sl, ps = _pool(k_pages, v_pages)
        _pair(k_tree, v_tree, (k_pages.dim(),), "tree")
        tl, tsl, ts = _layers(k_tree)
        B, T = k_tree.shape[-4:-2]
        _need(k_tree.dtype == k_pages.dtype and tl == layers and k_tree.shape[-2:] == (Hkv, d),
              "tree K/V must be [layers][B][T][Hkv][d] of the pool's dtype")
        _mat(page_table, B, None, "page_table")
        _mat(accepted_nodes, B, T, "accepted_nodes")
        a = CommitPagedArgs(dt, layers, B, T, Hkv, d, num_pages, P, page_table.shape[1],
                            k_pages.data_ptr(), v_pages.data_ptr(), sl, ps[0], ps[1], ps[2],
                            page_table.data_ptr(), page_table.stride(0), _vec(prefix_len, B, "prefix_len"),
                            _vec(prefix_len_out, B, "prefix_len_out"),
                            k_tree.data_ptr(), v_tree.data_ptr(), tsl, ts[0], ts[1], ts[2],
                            _vec(n_accepted, B, "n_accepted"), accepted_nodes.data_ptr(), accepted_nodes.stride(0),
                            None if dev_status is None else dev_status.data_ptr())
        c.run("tree_commit_kv_paged", a)
        return prefix_len_out


# --------------------------------------------------------------- page tables

def _table_out(c, out, B, W):
    if out is None:
        out = torch.empty(B, W, dtype=torch.int32, device=c.dev)
    return _mat(out, B, None, "out")


def tree_pages_update(k_pages, v_pages, page_table, source, keep, grow, pinned=None, out=None, n_free=None,
                      dev_status=None, stream=None):
    """The next step's page tables (include/tree_verify.h, tree_pages_update): new sequence b keeps the first keep[b]
    rows of row source[b] of page_table (-1: new and empty) and gets room for grow[b] rows of its own.  Whole pages are
    shared, a partly kept page that b will write into and others use is copied (all layers of k_pages, v_pages
    [layers][num_pages][page_size][Hkv][d], or without the layer dimension).  pinned [num_pages] int32: pages held
    outside the table.  out [B][max_pages] int32 (default: as wide as page_table) must not be page_table.  Returns
    (out, n_free), n_free int32 [1]; negative when the pool is too small (out is then all -1)."""
    with _Call(stream, k_pages, v_pages, page_table, source, keep, grow, pinned, out, n_free, dev_status) as c:
        dt = _dt(k_pages, "K/V")
        layers, num_pages, P, Hkv, d, sl, ps = _pool(k_pages, v_pages)
        _need(page_table.dim() == 2 and source.dim() == 1, "page_table must be [B_in][max_pages], source [B]")
        B_in, W_in = page_table.shape
        B = source.shape[0]
        _mat(page_table, B_in, W_in, "page_table")
        out = _table_out(c, out, B, W_in)
        if n_free is None:
            n_free = torch.empty(1, dtype=torch.int32, device=c.dev)
        a = PagesUpdateArgs(dt, layers, B_in, B, Hkv, d, num_pages, P, W_in, out.shape[1],
                            k_pages.data_ptr(), v_pages.data_ptr(), sl, ps[0], ps[1], ps[2],
                            page_table.data_ptr(), page_table.stride(0), _vec(source, B, "source"),
                            _vec(keep, B, "keep"), _vec(grow, B, "grow"), _vec(pinned, num_pages, "pinned"),
                            out.data_ptr(), out.stride(0), _vec(n_free, 1, "n_free"),
                            None if dev_status is None else dev_status.data_ptr())
        c.run("tree_pages_update", a)
        return out, n_free


def tree_pages_compact(k_pages, v_pages, page_table, length, pinned=None, out=None, n_used=None, dev_status=None,
                       stream=None):
    """Move the pages in use to the front of the pool (include/tree_verify.h, tree_pages_compact): sequence b uses the
    first ceil(length[b] / page_size) entries of its page_table row.  out [B][max_pages] may be page_table itself.
    Returns (out, n_used): the renamed tables and int32 [1], the pages used or pinned."""
    with _Call(stream, k_pages, v_pages, page_table, length, pinned, out, n_used, dev_status) as c:
        dt = _dt(k_pages, "K/V")
        layers, num_pages, P, Hkv, d, sl, ps = _pool(k_pages, v_pages)
        _need(page_table.dim() == 2, "page_table must be [B][max_pages]")
        B, W = page_table.shape
        _mat(page_table, B, W, "page_table")
        out = _table_out(c, out, B, W)
        _need(out.shape == page_table.shape, "out must have page_table's shape")
        if n_used is None:
            n_used = torch.empty(1, dtype=torch.int32, device=c.dev)
        a = PagesCompactArgs(dt, layers, B, Hkv, d, num_pages, P, W,
                             k_pages.data_ptr(), v_pages.data_ptr(), sl, ps[0], ps[1], ps[2],
                             page_table.data_ptr(), page_table.stride(0), _vec(length, B, "length"),
                             _vec(pinned, num_pages, "pinned"), out.data_ptr(), out.stride(0),
                             _vec(n_used, 1, "n_used"), None if dev_status is None else dev_status.data_ptr())
        c.run("tree_pages_compact", a)
        return out, n_used
