"""Verification over a paged K/V cache: the paged calls of
include/tree_verify.h.  Their argument checks and marshalling are compiled
(csrc/paged_binding.cpp); the structs below are the C ABI's for callers that
marshal themselves.

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
import os

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
    L.tv_attn_paged_set_lost.argtypes = [c_i32]
    L.tv_attn_paged_set_lost.restype = ctypes.c_int
    L.tv_attn_paged_path.argtypes = [ctypes.POINTER(AttnPagedArgs)]
    L.tv_attn_paged_path.restype = c_i32


# ------------------------------------------------------------------ binding

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_paged.so")
_FUNCTIONS = ("tree_verify_attn_paged", "tree_verify_attn_paged_workspace_size", "tree_accept_probs",
              "tree_commit_kv_paged", "tree_commit_kv_paged_workspace_size", "tree_pages_update",
              "tree_pages_update_workspace_size", "tree_pages_compact", "tree_pages_compact_workspace_size",
              "tv_status_string")
_binding = None


def binding():
    """The compiled binding (csrc/paged_binding.cpp), given the library's functions."""
    global _binding
    if _binding is None:
        if not os.path.exists(BINDING_PATH):
            raise _tv.TVError(f"{BINDING_PATH} is missing: build it with "
                              "`python -m tree_verification_verify_b200.build`")
        from . import build
        built = build.binding_built_against()
        if built not in ("", build.binding_against()):
            raise _tv.TVError(f"{BINDING_PATH} was built against {built}, this is {build.binding_against()}: build it "
                              "again with `python -m tree_verification_verify_b200.build`")
        from . import _paged
        L = _tv.lib()
        _paged.init({n: ctypes.cast(getattr(L, n), c_vp).value for n in _FUNCTIONS}, _tv.TVError)
        _binding = _paged
    return _binding


def _raw(stream, t):
    """The handle of the stream a caller asked for (None: the tensors' device's current one)."""
    if stream is None:
        return None
    if isinstance(t, torch.Tensor) and t.is_cuda and stream.device != t.device:
        raise _tv.TVError("stream must belong to the tensors' device")
    return stream.cuda_stream


# --------------------------------------------------------------- attention

def tree_verify_attn_paged(q, k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, parent, n_nodes=None,
                           scale: float = 0.0, out=None, lse=None, want_lse: bool = True, dev_status=None,
                           stream=None, prefix_only: bool = False):
    """Tree attention over a paged prefix (include/tree_verify.h, tree_verify_attn_paged): tree_verify_attn with the
    prefix rows of sequence b found in pages page_table[b] of k_pages, v_pages [num_pages][page_size][Hkv][d].
    q [B][T][Hq][d], tree K/V [B][T][Hkv][d], page_table [B][max_pages], prefix_len [B], parent [B][T], n_nodes [B] or
    None.  T = 1 decodes single tokens.  Returns (out, lse); rows past n_nodes[b] are not written."""
    return (_binding or binding()).attn(q, k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, parent, n_nodes, scale,
                                        out, lse, want_lse, dev_status, _raw(stream, q), prefix_only)


def attn_set_lost(lost: int) -> None:
    """Test hook (tv_attn_paged_set_lost): calls behave as if a wait of the tensor-core kernel had run out, for the pieces
    of work after a CTA's first (1) or for its products (2).  0 ends it."""
    _tv._check(_tv.lib().tv_attn_paged_set_lost(int(lost)), "tv_attn_paged_set_lost")


# --------------------------------------------------------------- acceptance

_PROB_MODES = {"auto": 0, "specsample": 2, "specexec": 3}
_PROB_OUTPUTS = ("n_accepted", "accepted_nodes", "out_tokens")


def tree_accept_probs(target_probs, draft_tokens, parent, u_child, u_sample, draft_probs=None, n_nodes=None,
                      mode: str = "auto", dev_status=None, stream=None, outputs=None):
    """Acceptance walk from given probabilities and random numbers (include/tree_verify.h, tree_accept_probs).
    target_probs, draft_probs fp32 [B][T][V] with contiguous rows; draft_tokens, parent int32 [B][T]; u_child (the test
    of each node; None for "specexec") and u_sample (the sample at each node) fp64 [B][T] in [0, 1).  Returns a dict of
    device tensors n_accepted [B], accepted_nodes [B][T], out_tokens [B][T+1]: `outputs` where it holds all three, else
    a new dict with those that it lacks made."""
    if mode not in _PROB_MODES:
        raise _tv.TVError(f"mode must be one of {sorted(_PROB_MODES)}")
    o = outputs or {}
    r = (_binding or binding()).accept(target_probs, draft_tokens, parent, u_child, u_sample, draft_probs, n_nodes,
                                       _PROB_MODES[mode], dev_status, _raw(stream, target_probs),
                                       *[o.get(n) for n in _PROB_OUTPUTS])
    made = dict(zip(_PROB_OUTPUTS, r))
    if not outputs:
        return made
    return outputs if all(o.get(n) is not None for n in _PROB_OUTPUTS) else {**outputs, **made}


# --------------------------------------------------------------- KV commit

def tree_commit_kv_paged(k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, n_accepted, accepted_nodes,
                         prefix_len_out=None, dev_status=None, stream=None):
    """Append each sequence's accepted path (the root, then the accepted nodes) to its pages, all layers in one launch
    (include/tree_verify.h, tree_commit_kv_paged).  k_pages, v_pages [layers][num_pages][page_size][Hkv][d] and tree
    K/V [layers][B][T][Hkv][d], or both without the layer dimension.  prefix_len advances in place unless
    prefix_len_out is given.  Returns the tensor that holds the new lengths."""
    return (_binding or binding()).commit(k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, n_accepted,
                                          accepted_nodes, prefix_len_out, dev_status, _raw(stream, k_pages))


# --------------------------------------------------------------- page tables

def tree_pages_update(k_pages, v_pages, page_table, source, keep, grow, pinned=None, out=None, n_free=None,
                      dev_status=None, stream=None):
    """The next step's page tables (include/tree_verify.h, tree_pages_update): new sequence b keeps the first keep[b]
    rows of row source[b] of page_table (-1: new and empty) and gets room for grow[b] rows of its own.  Whole pages are
    shared, a partly kept page that b will write into and others use is copied (all layers of k_pages, v_pages
    [layers][num_pages][page_size][Hkv][d], or without the layer dimension).  pinned [num_pages] int32: pages held
    outside the table.  out [B][max_pages] int32 (default: as wide as page_table) must not be page_table.  Returns
    (out, n_free), n_free int32 [1]; negative when the pool is too small (out is then all -1)."""
    return (_binding or binding()).update(k_pages, v_pages, page_table, source, keep, grow, pinned, out, n_free, dev_status,
                                          _raw(stream, k_pages))


def tree_pages_compact(k_pages, v_pages, page_table, length, pinned=None, out=None, n_used=None, dev_status=None,
                       stream=None):
    """Move the pages in use to the front of the pool (include/tree_verify.h, tree_pages_compact): sequence b uses the
    first ceil(length[b] / page_size) entries of its page_table row.  out [B][max_pages] may be page_table itself.
    Returns (out, n_used): the renamed tables and int32 [1], the pages used or pinned."""
    return (_binding or binding()).compact(k_pages, v_pages, page_table, length, pinned, out, n_used, dev_status,
                                           _raw(stream, k_pages))
