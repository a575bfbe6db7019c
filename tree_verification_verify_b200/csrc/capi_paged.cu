// The C ABI of the paged cache's calls (tree_verify_attn_paged,
// tree_accept_probs, tree_commit_kv_paged, tree_pages_update,
// tree_pages_compact): host-side argument checks, workspace layout and
// dispatch.  Declared in include/tree_verify.h.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn.cuh"
#include "attn_paged.cuh"

namespace tv {
int num_sms();
cudaError_t launch_accept_probs(const tv_accept_probs_args* a, bool sampled, cudaStream_t stream);
size_t commit_paged_workspace_bytes();
size_t pages_update_workspace_bytes(int B, int num_pages);
size_t pages_compact_workspace_bytes(int num_pages);
cudaError_t launch_commit_paged(const tv_commit_paged_args* a, void* ws, cudaStream_t stream);
cudaError_t launch_pages_update(const tv_pages_update_args* a, void* ws, cudaStream_t stream);
cudaError_t launch_pages_compact(const tv_pages_compact_args* a, void* ws, cudaStream_t stream);
}  // namespace tv

using namespace tv;

namespace {

constexpr int kMaxPageSize = 65536;
constexpr int kMaxPages = 1 << 24;
constexpr int kMaxSeqs = 16384;
constexpr int64_t kMost = 1ll << 31;             // elements of a page of a layer, entries of a new table

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

tv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TV_OK : TV_ERR_CUDA; }

bool ws_ok(const void* ws, size_t ws_bytes, size_t need) {
  return ws != nullptr && ws_bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

bool elt_aligned(int dtype, std::initializer_list<const void*> ptrs) {
  const uintptr_t es = dtype == TV_BF16 ? 2u : 4u;
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) % es != 0) return false;
  return true;
}

// What every paged call asks of its pool.
tv_status check_pool(int dtype, int Hkv, int d, int num_pages, int page_size) {
  if (dtype != TV_FP32 && dtype != TV_BF16) return TV_ERR_INVALID_ARG;
  if (Hkv <= 0 || d < 1 || num_pages < 0 || page_size < 1) return TV_ERR_INVALID_ARG;
  if (page_size > kMaxPageSize || num_pages > kMaxPages) return TV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(Hkv) * d > (kMost - 1) / page_size) return TV_ERR_UNSUPPORTED;
  return TV_OK;
}

// ------------------------------------------------------------ attention

tv_status check_attn_paged(const tv_attn_paged_args* a) {
  if (!a) return TV_ERR_INVALID_ARG;
  const tv_status st = check_pool(a->dtype, a->Hkv, a->d, a->num_pages, a->page_size);
  if (st != TV_OK) return st;
  if (a->B < 0 || a->T < 0 || a->Hq <= 0 || a->max_pages < 0) return TV_ERR_INVALID_ARG;
  if (a->Hq % a->Hkv != 0) return TV_ERR_INVALID_ARG;
  if (!(a->scale >= 0.f) || !std::isfinite(a->scale)) return TV_ERR_INVALID_ARG;
  if (a->prefix_only != 0 && a->prefix_only != 1) return TV_ERR_INVALID_ARG;
  if (a->d != 32 && a->d != 64 && a->d != 128) return TV_ERR_UNSUPPORTED;
  if (a->Hq / a->Hkv > 64) return TV_ERR_UNSUPPORTED;
  if (a->B > 0 && a->T > 0) {
    if (!a->q || !a->prefix_len || !a->k_tree || !a->v_tree || !a->parent || !a->out) return TV_ERR_INVALID_ARG;
    if (a->max_pages > 0 && !a->page_table) return TV_ERR_INVALID_ARG;
    if (a->max_pages > 0 && a->num_pages > 0 && (!a->k_pages || !a->v_pages)) return TV_ERR_INVALID_ARG;
    if (!elt_aligned(a->dtype, {a->q, a->k_pages, a->v_pages, a->k_tree, a->v_tree, a->out}))
      return TV_ERR_INVALID_ARG;
  }
  return TV_OK;
}

struct PagedPlan {
  bool tc;
  int rows, team, grid;        // grid: stretches times team
  bool fits;                   // the line has fewer than 2^31 places
  size_t off_o, off_lse, off_splits, total;
};

PagedPlan plan_attn_paged(const tv_attn_paged_args* a) {
  PagedPlan pl;
  const int G = a->Hq / a->Hkv;
  pl.tc = attn_paged_tc_supported(a);
  pl.team = pl.tc ? attn_paged_tc_team(a) : 1;
  pl.rows = pl.tc ? 128 / G * G * pl.team : attn_paged_simt_rows(static_cast<int64_t>(a->T) * G);
  const int keys = pl.tc ? 128 : 64;
  // no more CTAs than key tiles can be
  const int64_t rt = (static_cast<int64_t>(a->T) * G + pl.rows - 1) / pl.rows;
  const int64_t tiles = (static_cast<int64_t>(a->max_pages) * a->page_size + keys - 1) / keys + (a->T + keys - 1) / keys;
  const int64_t most = static_cast<int64_t>(a->B) * a->Hkv * rt * (tiles > 0 ? tiles : 1);
  pl.fits = most + static_cast<int64_t>(a->B) * a->Hkv * rt * (pl.tc ? kPagedTcCost : kPagedSimtCost) < (1ll << 31);
  const int64_t want = static_cast<int64_t>(num_sms()) * (pl.tc ? 1 : attn_paged_simt_ctas(pl.rows, a->d));
  const int64_t stretches = std::max<int64_t>(1, std::min(most, want / pl.team));
  pl.grid = static_cast<int>(stretches * pl.team);
  const size_t slots = static_cast<size_t>(stretches) * 2 * pl.rows;
  size_t off = kTicketBytes;
  pl.off_o = off;   off = align256(off + slots * a->d * sizeof(float));
  pl.off_lse = off; off = align256(off + slots * sizeof(float));
  pl.off_splits = off; off = align256(off + pl.grid * sizeof(SplitUnit));
  pl.total = off;
  return pl;
}

}  // namespace

extern "C" size_t tree_verify_attn_paged_workspace_size(const tv_attn_paged_args* a) {
  if (check_attn_paged(a) != TV_OK) return 0;
  const PagedPlan pl = plan_attn_paged(a);
  return pl.fits ? pl.total : 0;
}

extern "C" int32_t tv_attn_paged_path(const tv_attn_paged_args* a) {
  if (check_attn_paged(a) != TV_OK) return -1;
  const PagedPlan pl = plan_attn_paged(a);
  return pl.fits ? (pl.tc ? 1 : 0) : -1;
}

extern "C" tv_status tree_verify_attn_paged(const tv_attn_paged_args* a, void* ws, size_t ws_bytes,
                                            tv_stream_t stream) {
  const tv_status st = check_attn_paged(a);
  if (st != TV_OK) return st;
  if (a->B == 0 || a->T == 0) return TV_OK;
  const PagedPlan pl = plan_attn_paged(a);
  if (!pl.fits) return TV_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, pl.total)) return TV_ERR_WORKSPACE;
  PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.dtype = a->dtype;
  p.B = a->B; p.T = a->T; p.Hq = a->Hq; p.Hkv = a->Hkv; p.d = a->d; p.G = a->Hq / a->Hkv;
  p.num_pages = a->num_pages; p.page_size = a->page_size; p.max_pages = a->max_pages;
  p.q = a->q; p.q_sb = a->q_sb; p.q_st = a->q_st; p.q_sh = a->q_sh;
  p.kp = a->k_pages; p.vp = a->v_pages; p.kv_sp = a->kv_sp; p.kv_sr = a->kv_sr; p.kv_sh = a->kv_sh;
  p.table = a->page_table; p.pt_sb = a->pt_sb;
  p.prefix_len = a->prefix_len;
  p.kt = a->k_tree; p.vt = a->v_tree; p.kt_sb = a->kt_sb; p.kt_st = a->kt_st; p.kt_sh = a->kt_sh;
  p.parent = a->parent; p.par_sb = a->parent_sb;
  p.n_nodes = a->n_nodes;
  p.scale = a->scale > 0.f ? a->scale : 1.0f / std::sqrt(static_cast<float>(a->d));
  p.out = a->out; p.o_sb = a->o_sb; p.o_st = a->o_st; p.o_sh = a->o_sh;
  p.lse = a->lse;
  p.status = a->dev_status;
  p.prefix_only = a->prefix_only;
  p.rows = pl.rows; p.team = pl.team;
  p.box = pl.tc ? attn_paged_tc_box(a->page_size) : 0;
  unsigned char* w = static_cast<unsigned char*>(ws);
  p.splits = reinterpret_cast<SplitUnit*>(w + pl.off_splits);
  p.part_o = reinterpret_cast<float*>(w + pl.off_o);
  p.part_lse = reinterpret_cast<float*>(w + pl.off_lse);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = pl.tc ? launch_attn_paged_tc(p, pl.grid, s) : launch_attn_paged_simt(p, pl.grid, s);
  if (e != cudaSuccess) return TV_ERR_CUDA;
  return from_cuda(launch_attn_paged_merge(p, pl.grid / pl.team, s));
}

extern "C" tv_status tv_attn_paged_set_lost(int32_t lost) {
  if (lost < 0 || lost > 2) return TV_ERR_INVALID_ARG;
  attn_paged_set_lost(lost);
  return TV_OK;
}

// ------------------------------------------------------------ acceptance

extern "C" tv_status tree_accept_probs(const tv_accept_probs_args* a, tv_stream_t stream) {
  if (!a) return TV_ERR_INVALID_ARG;
  if (a->B < 0 || a->T < 0 || a->V < 1) return TV_ERR_INVALID_ARG;
  if (a->mode != TV_ACCEPT_AUTO && a->mode != TV_ACCEPT_SPECSAMPLE && a->mode != TV_ACCEPT_SPECEXEC)
    return TV_ERR_INVALID_ARG;
  const bool sampled = a->mode == TV_ACCEPT_SPECSAMPLE || (a->mode == TV_ACCEPT_AUTO && a->draft_probs);
  if (a->B > kMaxSeqs || a->T > 4096 || a->V > (1 << 30)) return TV_ERR_UNSUPPORTED;
  if (a->B == 0) return TV_OK;
  if (!a->n_accepted || !a->out_tokens) return TV_ERR_INVALID_ARG;
  if (a->T > 0) {
    if (!a->accepted_nodes || !a->target_probs || !a->draft_tokens || !a->parent || !a->u_sample)
      return TV_ERR_INVALID_ARG;
    if (a->T > 1 && a->tp_st < a->V) return TV_ERR_INVALID_ARG;
    if (sampled && (!a->draft_probs || !a->u_child || (a->T > 1 && a->dp_st < a->V))) return TV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->target_probs) % 4 || reinterpret_cast<uintptr_t>(a->draft_probs) % 4)
      return TV_ERR_INVALID_ARG;
  }
  return from_cuda(launch_accept_probs(a, sampled, reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------ KV commit

namespace {
tv_status check_commit_paged(const tv_commit_paged_args* a) {
  if (!a) return TV_ERR_INVALID_ARG;
  const tv_status st = check_pool(a->dtype, a->Hkv, a->d, a->num_pages, a->page_size);
  if (st != TV_OK) return st;
  if (a->B < 0 || a->T < 0 || a->layers < 0 || a->max_pages < 0) return TV_ERR_INVALID_ARG;
  if (a->d > 1024 || a->B > kMaxSeqs || a->layers > 65535) return TV_ERR_UNSUPPORTED;
  if (a->B > 0) {
    if (a->T < 1 || a->layers < 1) return TV_ERR_INVALID_ARG;
    if (!a->k_pages || !a->v_pages || !a->prefix_len || !a->prefix_len_out || !a->k_tree || !a->v_tree ||
        !a->n_accepted || !a->page_table)
      return TV_ERR_INVALID_ARG;
    if (a->T > 1 && !a->accepted_nodes) return TV_ERR_INVALID_ARG;
    if (!elt_aligned(a->dtype, {a->k_pages, a->v_pages, a->k_tree, a->v_tree})) return TV_ERR_INVALID_ARG;
  }
  return TV_OK;
}
}  // namespace

extern "C" size_t tree_commit_kv_paged_workspace_size(const tv_commit_paged_args* a) {
  return check_commit_paged(a) == TV_OK ? commit_paged_workspace_bytes() : 0;
}

extern "C" tv_status tree_commit_kv_paged(const tv_commit_paged_args* a, void* ws, size_t ws_bytes,
                                          tv_stream_t stream) {
  const tv_status st = check_commit_paged(a);
  if (st != TV_OK) return st;
  if (a->B == 0) return TV_OK;
  if (!ws_ok(ws, ws_bytes, commit_paged_workspace_bytes())) return TV_ERR_WORKSPACE;
  return from_cuda(launch_commit_paged(a, ws, reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------ page tables

namespace {

// First and one-past-last byte of a table; empty for no rows.
bool tables_overlap(const int32_t* a, int64_t rows_a, int64_t cols_a, int64_t sa, const int32_t* b, int64_t rows_b,
                    int64_t cols_b, int64_t sb) {
  if (!a || !b || rows_a == 0 || cols_a == 0 || rows_b == 0 || cols_b == 0) return false;
  const int32_t* ea = a + (rows_a - 1) * sa + cols_a;
  const int32_t* eb = b + (rows_b - 1) * sb + cols_b;
  return a < eb && b < ea;
}

tv_status check_update(const tv_pages_update_args* a) {
  if (!a) return TV_ERR_INVALID_ARG;
  const tv_status st = check_pool(a->dtype, a->Hkv, a->d, a->num_pages, a->page_size);
  if (st != TV_OK) return st;
  if (a->B < 0 || a->B_in < 0 || a->layers < 0 || a->max_pages < 0 || a->max_pages_in < 0) return TV_ERR_INVALID_ARG;
  if (a->d > 1024 || a->B > kMaxSeqs || a->B_in > kMaxSeqs || a->layers > 65535) return TV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a->B) * a->max_pages >= kMost) return TV_ERR_UNSUPPORTED;
  if (a->layers > 0 && a->num_pages > 0) {
    if (!a->k_pages || !a->v_pages) return TV_ERR_INVALID_ARG;
    if (!elt_aligned(a->dtype, {a->k_pages, a->v_pages})) return TV_ERR_INVALID_ARG;
  }
  if (a->B_in > 0 && a->max_pages_in > 0 && (!a->page_table || (a->B_in > 1 && a->pt_sb < a->max_pages_in)))
    return TV_ERR_INVALID_ARG;
  if (a->B > 0) {
    if (!a->source || !a->keep || !a->grow) return TV_ERR_INVALID_ARG;
    if (a->max_pages > 0 && (!a->page_table_out || (a->B > 1 && a->po_sb < a->max_pages))) return TV_ERR_INVALID_ARG;
    if (tables_overlap(a->page_table, a->B_in, a->max_pages_in, a->pt_sb, a->page_table_out, a->B, a->max_pages,
                       a->po_sb))
      return TV_ERR_INVALID_ARG;
  }
  return TV_OK;
}

tv_status check_compact(const tv_pages_compact_args* a) {
  if (!a) return TV_ERR_INVALID_ARG;
  const tv_status st = check_pool(a->dtype, a->Hkv, a->d, a->num_pages, a->page_size);
  if (st != TV_OK) return st;
  if (a->B < 0 || a->layers < 0 || a->max_pages < 0) return TV_ERR_INVALID_ARG;
  if (a->d > 1024 || a->B > kMaxSeqs || a->layers > 65535) return TV_ERR_UNSUPPORTED;
  if (a->layers > 0 && a->num_pages > 0) {
    if (!a->k_pages || !a->v_pages) return TV_ERR_INVALID_ARG;
    if (!elt_aligned(a->dtype, {a->k_pages, a->v_pages})) return TV_ERR_INVALID_ARG;
  }
  if (a->B > 0) {
    if (!a->length) return TV_ERR_INVALID_ARG;
    if (a->max_pages > 0) {
      if (!a->page_table || !a->page_table_out) return TV_ERR_INVALID_ARG;
      if (a->B > 1 && (a->pt_sb < a->max_pages || a->po_sb < a->max_pages)) return TV_ERR_INVALID_ARG;
      const bool same = a->page_table == a->page_table_out && (a->B == 1 || a->pt_sb == a->po_sb);
      if (!same && tables_overlap(a->page_table, a->B, a->max_pages, a->pt_sb, a->page_table_out, a->B, a->max_pages,
                                  a->po_sb))
        return TV_ERR_INVALID_ARG;
    }
  }
  return TV_OK;
}

}  // namespace

extern "C" size_t tree_pages_update_workspace_size(const tv_pages_update_args* a) {
  return check_update(a) == TV_OK ? pages_update_workspace_bytes(a->B, a->num_pages) : 0;
}

extern "C" tv_status tree_pages_update(const tv_pages_update_args* a, void* ws, size_t ws_bytes, tv_stream_t stream) {
  const tv_status st = check_update(a);
  if (st != TV_OK) return st;
  if (!ws_ok(ws, ws_bytes, pages_update_workspace_bytes(a->B, a->num_pages))) return TV_ERR_WORKSPACE;
  return from_cuda(launch_pages_update(a, ws, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t tree_pages_compact_workspace_size(const tv_pages_compact_args* a) {
  return check_compact(a) == TV_OK ? pages_compact_workspace_bytes(a->num_pages) : 0;
}

extern "C" tv_status tree_pages_compact(const tv_pages_compact_args* a, void* ws, size_t ws_bytes, tv_stream_t stream) {
  const tv_status st = check_compact(a);
  if (st != TV_OK) return st;
  if (!ws_ok(ws, ws_bytes, pages_compact_workspace_bytes(a->num_pages))) return TV_ERR_WORKSPACE;
  return from_cuda(launch_pages_compact(a, ws, reinterpret_cast<cudaStream_t>(stream)));
}
