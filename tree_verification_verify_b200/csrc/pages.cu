// The paged cache's rows and pages: tree_commit_kv_paged, tree_pages_update,
// tree_pages_compact.
//
// All three move rows of K and V between places that tables on the device
// name.  Update and compaction first need a plan of the whole pool: the pages
// in use as a bitmap, the free ones ranked by a prefix sum over its words,
// every sequence's place in that order.
//   Small pools (16384 table entries, 32768 pages, 256 sequences at most)
//   run as one kernel: every CTA makes the plan for itself in shared memory,
//   a few us of three dependent reads, and does its part of the copies.
//   (With the plan in a kernel of its own, most of it launches and cluster
//   barriers: 4 beams 18.5 us for 8.3, 128 sequences 24.7 for 14.4, 250 in
//   16000 pages 22.7 for 18.5.  At 32700 pages the two are equal, 22.6; beyond
//   the limits one kernel loses: 500 sequences 30.8 for 25.7, 256 in 60000
//   pages 30.8 for 24.7.  Compaction likewise: 18.2 for 8.3 and 36.7 for 22.6,
//   then 293 for 271 in 60000 pages.)
//   Larger ones run as two: one cluster of eight CTAs makes the plan, its
//   steps separated by cluster barriers, so it needs neither a cleared
//   workspace nor a grid-wide wait; the second kernel writes the new tables
//   and copies the rows over the whole GPU.
// Measured: commit of 32 paths of up to 16 rows in 32 layers 14.4 us (38 MB;
// 10.3 where the rows lie in the L2); update of 128 sequences in a pool of 1200
// pages of 64 rows, 2 layers 17.2 us (29 MB); compaction of 3500 pages of 16
// rows, 2 layers 37 us (153 MB), of 60000 pages 271 us (1.5 GB); 4 sequences 8.4
// us each.  The plan's dependent reads bound the small ones, HBM the copies.
// Results depend on ranks alone, never on the order in which threads arrive.
#include <cooperative_groups.h>

#include <algorithm>
#include <initializer_list>

#include "tv_common.cuh"

namespace cg = cooperative_groups;

namespace tv {

namespace pages {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;               // of one CTA of the plan
constexpr int kPlanCtas = 8;                     // a portable cluster
constexpr int kSmallThreads = 512;               // of a CTA that plans for itself
constexpr uint32_t kSmallSlice = 4 * kSmallThreads;   // words of a page of a layer that a CTA copies at a time
constexpr int64_t kSmallEntries = 16384;
constexpr int kSmallPages = 32768, kSmallSeqs = 256;
constexpr int kTicketBytes = 64 * 1024;

// Rows of one tensor: element strides of a (row, head) vector, and whether
// the rows of a page follow one another without gaps.
struct Pool {
  char* k;
  char* v;
  int64_t sl, sp, sr, sh;      // bytes: layer, page, row, head
  int Hkv, vec_bytes;          // bytes of a (row, head) vector
  int dense;                   // a page's rows are one run of bytes
};

__host__ __device__ inline int small_slices(int P, int words_per_row) {
  return static_cast<int>((static_cast<int64_t>(P) * words_per_row + kSmallSlice - 1) / kSmallSlice);
}

template <typename W>
__device__ __forceinline__ W ldw(const char* p) { return *reinterpret_cast<const W*>(p); }
template <typename W>
__device__ __forceinline__ void stw(char* p, W v) { *reinterpret_cast<W*>(p) = v; }

// Words of a page of a layer; the host refuses pages of 2^31 elements.  Places
// a slice or a step past the last word still fit 32 bits without a sign.
template <typename W>
__device__ __forceinline__ uint32_t page_words(const Pool& pl, int P) {
  return static_cast<uint32_t>(P) * pl.Hkv * (pl.vec_bytes / static_cast<int>(sizeof(W)));
}

// Copies words [w0, w1) from page address s to page address d (byte offsets
// into k and v), by the calling CTA.
template <typename W, int NT>
__device__ __forceinline__ void copy_words(const Pool& pl, int64_t d, int64_t s, uint32_t w0, uint32_t w1) {
  const uint32_t wpv = pl.vec_bytes / static_cast<uint32_t>(sizeof(W));
  const uint32_t wpr = wpv * pl.Hkv;
  constexpr int U = 4;
  for (uint32_t i0 = w0 + threadIdx.x; i0 < w1; i0 += U * NT) {
    W a[U], b[U];
    int64_t off[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + u * NT;
      if (i < w1) {
        if (pl.dense) {
          off[u] = static_cast<int64_t>(i) * sizeof(W);
        } else {
          const uint32_t r = i / wpr, h = i % wpr / wpv, w = i % wpv;
          off[u] = r * pl.sr + h * pl.sh + static_cast<int64_t>(w) * sizeof(W);
        }
        a[u] = ldw<W>(pl.k + s + off[u]);
        b[u] = ldw<W>(pl.v + s + off[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * NT < w1) {
        stw<W>(pl.k + d + off[u], a[u]);
        stw<W>(pl.v + d + off[u], b[u]);
      }
    }
  }
}

// Exclusive prefix sum of v over a CTA of NT threads; *total is the sum.
template <int NT = kPlanThreads>
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int ws[NT / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();                               // ws of the last call is read
  if (lane == 31) ws[warp] = incl;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    before += w < warp ? ws[w] : 0;
    sum += ws[w];
  }
  *total = sum;
  return before + incl - v;
}

// Exclusive prefix sums of n shared-memory counts in place; returns the sum.
template <int NT>
__device__ __forceinline__ int scan_array(int* v, int n) {
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += NT) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    const int x = i < n ? v[i] : 0;
    int sum;
    const int before = block_scan<NT>(x, &sum);
    if (i < n) v[i] = base + before;
    base += sum;
  }
  __syncthreads();
  return base;
}

// f(b, i, entry i of row(b)) for the first held(b) entries of every sequence: a
// warp per sequence, four sequences' loads in flight.
template <int NT, typename Held, typename Row, typename F>
__device__ __forceinline__ void for_entries(int B, Held held, Row row, F f) {
  constexpr int kWarps = NT / 32, U = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b0 = warp; b0 < B; b0 += U * kWarps) {
    int h[U], most = 0;
    const int32_t* r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * kWarps;
      h[u] = b < B ? held(b) : 0;
      r[u] = b < B ? row(b) : nullptr;
      most = max(most, h[u]);
    }
    for (int i = lane; i < most; i += 32) {
      int page[U];
#pragma unroll
      for (int u = 0; u < U; ++u) page[u] = i < h[u] ? __ldg(r[u] + i) : 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i < h[u]) f(b0 + u * kWarps, i, page[u]);
    }
  }
}

// Index of set bit number k of a bitmap whose words' prefix counts are known.
template <typename F>
__device__ __forceinline__ int select_bit(const int* before, int words, int k, F word) {
  int lo = 0, hi = words;                        // last word with before <= k
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= k) lo = mid; else hi = mid;
  }
  uint32_t m = word(lo);
  for (int r = k - before[lo]; r > 0; --r) m &= m - 1u;
  return lo * 32 + __ffs(m) - 1;
}

// The CTAs' shares of a sum: every CTA posts `mine`, and after a cluster
// barrier the sum of the CTAs before this one and the whole sum are known.
// `slots` is a place of kPlanCtas ints of its own for every call.
__device__ __forceinline__ int cluster_base(cg::cluster_group& cl, int* slots, int mine, int* total) {
  const int rank = static_cast<int>(cl.block_rank());
  if (threadIdx.x < kPlanCtas) cl.map_shared_rank(slots, threadIdx.x)[rank] = mine;
  cl.sync();
  int before = 0, sum = 0;
#pragma unroll
  for (int c = 0; c < kPlanCtas; ++c) {
    before += c < rank ? slots[c] : 0;
    sum += slots[c];
  }
  *total = sum;
  return before;
}

}  // namespace pages

using namespace pages;

// ------------------------------------------------------------------ commit

struct CommitPagedParams {
  Pool pool;
  int layers, B, T, P, num_pages;
  int64_t cap;                                   // rows of a table row
  const int32_t* table; int64_t pt_sb;
  const int32_t* len;
  int32_t* len_out;
  const char* kt; const char* vt; int64_t tl, tb, tt, th;   // bytes
  const int32_t* n_acc;
  const int32_t* acc; int64_t acc_sb;
  int32_t* tickets;
  uint32_t* status;
  int step;                                      // path rows at a time: their words are fewer than 2^31
};

constexpr int kCommitRows = 256;                 // path rows looked up at a time, at most

// One CTA per (sequence, layer).  Path row r goes from tree node rows[r] to
// row (L + r) % P of page table[(L + r) / P]; the rows' addresses are looked
// up once per CTA into shared memory, then all (row, head) vectors are
// copied word by word.  Every CTA checks the whole path and its pages before
// it writes, so a sequence is committed in all layers or in none.
template <typename W>
__global__ void __launch_bounds__(kThreads) commit_paged_kernel(CommitPagedParams p) {
  __shared__ int64_t s_src[kCommitRows], s_dst[kCommitRows];
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const int L = p.len[b], n = p.n_acc[b];
  const int32_t* acc = p.acc + b * p.acc_sb;
  const int32_t* table = p.table + b * p.pt_sb;
  const bool ok_len = n >= 0 && n < p.T && L >= 0 && static_cast<int64_t>(L) + n + 1 <= p.cap;
  int bad = 0;
  if (ok_len) {
    for (int r = tid; r <= n; r += kThreads) {
      const int x = r == 0 ? 0 : acc[r - 1];
      if (r > 0 && (x < 1 || x >= p.T || (r > 1 && acc[r - 2] >= x))) bad |= 1;
      const int page = table[(L + r) / p.P];
      if (page < 0 || page >= p.num_pages) bad |= 2;
      if (r < kCommitRows) {
        s_src[r] = b * p.tb + x * p.tt;
        s_dst[r] = page * p.pool.sp + static_cast<int64_t>((L + r) % p.P) * p.pool.sr;
      }
    }
  }
  const int bad_row = __syncthreads_or(bad & 1), bad_page = __syncthreads_or(bad & 2);
  const bool ok = ok_len && !bad_row && !bad_page;
  if (tid == 0 && layer == 0 && !ok)
    set_status(p.status, !ok_len ? TV_DEV_BAD_LEN : (bad_row ? TV_DEV_BAD_ROW : 0u) | (bad_page ? TV_DEV_BAD_PAGE : 0u));
  if (ok) {
    const uint32_t wpv = p.pool.vec_bytes / static_cast<uint32_t>(sizeof(W));
    const uint32_t wpr = wpv * p.pool.Hkv;
    for (int r0 = 0; r0 <= n; r0 += p.step) {
      const int rows = min(p.step, n + 1 - r0);
      if (r0 > 0) {
        __syncthreads();
        if (tid < rows) {
          const int r = r0 + tid;
          s_src[tid] = b * p.tb + acc[r - 1] * p.tt;
          s_dst[tid] = table[(L + r) / p.P] * p.pool.sp + static_cast<int64_t>((L + r) % p.P) * p.pool.sr;
        }
        __syncthreads();
      }
      for (uint32_t i = tid; i < rows * wpr; i += kThreads) {
        const uint32_t r = i / wpr, h = i % wpr / wpv, w = i % wpv;
        const int64_t s = layer * p.tl + s_src[r] + h * p.th + static_cast<int64_t>(w) * sizeof(W);
        const int64_t d = layer * p.pool.sl + s_dst[r] + h * p.pool.sh + static_cast<int64_t>(w) * sizeof(W);
        const W kw = ldw<W>(p.kt + s), vw = ldw<W>(p.vt + s);
        stw<W>(p.pool.k + d, kw);
        stw<W>(p.pool.v + d, vw);
      }
    }
  }
  // the sequence's last CTA to have read its length writes the new one
  if (tid == 0) {
    const int arrived = atomicAdd(p.tickets + b, 1);
    if (arrived == p.layers - 1) {
      p.tickets[b] = 0;
      p.len_out[b] = ok ? L + n + 1 : L;
    }
  }
}

// ------------------------------------------------------------------ update

struct PlanHead {              // what the plan leaves for the second kernel
  int32_t fail;                // update: fewer free pages than needed
  int32_t moves;               // compact: pages that move
  int32_t total;               // compact: pages used or pinned
};

struct UpdateParams {
  Pool pool;
  int layers, B_in, B, P, num_pages, W_in, W;
  const int32_t* table; int64_t pt_sb;
  const int32_t* source;
  const int32_t* keep;
  const int32_t* grow;
  const int32_t* pinned;
  int32_t* out; int64_t po_sb;
  int32_t* n_free;
  uint32_t* status;
  // workspace
  uint32_t* read;              // pages that some sequence, or a pin, reads on
  uint32_t* write;             // partly kept last pages that a sequence goes on writing
  int32_t* first;              // [page] the first such sequence (such pages only)
  PlanHead* head;
  int32_t* good;               // [B]
  int32_t* off;                // [B] place of the sequence's fresh pages in the list; bit 31: copies its last page
  int32_t* list;               // [num_pages] free pages, ascending, as many as are needed
};

struct Turn {
  int s, keep, grow;
  int held, want;              // pages kept, pages in all
  bool partial;                // the last kept page is partly kept and will be written
};

__device__ __forceinline__ Turn turn_of(const UpdateParams& p, int b) {
  Turn t;
  t.s = p.source[b];
  t.keep = t.s == -1 ? 0 : p.keep[b];
  t.grow = p.grow[b];
  t.held = t.want = 0;
  t.partial = false;
  return t;
}
__device__ __forceinline__ void turn_pages(const UpdateParams& p, Turn& t) {
  t.held = static_cast<int>((static_cast<int64_t>(t.keep) + p.P - 1) / p.P);
  t.want = static_cast<int>((static_cast<int64_t>(t.keep) + t.grow + p.P - 1) / p.P);
  t.partial = t.keep % p.P != 0 && t.grow > 0;
}

// The status bits of what is wrong with a sequence's numbers.
__device__ __forceinline__ uint32_t check_rows(const UpdateParams& p, const Turn& t) {
  uint32_t bits = 0;
  if (t.s < -1 || t.s >= p.B_in) bits |= TV_DEV_BAD_ROW;
  if (t.keep < 0 || t.grow < 0 || t.keep > static_cast<int64_t>(p.W_in) * p.P ||
      static_cast<int64_t>(t.keep) + t.grow > static_cast<int64_t>(p.W) * p.P)
    bits |= TV_DEV_BAD_LEN;
  return bits;
}

// A warp's check of sequence b, its kept pages too.
__device__ __forceinline__ uint32_t check_turn(const UpdateParams& p, Turn& t, const int32_t* row) {
  const uint32_t bits = check_rows(p, t);
  if (bits) return bits;
  turn_pages(p, t);
  bool bad = false;
  for (int i = threadIdx.x & 31; i < t.held; i += 32) {
    const int page = row[i];
    bad |= page < 0 || page >= p.num_pages;
  }
  return __any_sync(0xffffffffu, bad) ? TV_DEV_BAD_PAGE : 0u;
}

__global__ void __launch_bounds__(kPlanThreads) update_plan_kernel(UpdateParams p) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int slots[3][kPlanCtas];
  const int rank = static_cast<int>(cl.block_rank());
  const int tid = threadIdx.x, lane = tid & 31;
  const int gtid = rank * kPlanThreads + tid, gsize = kPlanCtas * kPlanThreads;
  const int gwarp = gtid >> 5, nwarp = gsize >> 5;
  const int words = (p.num_pages + 31) / 32;
  // 1: the pins, 32 pages to a warp's vote (or nothing), start the bitmap
  for (int w = gwarp; w < words; w += nwarp) {
    const int page = w * 32 + lane;
    const bool pin = p.pinned && page < p.num_pages && p.pinned[page] != 0;
    const unsigned m = __ballot_sync(0xffffffffu, pin);
    if (lane == 0) {
      p.read[w] = m;
      p.write[w] = 0;
    }
  }
  for (int b = gwarp; b < p.B; b += nwarp) {
    Turn t = turn_of(p, b);
    const int32_t* row = p.table + static_cast<int64_t>(max(t.s, 0)) * p.pt_sb;
    const uint32_t bits = check_turn(p, t, row);
    if (lane == 0) {
      p.good[b] = bits == 0;
      set_status(p.status, bits);
      if (!bits && t.partial) p.first[row[t.held - 1]] = 0x7fffffff;
    }
  }
  cl.sync();
  // 2: the kept pages
  for (int b = gwarp; b < p.B; b += nwarp) {
    if (!__ldcg(p.good + b)) continue;
    Turn t = turn_of(p, b);
    turn_pages(p, t);
    const int32_t* row = p.table + static_cast<int64_t>(max(t.s, 0)) * p.pt_sb;
    for (int i = lane; i < t.held; i += 32) {
      const int page = row[i];
      if (t.partial && i == t.held - 1) {
        atomicOr(p.write + (page >> 5), 1u << (page & 31));
        atomicMin(p.first + page, b);
      } else {
        atomicOr(p.read + (page >> 5), 1u << (page & 31));
      }
    }
  }
  cl.sync();
  // 3: every sequence's fresh pages and its place in the list.  CTA r takes
  // sequences [r * per, ...), so the order is that of the sequences.
  const int per = (p.B + kPlanCtas - 1) / kPlanCtas;
  const int blo = min(p.B, rank * per), bhi = min(p.B, blo + per);
  int need = 0;
  for (int b0 = blo; b0 < bhi; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int mine = 0, copies = 0;
    if (b < bhi && __ldcg(p.good + b)) {
      Turn t = turn_of(p, b);
      turn_pages(p, t);
      mine = t.want - t.held;
      if (t.partial) {
        const int page = p.table[static_cast<int64_t>(t.s) * p.pt_sb + t.held - 1];
        copies = ((__ldcg(p.read + (page >> 5)) >> (page & 31)) & 1u) || __ldcg(p.first + page) != b;
        mine += copies;
      }
    }
    int sum;
    const int before = block_scan(mine, &sum);
    if (b < bhi) p.off[b] = (need + before) | (copies ? 0x80000000 : 0);
    need += sum;
  }
  int need_all, free_all;
  const int need0 = cluster_base(cl, slots[0], need, &need_all);
  for (int b = blo + tid; b < bhi; b += kPlanThreads) p.off[b] += need0;
  // 4: the free pages in ascending order, words [r * pw, ...) in CTA r
  const int pw = (words + kPlanCtas - 1) / kPlanCtas;
  const int wlo = min(words, rank * pw), whi = min(words, wlo + pw);
  auto free_word = [&](int w) -> uint32_t {
    uint32_t f = ~(__ldcg(p.read + w) | __ldcg(p.write + w));
    if (w == words - 1 && (p.num_pages & 31)) f &= (1u << (p.num_pages & 31)) - 1u;
    return f;
  };
  int mine = 0, here;
  for (int w = wlo + tid; w < whi; w += kPlanThreads) mine += __popc(free_word(w));
  block_scan(mine, &here);
  int at0 = cluster_base(cl, slots[1], here, &free_all);
  for (int w0 = wlo; w0 < whi && at0 < need_all; w0 += kPlanThreads) {
    const int w = w0 + tid;
    uint32_t f = w < whi ? free_word(w) : 0u;
    int sum;
    int at = at0 + block_scan(__popc(f), &sum);
    while (f && at < need_all) {
      p.list[at++] = w * 32 + __ffs(f) - 1;
      f &= f - 1u;
    }
    at0 += sum;
  }
  if (gtid == 0) {
    p.head->fail = need_all > free_all;
    if (need_all > free_all) set_status(p.status, TV_DEV_NO_PAGES);
    if (p.n_free) *p.n_free = free_all - need_all;
  }
  cl.sync();                                     // no CTA's shared memory goes while a peer may post to it
}

// CTA (b, layer): the row of the new table (layer 0), and the kept rows of a
// last page that b may not write into.
template <typename W>
__global__ void __launch_bounds__(kThreads) update_apply_kernel(UpdateParams p) {
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const bool live = p.good[b] && !p.head->fail;
  Turn t = turn_of(p, b);
  if (live) turn_pages(p, t);
  const int32_t* row = p.table + static_cast<int64_t>(max(t.s, 0)) * p.pt_sb;
  const int at = p.off[b] & 0x7fffffff;
  const bool copies = live && p.off[b] < 0;
  if (layer == 0) {
    const int fresh0 = t.held - (copies ? 1 : 0);      // first position of a fresh page
    for (int i = tid; i < p.W; i += kThreads) {
      int page = -1;
      if (live && i < t.want) page = i < fresh0 ? row[i] : p.list[at + i - fresh0];
      p.out[b * p.po_sb + i] = page;
    }
  }
  if (copies && layer < p.layers) {
    const int wpr = p.pool.Hkv * p.pool.vec_bytes / static_cast<int>(sizeof(W));
    copy_words<W, kThreads>(p.pool, layer * p.pool.sl + p.list[at] * p.pool.sp, layer * p.pool.sl + row[t.held - 1] * p.pool.sp,
                  0, t.keep % p.P * wpr);
  }
}

// The whole update in one kernel, for small pools: every CTA plans, then takes
// its share of the new table's rows and of the copies' slices.
template <typename W>
__global__ void __launch_bounds__(kSmallThreads) update_small_kernel(UpdateParams p) {
  constexpr int NT = kSmallThreads;
  extern __shared__ uint32_t dyn[];
  const int words = (p.num_pages + 31) / 32;
  uint32_t* read = dyn;                          // as in UpdateParams
  uint32_t* write = read + words;
  int* before = reinterpret_cast<int*>(write + words);   // free pages below a word
  __shared__ Turn s_turn[kSmallSeqs];
  __shared__ uint32_t s_bits[kSmallSeqs];        // what is wrong with the sequence
  __shared__ int s_page[kSmallSeqs];             // the last page, where it is partly kept; -1
  __shared__ int s_off[kSmallSeqs];              // place of the sequence's fresh pages
  __shared__ int s_first[kSmallSeqs], s_list[kSmallSeqs];
  __shared__ uint8_t s_copies[kSmallSeqs];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < p.B) {
    Turn t = turn_of(p, tid);
    uint32_t bits = check_rows(p, t);
    if (!bits) turn_pages(p, t);
    s_turn[tid] = t;
    s_bits[tid] = bits;
  }
  // Mark the kept pages, all entries at once.  A bad page among them shows
  // only here; its sequence keeps nothing, so the marks are made again
  // without it (one round where there is none).
  int again = 0;
  do {
    for (int w = tid; w < words; w += NT) write[w] = 0;
    for (int w = warp; w < words; w += NT / 32) {
      const int page = w * 32 + lane;
      const unsigned m = __ballot_sync(0xffffffffu, p.pinned && page < p.num_pages && p.pinned[page] != 0);
      if (lane == 0) read[w] = m;
    }
    if (tid < p.B) {
      if (s_bits[tid]) {
        s_turn[tid].held = s_turn[tid].want = 0;
        s_turn[tid].partial = false;
      }
      s_page[tid] = -1;
    }
    __syncthreads();
    int bad = 0;
    for_entries<NT>(
        p.B, [&](int b) { return s_turn[b].held; },
        [&](int b) { return p.table + static_cast<int64_t>(max(s_turn[b].s, 0)) * p.pt_sb; },
        [&](int b, int i, int page) {
          if (page < 0 || page >= p.num_pages) {
            s_bits[b] = TV_DEV_BAD_PAGE;
            bad = 1;
          } else if (i == s_turn[b].held - 1 && s_turn[b].partial) {
            atomicOr(write + (page >> 5), 1u << (page & 31));
            s_page[b] = page;
          } else {
            atomicOr(read + (page >> 5), 1u << (page & 31));
          }
        });
    again = __syncthreads_or(bad);
  } while (again);
  if (blockIdx.x == 0 && tid < p.B) set_status(p.status, s_bits[tid]);
  // the first sequence that writes into each partly kept page: such pages
  // are numbered by their bits' ranks, one for a sequence at most
  for (int w = tid; w < words; w += NT) before[w] = __popc(write[w]);
  if (tid < p.B) s_first[tid] = p.B;
  __syncthreads();
  scan_array<NT>(before, words);
  int* first = nullptr;
  bool copies = false;                           // others read on in my last page, or an earlier sequence writes in it
  if (tid < p.B && s_page[tid] >= 0) {
    const int w = s_page[tid] >> 5, bit = s_page[tid] & 31;
    first = s_first + before[w] + __popc(write[w] & ((1u << bit) - 1u));
    atomicMin(first, tid);
    copies = (read[w] >> bit) & 1u;
  }
  __syncthreads();
  if (first) copies = copies || *first != tid;
  int demand = 0;
  if (tid < p.B) demand = s_turn[tid].want - s_turn[tid].held + (copies ? 1 : 0);
  int need;
  const int off = block_scan<NT>(demand, &need);
  int n_copies;
  const int k = block_scan<NT>(copies ? 1 : 0, &n_copies);
  if (tid < p.B) {
    s_off[tid] = off;
    s_copies[tid] = copies;
    if (copies) s_list[k] = tid;
  }
  auto free_word = [&](int w) -> uint32_t {
    uint32_t f = ~(read[w] | write[w]);
    if (w == words - 1 && (p.num_pages & 31)) f &= (1u << (p.num_pages & 31)) - 1u;
    return f;
  };
  for (int w = tid; w < words; w += NT) before[w] = __popc(free_word(w));
  __syncthreads();
  const int free_pages = scan_array<NT>(before, words);
  const bool fail = need > free_pages;
  if (blockIdx.x == 0 && tid == 0) {
    if (fail) set_status(p.status, TV_DEV_NO_PAGES);
    if (p.n_free) *p.n_free = free_pages - need;
  }
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const Turn t = s_turn[b];
    const int32_t* row = p.table + static_cast<int64_t>(max(t.s, 0)) * p.pt_sb;
    const int fresh0 = t.held - s_copies[b];     // first position of a fresh page
    for (int i = tid; i < p.W; i += NT) {
      int page = -1;
      if (!fail && i < t.want) page = i < fresh0 ? row[i] : select_bit(before, words, s_off[b] + i - fresh0, free_word);
      p.out[b * p.po_sb + i] = page;
    }
  }
  if (fail) return;
  const uint32_t wpr = page_words<W>(p.pool, 1);   // words of a row
  const int slices = small_slices(p.P, wpr);
  const int64_t jobs = static_cast<int64_t>(n_copies) * p.layers * slices;
  for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int64_t k = j / slices;                // the copy's layer
    const int b = s_list[k / p.layers], layer = static_cast<int>(k % p.layers);
    const uint32_t w0 = static_cast<uint32_t>(j % slices) * kSmallSlice;
    copy_words<W, NT>(p.pool, layer * p.pool.sl + select_bit(before, words, s_off[b], free_word) * p.pool.sp,
                      layer * p.pool.sl + s_page[b] * p.pool.sp, w0,
                      min(s_turn[b].keep % p.P * wpr, w0 + kSmallSlice));
  }
}

// ------------------------------------------------------------------ compact

struct CompactParams {
  Pool pool;
  int layers, B, P, num_pages, W;
  const int32_t* table; int64_t pt_sb;
  const int32_t* length;
  const int32_t* pinned;
  int32_t* out; int64_t po_sb;
  int32_t* n_used;
  uint32_t* status;
  // workspace
  uint32_t* used;
  uint32_t* pin;
  PlanHead* head;
  int32_t* from;               // [num_pages] pages that move, ascending
  int32_t* to;                 // [num_pages] where they go (the holes, ascending)
  int32_t* name;               // [num_pages] new index of a used page past the packed end
};

__device__ __forceinline__ int used_entries(const CompactParams& p, int len) {
  const int64_t cap = static_cast<int64_t>(p.W) * p.P;
  const int64_t n = len < 0 ? 0 : (len > cap ? cap : len);
  return static_cast<int>((n + p.P - 1) / p.P);
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(CompactParams p) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int slots[3][kPlanCtas];
  const int rank = static_cast<int>(cl.block_rank());
  const int tid = threadIdx.x, lane = tid & 31;
  const int gtid = rank * kPlanThreads + tid, gsize = kPlanCtas * kPlanThreads;
  const int gwarp = gtid >> 5, nwarp = gsize >> 5;
  const int words = (p.num_pages + 31) / 32;
  for (int w = gwarp; w < words; w += nwarp) {
    const int page = w * 32 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, p.pinned && page < p.num_pages && p.pinned[page] != 0);
    if (lane == 0) {
      p.used[w] = 0;
      p.pin[w] = m;
    }
  }
  cl.sync();
  for (int b = gwarp; b < p.B; b += nwarp) {
    const int len = p.length[b];
    uint32_t bits = 0;
    if (len < 0 || len > static_cast<int64_t>(p.W) * p.P) bits |= TV_DEV_BAD_LEN;
    const int held = used_entries(p, len);
    for (int i = lane; i < held; i += 32) {
      const int page = p.table[b * p.pt_sb + i];
      if (page < 0 || page >= p.num_pages) bits |= TV_DEV_BAD_PAGE;
      else atomicOr(p.used + (page >> 5), 1u << (page & 31));
    }
    set_status(p.status, bits);
  }
  cl.sync();
  // CTA r takes words [r * pw, ...): the pages that stay or move, then the
  // holes below the packed end, then the pages above it
  const int pw = (words + kPlanCtas - 1) / kPlanCtas;
  const int wlo = min(words, rank * pw), whi = min(words, wlo + pw);
  int mine = 0, here, total;
  for (int w = wlo + tid; w < whi; w += kPlanThreads) mine += __popc(__ldcg(p.used + w) | __ldcg(p.pin + w));
  block_scan(mine, &here);
  cluster_base(cl, slots[0], here, &total);
  auto below = [&](int w) -> uint32_t {            // bits of word w that lie below `total`
    return w * 32 + 32 <= total ? 0xffffffffu : (w * 32 >= total ? 0u : (1u << (total - w * 32)) - 1u);
  };
  int holes = 0, moves = 0;
  for (int w = wlo + tid; w < whi; w += kPlanThreads) {
    const uint32_t u = __ldcg(p.used + w), pin = __ldcg(p.pin + w);
    holes += __popc(~(u | pin) & below(w));
    moves += __popc(u & ~pin & ~below(w));
  }
  int holes_here, moves_here, holes_all, moves_all;
  block_scan(holes, &holes_here);
  block_scan(moves, &moves_here);
  int hat = cluster_base(cl, slots[1], holes_here, &holes_all);
  int mat = cluster_base(cl, slots[2], moves_here, &moves_all);
  for (int w0 = wlo; w0 < whi; w0 += kPlanThreads) {
    const int w = w0 + tid;
    uint32_t f = w < whi ? ~(__ldcg(p.used + w) | __ldcg(p.pin + w)) & below(w) : 0u;
    int sum;
    int at = hat + block_scan(__popc(f), &sum);
    while (f) {
      p.to[at++] = w * 32 + __ffs(f) - 1;
      f &= f - 1u;
    }
    hat += sum;
  }
  cl.sync();                                       // the list of holes is whole
  for (int w0 = wlo; w0 < whi; w0 += kPlanThreads) {
    const int w = w0 + tid;
    uint32_t u = 0, pin = 0;
    if (w < whi) {
      u = __ldcg(p.used + w) & ~below(w);
      pin = __ldcg(p.pin + w);
    }
    int sum;
    int at = mat + block_scan(__popc(u & ~pin), &sum);
    while (u) {
      const int bit = __ffs(u) - 1, page = w * 32 + bit;
      if ((pin >> bit) & 1u) {
        p.name[page] = page;
      } else {
        p.from[at] = page;
        p.name[page] = __ldcg(p.to + at);
        ++at;
      }
      u &= u - 1u;
    }
    mat += sum;
  }
  if (gtid == 0) {
    p.head->moves = moves_all;
    p.head->total = total;
    if (p.n_used) *p.n_used = total;
  }
}

// The tables' new names, then the pages, split over the grid in slices of
// kSliceWords words of a page of one layer.
constexpr uint32_t kSliceWords = 4 * kThreads;

template <typename W>
__global__ void __launch_bounds__(kThreads) compact_apply_kernel(CompactParams p) {
  const int total = p.head->total, moves = p.head->moves;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int held = used_entries(p, p.length[b]);
    for (int i = threadIdx.x; i < p.W; i += kThreads) {
      int page = -1;
      if (i < held) {
        page = p.table[b * p.pt_sb + i];
        if (page >= total && page < p.num_pages) page = p.name[page];
      }
      p.out[b * p.po_sb + i] = page;
    }
  }
  const uint32_t words = page_words<W>(p.pool, p.P);
  const int slices = static_cast<int>((words + kSliceWords - 1) / kSliceWords);
  const int64_t jobs = static_cast<int64_t>(moves) * p.layers * slices;
  for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int64_t k = j / slices;                // the move's layer
    const int m = static_cast<int>(k / p.layers), layer = static_cast<int>(k % p.layers);
    const uint32_t w0 = static_cast<uint32_t>(j % slices) * kSliceWords;
    copy_words<W, kThreads>(p.pool, layer * p.pool.sl + p.to[m] * p.pool.sp, layer * p.pool.sl + p.from[m] * p.pool.sp, w0,
                  min(words, w0 + kSliceWords));
  }
}

// The whole compaction in one kernel, for small pools: every CTA plans, then
// takes its share of the table rows and of the moves' slices.
template <typename W>
__global__ void __launch_bounds__(kSmallThreads) compact_small_kernel(CompactParams p) {
  constexpr int NT = kSmallThreads;
  extern __shared__ uint32_t dyn[];
  const int words = (p.num_pages + 31) / 32;
  uint32_t* used = dyn;
  uint32_t* pin = used + words;
  int* holes = reinterpret_cast<int*>(pin + words);      // holes, moves before a word
  int* moves = holes + words;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int w = warp; w < words; w += NT / 32) {
    const int page = w * 32 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, p.pinned && page < p.num_pages && p.pinned[page] != 0);
    if (lane == 0) {
      used[w] = 0;
      pin[w] = m;
    }
  }
  __syncthreads();
  __shared__ int s_held[kSmallSeqs];
  if (tid < p.B) {
    const int len = p.length[tid];
    s_held[tid] = used_entries(p, len);
    if (blockIdx.x == 0 && (len < 0 || len > static_cast<int64_t>(p.W) * p.P)) set_status(p.status, TV_DEV_BAD_LEN);
  }
  __syncthreads();
  const int entries = p.B * p.W;
  uint32_t bits = 0;
  for_entries<NT>(
      p.B, [&](int b) { return s_held[b]; }, [&](int b) { return p.table + b * p.pt_sb; },
      [&](int, int, int page) {
        if (page < 0 || page >= p.num_pages) bits = TV_DEV_BAD_PAGE;
        else atomicOr(used + (page >> 5), 1u << (page & 31));
      });
  if (blockIdx.x == 0) set_status(p.status, bits);
  __syncthreads();
  int mine = 0, total;
  for (int w = tid; w < words; w += NT) mine += __popc(used[w] | pin[w]);
  block_scan<NT>(mine, &total);
  auto below = [&](int w) -> uint32_t {          // bits of word w that lie below `total`
    return w * 32 + 32 <= total ? 0xffffffffu : (w * 32 >= total ? 0u : (1u << (total - w * 32)) - 1u);
  };
  auto hole_word = [&](int w) -> uint32_t { return ~(used[w] | pin[w]) & below(w); };
  auto move_word = [&](int w) -> uint32_t { return used[w] & ~pin[w] & ~below(w); };
  for (int w = tid; w < words; w += NT) {
    holes[w] = __popc(hole_word(w));
    moves[w] = __popc(move_word(w));
  }
  __syncthreads();
  scan_array<NT>(holes, words);
  const int n = scan_array<NT>(moves, words);
  if (blockIdx.x == 0 && tid == 0 && p.n_used) *p.n_used = total;
  for (int e = blockIdx.x * NT + tid; e < entries; e += gridDim.x * NT) {
    const int b = e / p.W, i = e - b * p.W;
    int page = -1;
    if (i < s_held[b]) {
      page = p.table[b * p.pt_sb + i];
      if (page >= total && page < p.num_pages && !((pin[page >> 5] >> (page & 31)) & 1u)) {
        const int k = moves[page >> 5] + __popc(move_word(page >> 5) & ((1u << (page & 31)) - 1u));
        page = select_bit(holes, words, k, hole_word);
      }
    }
    p.out[b * p.po_sb + i] = page;
  }
  const uint32_t wpp = page_words<W>(p.pool, p.P);
  const int slices = static_cast<int>((wpp + kSmallSlice - 1) / kSmallSlice);
  const int64_t jobs = static_cast<int64_t>(n) * p.layers * slices;
  for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int64_t k = j / slices;                // the move's layer
    const int m = static_cast<int>(k / p.layers), layer = static_cast<int>(k % p.layers);
    const uint32_t w0 = static_cast<uint32_t>(j % slices) * kSmallSlice;
    const int from = select_bit(moves, words, m, move_word), to = select_bit(holes, words, m, hole_word);
    copy_words<W, NT>(p.pool, layer * p.pool.sl + to * p.pool.sp, layer * p.pool.sl + from * p.pool.sp, w0,
                      min(wpp, w0 + kSmallSlice));
  }
}

// ------------------------------------------------------------------ host side

namespace {

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Widest word that every base and every stride (bytes) and the vector allow.
int word_bytes(std::initializer_list<const void*> bases, std::initializer_list<int64_t> strides) {
  for (int w : {16, 4}) {
    bool ok = true;
    for (const void* b : bases) ok = ok && reinterpret_cast<uintptr_t>(b) % w == 0;
    for (int64_t s : strides) ok = ok && s % w == 0;
    if (ok) return w;
  }
  return 2;
}

template <typename A>
Pool make_pool(const A* a) {
  const int es = a->dtype == TV_BF16 ? 2 : 4;
  Pool p;
  p.k = static_cast<char*>(a->k_pages);
  p.v = static_cast<char*>(a->v_pages);
  p.sl = a->kv_sl * es; p.sp = a->kv_sp * es; p.sr = a->kv_sr * es; p.sh = a->kv_sh * es;
  p.Hkv = a->Hkv;
  p.vec_bytes = a->d * es;
  p.dense = p.sh == p.vec_bytes && p.sr == static_cast<int64_t>(p.Hkv) * p.vec_bytes;
  return p;
}

struct Carve {
  unsigned char* base;
  size_t off;
  template <typename T>
  T* take(size_t n) {
    T* r = reinterpret_cast<T*>(base + off);
    off = up256(off + n * sizeof(T));
    return r;
  }
};

}  // namespace

namespace {

size_t carve_update(unsigned char* ws, int B, int num_pages, UpdateParams& u) {
  Carve c{ws, kTicketBytes};
  const size_t words = (static_cast<size_t>(num_pages) + 31) / 32;
  u.read = c.take<uint32_t>(words);
  u.write = c.take<uint32_t>(words);
  u.first = c.take<int32_t>(num_pages);
  u.head = c.take<PlanHead>(1);
  u.good = c.take<int32_t>(B);
  u.off = c.take<int32_t>(B);
  u.list = c.take<int32_t>(num_pages);
  return c.off;
}

size_t carve_compact(unsigned char* ws, int num_pages, CompactParams& u) {
  Carve c{ws, kTicketBytes};
  const size_t words = (static_cast<size_t>(num_pages) + 31) / 32;
  u.used = c.take<uint32_t>(words);
  u.pin = c.take<uint32_t>(words);
  u.head = c.take<PlanHead>(1);
  u.from = c.take<int32_t>(num_pages);
  u.to = c.take<int32_t>(num_pages);
  u.name = c.take<int32_t>(num_pages);
  return c.off;
}

template <typename P>
cudaError_t launch_plan(void (*kernel)(P), const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

int num_sms();

namespace {
bool small_pool(int B, int64_t entries, int num_pages) {
  return B <= kSmallSeqs && entries <= kSmallEntries && num_pages <= kSmallPages;
}
}  // namespace

size_t commit_paged_workspace_bytes() { return kTicketBytes; }
size_t pages_update_workspace_bytes(int B, int num_pages) {
  UpdateParams u;
  return carve_update(nullptr, B, num_pages, u);
}
size_t pages_compact_workspace_bytes(int num_pages) {
  CompactParams u;
  return carve_compact(nullptr, num_pages, u);
}

cudaError_t launch_commit_paged(const tv_commit_paged_args* a, void* ws, cudaStream_t stream) {
  const int es = a->dtype == TV_BF16 ? 2 : 4;
  CommitPagedParams p;
  p.pool = make_pool(a);
  p.layers = a->layers; p.B = a->B; p.T = a->T; p.P = a->page_size; p.num_pages = a->num_pages;
  p.cap = std::min<int64_t>(static_cast<int64_t>(a->max_pages) * a->page_size, INT32_MAX);   // (a length is an int32)
  p.table = a->page_table; p.pt_sb = a->pt_sb;
  p.len = a->prefix_len;
  p.len_out = a->prefix_len_out;
  p.kt = static_cast<const char*>(a->k_tree);
  p.vt = static_cast<const char*>(a->v_tree);
  p.tl = a->kt_sl * es; p.tb = a->kt_sb * es; p.tt = a->kt_st * es; p.th = a->kt_sh * es;
  p.n_acc = a->n_accepted;
  p.acc = a->accepted_nodes; p.acc_sb = a->acc_sb;
  p.tickets = static_cast<int32_t*>(ws);
  p.status = a->dev_status;
  const Pool& o = p.pool;
  const dim3 grid(static_cast<unsigned>(a->B), static_cast<unsigned>(a->layers));
  const int w = word_bytes({o.k, o.v, p.kt, p.vt}, {o.sl, o.sp, o.sr, o.sh, o.vec_bytes, p.tl, p.tb, p.tt, p.th});
  p.step = static_cast<int>(std::min<int64_t>(kCommitRows, INT32_MAX / (static_cast<int64_t>(a->Hkv) * (o.vec_bytes / w))));
  switch (w) {
    case 16: commit_paged_kernel<uint4><<<grid, kThreads, 0, stream>>>(p); break;
    case 4: commit_paged_kernel<uint32_t><<<grid, kThreads, 0, stream>>>(p); break;
    default: commit_paged_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_pages_update(const tv_pages_update_args* a, void* ws, cudaStream_t stream) {
  UpdateParams p;
  p.pool = make_pool(a);
  p.layers = a->layers; p.B_in = a->B_in; p.B = a->B; p.P = a->page_size; p.num_pages = a->num_pages;
  p.W_in = a->max_pages_in; p.W = a->max_pages;
  p.table = a->page_table; p.pt_sb = a->pt_sb;
  p.source = a->source; p.keep = a->keep; p.grow = a->grow; p.pinned = a->pinned;
  p.out = a->page_table_out; p.po_sb = a->po_sb;
  p.n_free = a->n_free;
  p.status = a->dev_status;
  if (small_pool(a->B, static_cast<int64_t>(a->B) * a->max_pages_in, a->num_pages)) {
    const int w = word_bytes({p.pool.k, p.pool.v}, {p.pool.sl, p.pool.sp, p.pool.sr, p.pool.sh, p.pool.vec_bytes});
    const size_t smem = static_cast<size_t>((a->num_pages + 31) / 32) * 12;
    // a CTA for every row and every slice that can be copied, two to an SM at most
    const int64_t jobs = static_cast<int64_t>(a->B) * a->layers * small_slices(a->page_size, a->Hkv * (p.pool.vec_bytes / w));
    const int grid = static_cast<int>(std::min<int64_t>(std::max<int64_t>(jobs, std::max(1, a->B)), 2 * num_sms()));
    switch (w) {
      case 16: update_small_kernel<uint4><<<grid, kSmallThreads, smem, stream>>>(p); break;
      case 4: update_small_kernel<uint32_t><<<grid, kSmallThreads, smem, stream>>>(p); break;
      default: update_small_kernel<uint16_t><<<grid, kSmallThreads, smem, stream>>>(p); break;
    }
    return cudaGetLastError();
  }
  carve_update(static_cast<unsigned char*>(ws), a->B, a->num_pages, p);
  cudaError_t e = launch_plan(update_plan_kernel, p, stream);
  if (e != cudaSuccess || a->B == 0) return e;
  const Pool& o = p.pool;
  const dim3 grid(static_cast<unsigned>(a->B), static_cast<unsigned>(a->layers > 0 ? a->layers : 1));
  switch (word_bytes({o.k, o.v}, {o.sl, o.sp, o.sr, o.sh, o.vec_bytes})) {
    case 16: update_apply_kernel<uint4><<<grid, kThreads, 0, stream>>>(p); break;
    case 4: update_apply_kernel<uint32_t><<<grid, kThreads, 0, stream>>>(p); break;
    default: update_apply_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const tv_pages_compact_args* a, void* ws, cudaStream_t stream) {
  CompactParams p;
  p.pool = make_pool(a);
  p.layers = a->layers; p.B = a->B; p.P = a->page_size; p.num_pages = a->num_pages; p.W = a->max_pages;
  p.table = a->page_table; p.pt_sb = a->pt_sb;
  p.length = a->length; p.pinned = a->pinned;
  p.out = a->page_table_out; p.po_sb = a->po_sb;
  p.n_used = a->n_used;
  p.status = a->dev_status;
  // (in place the table may not change while another CTA still plans from it)
  if (a->page_table_out != a->page_table &&
      small_pool(a->B, static_cast<int64_t>(a->B) * a->max_pages, a->num_pages)) {
    const size_t smem = static_cast<size_t>((a->num_pages + 31) / 32) * 16;
    const int w = word_bytes({p.pool.k, p.pool.v}, {p.pool.sl, p.pool.sp, p.pool.sr, p.pool.sh, p.pool.vec_bytes});
    // at most half of the pages can move
    const int64_t most = static_cast<int64_t>(a->num_pages) / 2 * a->layers * a->page_size * a->Hkv * (p.pool.vec_bytes / w);
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most / (4 * kSmallThreads) + 1, 2 * num_sms())));
    switch (w) {
      case 16: compact_small_kernel<uint4><<<grid, kSmallThreads, smem, stream>>>(p); break;
      case 4: compact_small_kernel<uint32_t><<<grid, kSmallThreads, smem, stream>>>(p); break;
      default: compact_small_kernel<uint16_t><<<grid, kSmallThreads, smem, stream>>>(p); break;
    }
    return cudaGetLastError();
  }
  carve_compact(static_cast<unsigned char*>(ws), a->num_pages, p);
  cudaError_t e = launch_plan(compact_plan_kernel, p, stream);
  if (e != cudaSuccess) return e;
  const Pool& o = p.pool;
  const int grid = 8 * num_sms();
  switch (word_bytes({o.k, o.v}, {o.sl, o.sp, o.sr, o.sh, o.vec_bytes})) {
    case 16: compact_apply_kernel<uint4><<<grid, kThreads, 0, stream>>>(p); break;
    case 4: compact_apply_kernel<uint32_t><<<grid, kThreads, 0, stream>>>(p); break;
    default: compact_apply_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace tv
