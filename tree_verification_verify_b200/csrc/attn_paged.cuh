// Shared parts of the paged tree attention kernels (tree_verify_attn_paged):
// the parameters, the split of the work over the CTAs and the merge of
// partial rows.
//
// The split.  A unit is (sequence, kv head, row tile of packed (node, head)
// rows); its key tiles are the prefix tiles of its sequence, then the tree
// tiles.  All units' key tiles lie in one line, sequence by sequence, and
// each CTA of a grid of about one CTA per SM takes an equal stretch of it:
// a piece of a unit at either end, whole units between.  Behind its tiles a
// unit has COST more places with nothing in them, as many as tiles could run
// in the time that a kernel loses at the border of units.  Where a stretch is
// shorter than four tiles that is too coarse: there every unit begins a
// stretch of its own, if the stretches suffice for that or do when they are
// one tile longer (one sequence of 4096 rows and 64 nodes: 33 us, so 28).  (Where sequences
// have several row tiles on the tensor cores, a team of CTAs takes a stretch
// together, a row tile each, so that they read the same keys at the same
// time and all but one find them in the L2.)  The line's length
// and every CTA's stretch follow from prefix_len and n_nodes on the device,
// so ragged batches are balanced to one tile, a long table costs nothing,
// and a single long sequence fills the GPU.  A unit that crosses stretches
// leaves one normalised partial and a log-sum-exp per piece in the workspace,
// and its first CTA a note of where they are; a second kernel, a warp per
// row, combines them in piece order.  (The last CTA of a unit to finish did
// that at first: 28 us for 128 rows of 9 pieces, where each of the warp's
// dependent reads of another SM's fresh rows took about 1 us; spread over
// the GPU it is a few us.)
#pragma once

#include "tv_common.cuh"

namespace tv {

struct PagedAttnParams {
  int dtype;
  int B, T, Hq, Hkv, d, G;
  int num_pages, page_size, max_pages;
  const void* q;  int64_t q_sb, q_st, q_sh;
  const void* kp; const void* vp; int64_t kv_sp, kv_sr, kv_sh;
  const int32_t* table; int64_t pt_sb;
  const int32_t* prefix_len;
  const void* kt; const void* vt; int64_t kt_sb, kt_st, kt_sh;
  const int32_t* parent; int64_t par_sb;
  const int32_t* n_nodes;
  float scale;
  void* out; int64_t o_sb, o_st, o_sh;
  float* lse;
  uint32_t* status;
  int prefix_only;
  int rows;                    // query rows of a unit
  int team;                    // CTAs that share a stretch, each with one row tile of its units
  int box;                     // tensor cores: rows of a page that one TMA box takes (0: row by row)
  int lost;                    // tensor cores, a test hook: 1 no piece after a CTA's first comes, 2 no product
  float* part_o;               // [stretch][2][rows][d]: the piece that continues a unit, the one that begins one
  float* part_lse;             // [stretch][2][rows], log2 units
  struct SplitUnit* splits;    // [stretch] the unit that begins in it and ends in a later one
};

// A unit in pieces: it begins in stretch c0 (the second slot) and goes on in
// c0 + 1 .. c1 (their first); c1 < 0: none.
struct SplitUnit {
  int32_t c1, b, g, packed0, rows;
};

namespace paged {

// Sequence b's share of the line.
struct SeqInfo {
  int n;                       // nodes with rows (0: none)
  int L;                       // prefix rows (0 when prefix_len is out of range)
  bool bad_len;
  int nprefix, ntree;          // key tiles of a unit
  int rem, off;                // the prefix's last rem rows share the one tree tile, whose nodes begin at row off
  int tiles;                   // max(1, nprefix + ntree): a unit without keys still writes its rows
  int units;                   // row tiles * kv heads
};

// align > 0: the prefix's rows past its whole tiles and a tree of at most one
// tile go into one tile where they fit (nodes at a multiple of align).
template <int KEYS>
__device__ __forceinline__ SeqInfo seq_info(const PagedAttnParams& p, int b, int align) {
  SeqInfo s;
  const int n = p.n_nodes ? p.n_nodes[b] : p.T;
  const int L = p.prefix_len[b];
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  s.n = (n < 0 || n > p.T) ? 0 : n;
  s.bad_len = L < 0 || L > cap;
  s.L = s.bad_len ? 0 : L;
  s.nprefix = static_cast<int>((static_cast<unsigned>(s.L) + KEYS - 1) / KEYS);
  s.ntree = p.prefix_only ? 0 : (s.n + KEYS - 1) / KEYS;
  s.rem = s.off = 0;
  const int rem = s.L % KEYS, off = align > 0 ? (rem + align - 1) / align * align : 0;
  if (align > 0 && s.ntree == 1 && rem > 0 && off + s.n <= KEYS) {
    --s.nprefix;
    s.rem = rem;
    s.off = off;
  }
  s.tiles = max(1, s.nprefix + s.ntree);
  s.units = (s.n * p.G + p.rows - 1) / p.rows * p.Hkv;
  return s;
}

__device__ __forceinline__ int round_up(int x, int m) { return (x + m - 1) / m * m; }

constexpr int kMaxSlots = 512;

// The line's prefix sums: slot t holds sequences [t * per, (t + 1) * per).
struct Line {
  int cum[kMaxSlots + 1];      // (the host refuses lines of 2^31 places)
  int warp_sum[32], warp_units[32];
  int cost, pad;               // a unit has its tiles, rounded up to `pad`, and `cost` more places
  int per;                     // sequences per slot
  int nslot;
  int first, last;             // this CTA's stretch
  int step;                    // places of a stretch
  int stretch;                 // this CTA's
};

// Places of a unit.
__device__ __forceinline__ int places(int tiles, const Line& ln) {
  return (ln.pad == 1 ? tiles : round_up(tiles, ln.pad)) + ln.cost;
}

// Called by all NT threads of the CTA (NT <= kMaxSlots, a multiple of 32).
template <int KEYS, int COST, int NT>
__device__ __forceinline__ void build_line(const PagedAttnParams& p, Line& ln, int align) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + NT - 1) / NT;
  const int stretches = static_cast<int>(gridDim.x) / p.team;
  // exclusive sums over the threads, and the totals
  int before, before_u, sum, sum_u;
  auto scan = [&](int v, int u) {
    int incl = v, incl_u = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o), tu = __shfl_up_sync(0xffffffffu, incl_u, o);
      if (lane >= o) {
        incl += t;
        incl_u += tu;
      }
    }
    if (lane == 31) {
      ln.warp_sum[warp] = incl;
      ln.warp_units[warp] = incl_u;
    }
    __syncthreads();
    before = incl - v;
    before_u = incl_u - u;
    sum = sum_u = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const int t = ln.warp_sum[w], tu = ln.warp_units[w];
      before += w < warp ? t : 0;
      before_u += w < warp ? tu : 0;
      sum += t;
      sum_u += tu;
    }
  };
  int v = 0, u = 0;                                // tiles, units
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= p.B) break;
    const SeqInfo s = seq_info<KEYS>(p, b, align);
    v += s.units * s.tiles;
    u += s.units;
    if (blockIdx.x == 0 && p.n_nodes) {
      const int n = p.n_nodes[b];
      if (n < 0 || n > p.T) set_status(p.status, TV_DEV_BAD_LEN);
    }
    if (blockIdx.x == 0 && s.bad_len && s.n > 0) set_status(p.status, TV_DEV_BAD_LEN);
  }
  scan(v, u);
  const bool brief = sum / 4 < stretches;          // stretches of up to four tiles
  const int cost = brief ? 0 : COST;
  int cum = before + cost * before_u, total = sum + cost * sum_u, pad = 1;
  if (brief && sum > stretches) {
    const int step = 2 + (sum > 2 * stretches) + (sum > 3 * stretches);
    v = u = 0;                                     // places with the units' tiles rounded up to step, to step + 1
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= p.B) break;
      const SeqInfo s = seq_info<KEYS>(p, b, align);
      v += s.units * round_up(s.tiles, step);
      u += s.units * round_up(s.tiles, step + 1);
    }
    __syncthreads();                               // the sums have been read
    scan(v, u);
    if (sum <= step * stretches) {
      cum = before;
      total = sum;
      pad = step;
    } else if (sum_u <= (step + 1) * stretches) {
      cum = before_u;
      total = sum_u;
      pad = step + 1;
    }
  }
  ln.cum[tid] = cum;
  if (tid == 0) {
    ln.cum[NT] = total;
    ln.per = per;
    ln.nslot = NT;
    ln.cost = cost;
    ln.pad = pad;
    const int c = static_cast<int>(blockIdx.x) / p.team;
    const int step = pad > 1 ? pad : max(1, (total + stretches - 1) / stretches);
    ln.step = step;
    ln.stretch = c;
    ln.first = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(step) * c));
    ln.last = ln.first + min(step, total - ln.first);
  }
  __syncthreads();
  // the merge kernel's CTAs may take the places of CTAs that end from here on
  asm volatile("griddepcontrol.launch_dependents;");
}

// One piece: key tiles [t0, t1) of a unit.
struct Piece {
  int b, g, rt;
  SeqInfo s;
  int t0, t1;                  // (t0 >= t1: only places behind the unit's tiles)
  int next;                    // the place after the piece
  int unit_first;              // the unit's first place
};

// The piece that begins at `pos` (ln.first <= pos < ln.last).
template <int KEYS>
__device__ __forceinline__ Piece piece_at(const PagedAttnParams& p, const Line& ln, int pos, int align) {
  int lo = 0, hi = min(ln.nslot, p.B);             // last slot whose sum is <= pos: the one that holds pos
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ln.cum[mid] <= pos) lo = mid; else hi = mid;
  }
  Piece c;
  int base = ln.cum[lo];
  int b = lo * ln.per;
#pragma unroll 1
  for (int i = 0; i < ln.per; ++i, ++b) {          // one step when B is at most the thread count
    c.s = seq_info<KEYS>(p, b, align);
    const int w = c.s.units * places(c.s.tiles, ln);
    if (pos < base + w) break;
    base += w;
  }
  c.b = b;
  const int off = pos - base;
  const int len = places(c.s.tiles, ln);
  const int u = off / len;
  c.t0 = off - u * len;
  const int left = min(len - c.t0, ln.last - pos);
  c.t1 = min(c.s.tiles, c.t0 + left);
  c.next = pos + left;
  const int nrt = c.s.units / p.Hkv;
  c.g = u / nrt;
  c.rt = u - c.g * nrt;
  c.unit_first = pos - c.t0;
  return c;
}

__device__ __forceinline__ int64_t part_slot(const PagedAttnParams& p, int cta, int which) {
  return (static_cast<int64_t>(cta) * 2 + which) * p.rows;
}

// Where packed row r (node r / G, head r % G of kv head g) of sequence b goes.
template <typename T>
__device__ __forceinline__ T* out_row(const PagedAttnParams& p, int b, int g, int packed) {
  const int node = packed / p.G, head = g * p.G + packed % p.G;
  return static_cast<T*>(p.out) + b * p.o_sb + static_cast<int64_t>(node) * p.o_st + static_cast<int64_t>(head) * p.o_sh;
}
__device__ __forceinline__ int64_t lse_row(const PagedAttnParams& p, int b, int g, int packed) {
  return (static_cast<int64_t>(b) * p.T + packed / p.G) * p.Hq + g * p.G + packed % p.G;
}

// The stretch that holds the unit's last tile.
__device__ __forceinline__ int last_stretch(const Line& ln, const Piece& c) {
  return (c.unit_first + c.s.tiles - 1) / ln.step;
}

// The note of a piece that begins a unit and does not end it.
__device__ __forceinline__ SplitUnit split_of(const Line& ln, const Piece& c, int packed0, int rows) {
  return SplitUnit{last_stretch(ln, c), c.b, c.g, packed0, rows};
}

constexpr float kLn2 = 0.6931471805599453f;

}  // namespace paged

// Places of the line behind a unit's tiles, at most.  On the tensor cores a
// border costs 5 us, 3 to 4 tiles' time: with none, CTAs of one piece were
// done after 185 us and those of ten after 234 (32 sequences of 16 to 64
// nodes, prefixes up to 16384); the call took 245 us so and 220 with 3.
// CUDA cores: 255 us with 0, 248 with 1, 257 with 3 (16 sequences, fp32).
constexpr int kPagedSimtCost = 1, kPagedTcCost = 3;

cudaError_t launch_attn_paged_simt(const PagedAttnParams& p, int grid, cudaStream_t stream);
// Combines the split units' rows.
cudaError_t launch_attn_paged_merge(const PagedAttnParams& p, int grid, cudaStream_t stream);
bool attn_paged_tc_supported(const tv_attn_paged_args* a);
// Row tiles of a unit of the tensor-core kernel (a CTA each), and its TMA boxes.
int attn_paged_tc_team(const tv_attn_paged_args* a);
int attn_paged_tc_box(int page_size);
cudaError_t launch_attn_paged_tc(PagedAttnParams& p, int grid, cudaStream_t stream);
void attn_paged_set_lost(int lost);                        // tv_attn_paged_set_lost
// Query rows of the CUDA-core kernel's row tile and its CTAs per SM.
int attn_paged_simt_rows(int64_t rows);
int attn_paged_simt_ctas(int rows, int d);

}  // namespace tv
