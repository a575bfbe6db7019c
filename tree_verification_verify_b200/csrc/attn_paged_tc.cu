// tree_verify_attn_paged on the tensor cores (tcgen05 + TMEM + TMA), bf16
// with d = 64 or 128.
//
// A persistent CTA per SM works through its stretch of the line
// (attn_paged.cuh).  A unit's 128 query rows are the G heads of one kv head
// of 128 / G nodes; its key tiles are 128 prefix rows, fetched page by page,
// then tree nodes 128 at a time from the last ones down, masked per row by
// the row's root path.  Loads, products and softmax of consecutive tiles
// overlap across the borders of units: the producers run ahead into the next
// unit while the softmax warps write the last one out.
//
// Warp roles (384 threads):
//   warps 0-7  softmax and output: two warpgroups of a thread per query row
//              (TMEM lane) take the tiles in turn, each with an online
//              softmax state and an accumulator (O_0, O_1 in TMEM) of its
//              own that meet once per piece.  One group's exponentials run
//              while the other waits for TMEM and barriers (about 2000 of
//              the 5000 cycles of a tile when both worked on halves of the
//              same tile).  Warps without a valid row skip the arithmetic
//              (decoding: G of 128 rows are real);
//   warp 8     K tiles, warp 10 V tiles.  Page sizes that are multiples of
//              8 rows: one TMA box per run of rows that both the page and
//              the tile divide into (gcd(page size, 128) rows), a box per
//              lane; the page table is read for several tiles at a time, one
//              batch ahead.  Other page sizes: 16-byte cp.async per row
//              into the same swizzled layout;
//   warp 9     MMA: one thread polls what is ready and issues S = Q K^T two
//              tiles ahead or O_h += P V (P read from TMEM), so neither
//              waits for the other's operands;
//   warp 11    Q of the next unit, and parent[] for the tree tiles.
// Online softmax in base 2; O is rescaled only when a row's maximum grows by
// more than 2^8 (P <= 256, exact in O / l).  P is rounded to bf16
// for the product with V (the tensor cores' operand type); sums use the
// unrounded fp32 weights.
//
// V of a tree tile may hold infinities or NaN in nodes that a row does not
// see, and 0 * NaN would reach that row.  The softmax warps look the tile
// over, put 0 in such places and note them; a row that does see one adds
// those values to its output at the end (an infinity or a NaN takes over
// whatever its weight).  Rows of a tile past the prefix or past n_nodes are
// cleared the same way.
// Every mbarrier wait is bounded: on expiry the CTA records TV_DEV_TIMEOUT,
// drains what it issued, frees its TMEM, and its rows come out as NaN.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn.cuh"
#include "attn_paged.cuh"
#include "tc_prims.cuh"

namespace tv {

using namespace paged;
using namespace tc;

namespace ptc {

constexpr int kThreads = 384;
constexpr int kSoftmaxThreads = 256;
constexpr int kWarpK = 8, kWarpMma = 9, kWarpV = 10, kWarpTree = 11;
constexpr int kRows = 128, kKeys = 128;
constexpr int kMaxT = 2048;
constexpr uint32_t kHalfBytes = kRows * 128;              // 128 rows x 64 bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;                // S buffers 128 apart, O_0 and O_1 128 apart
constexpr uint16_t kRootMark = 0xFFFEu, kBadMark = 0xFFFFu;

template <int D>
struct Shape {
  static constexpr uint32_t kTile = D / 64 * kHalfBytes;  // bytes of a K, V or Q tile
  static constexpr int kKS = 3 * 128 / D, kVS = 2 * 128 / D;   // ring stages: 96 KB of K, 64 KB of V
  static constexpr uint32_t kQ = 0, kK = kTile, kV = kK + kKS * kTile, kPar = kV + kVS * kTile;
  static constexpr uint32_t kBytes = kPar + 2 * kMaxT * 2;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], k_empty[6], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], pv_done[2];              // by tile parity: S buffer, warpgroup, accumulator
  uint64_t o_free;                                        // a piece's accumulators have been read
  uint64_t t_full[2], t_empty[2];                         // parent[] buffers
  uint32_t tmem_base;
  int abort;
  int bad_piece[8];                                       // piece number + 1 that met a bad page
  uint32_t vbad[2][2][4];                                 // [group][its tile parity] V rows with infinities or NaN
  float red_m[2][kRows], red_l[2][kRows];
  uint8_t red_nf[2][kRows];
};

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// 16 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i]);
  tmem_st16u(taddr, u);
}

// The real tiles of a piece: prefix tiles [a0, a1), tree tiles [b0, b1)
// (tree tiles of later nodes than the row tile's are left out).
struct Tiles {
  int a0, a1, b0, b1;
  __device__ __forceinline__ int count() const { return a1 - a0 + b1 - b0; }
};

__device__ __forceinline__ Tiles tiles_of(const Piece& c, int node_hi) {
  Tiles t;
  t.a0 = min(c.t0, c.s.nprefix);
  t.a1 = min(c.t1, c.s.nprefix);
  const int skip = c.s.ntree > 0 ? c.s.ntree - (node_hi / kKeys + 1) : 0;
  t.b1 = min(c.t1, c.s.nprefix + c.s.ntree);
  t.b0 = max(c.t0, c.s.nprefix + skip);
  t.b1 = max(t.b0, t.b1);
  return t;
}

}  // namespace ptc

using namespace ptc;

// Walks a CTA's pieces; every role has its own.
struct PieceWalk {
  int pos;
  int index;                    // pieces before this one
  int queue;                    // of those, pieces with tiles
  Piece c;
  Tiles t;
  int i0, nodes, cnt;
  __device__ __forceinline__ void start(const Line& ln) { pos = ln.first; index = -1; queue = -1; cnt = 0; }
  __device__ __forceinline__ bool next(const PagedAttnParams& p, const Line& ln) {
    if (pos >= ln.last) return false;
    c = piece_at<kKeys>(p, ln, pos);
    pos += c.t1 - c.t0;
    const int npt = p.rows / p.G;
    i0 = c.rt * npt;
    nodes = min(npt, c.s.n - i0);
    t = tiles_of(c, i0 + nodes - 1);
    cnt = t.count();
    ++index;
    queue += cnt > 0;
    return true;
  }
};

// The MMA thread needs a piece's tile count alone.
struct CountWalk {
  int pos, queue, cnt;
};
__device__ __forceinline__ bool next_count(const PagedAttnParams& p, const Line& ln, CountWalk& x) {
  PieceWalk w;
  w.pos = x.pos;
  w.index = 0;
  w.queue = x.queue;
  do {
    if (!w.next(p, ln)) return false;
  } while (w.cnt == 0);
  x.pos = w.pos;
  x.queue = w.queue;
  x.cnt = w.cnt;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_paged_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_kt,
                     const __grid_constant__ CUtensorMap map_vt, PagedAttnParams p, int box) {
  using Sh = Shape<D>;
  constexpr int KS = Sh::kKS, VS = Sh::kVS;
  constexpr uint32_t TB = Sh::kTile;
  constexpr int DH = D / 2;                               // output columns of a half
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ Bars bars;
  __shared__ Line ln;
  __shared__ PieceWalk walks[kSoftmaxThreads / 32];       // the softmax warps': registers are for scores
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.G;
  const uint32_t raw = smem_u32(dsmem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;           // 128B swizzle atoms are 1 KB
  uint8_t* gbase = dsmem_raw + (base - raw);
  uint16_t* spar = reinterpret_cast<uint16_t*>(gbase + Sh::kPar);
  volatile int* abort = &bars.abort;

  if (tid >= 32 && tid < 37) {
    const CUtensorMap* m = tid == 32 ? &map_q : (tid == 33 ? &map_k : (tid == 34 ? &map_v : (tid == 35 ? &map_kt : &map_vt)));
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (tid == 0) {
    mbar_init(&bars.q_full, 1); mbar_init(&bars.q_empty, 1);
    for (int s = 0; s < KS; ++s) { mbar_init(&bars.k_full[s], 1); mbar_init(&bars.k_empty[s], 1); }
    for (int s = 0; s < VS; ++s) { mbar_init(&bars.v_full[s], 1); mbar_init(&bars.v_empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.p_full[s], 4);
      mbar_init(&bars.pv_done[s], 1);
      mbar_init(&bars.t_full[s], 1); mbar_init(&bars.t_empty[s], 8);
      for (int i = 0; i < 8; ++i) bars.vbad[s][i >> 2][i & 3] = 0;
    }
    mbar_init(&bars.o_free, 8);
    for (int i = 0; i < 8; ++i) bars.bad_piece[i] = 0;
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  build_line<kKeys, kThreads>(p, ln);                     // ends with a CTA barrier
  fence_after();
  const uint32_t tmem = bars.tmem_base;
  PieceWalk w;
  w.start(ln);

  // 384 threads launch with 168 registers: 256 softmax threads take 208, the
  // other 128 keep 88 (256 * 208 + 128 * 88 = 384 * 168)
  if (warp >= kSoftmaxThreads / 32) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == kWarpK || warp == kWarpV) {
    // ------------------------------------------------------------ producers
    const bool isk = warp == kWarpK;
    const int NS = isk ? KS : VS;
    uint64_t* full = isk ? bars.k_full : bars.v_full;
    uint64_t* empty = isk ? bars.k_empty : bars.v_empty;
    const CUtensorMap* map = isk ? &map_k : &map_v;
    const CUtensorMap* map_tree = isk ? &map_kt : &map_vt;
    const uint32_t ring = base + (isk ? Sh::kK : Sh::kV);
    const unsigned P = p.page_size;
    int it = 0;
    bool ok = true;
    int pending = -1;                                     // stage whose cp.async copies are not announced yet
    auto flush = [&]() {
      if (pending < 0) return;
      cp_async_wait_all();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[pending]);
      pending = -1;
    };
    auto acquire = [&](int s) -> bool {                   // the stage is free
      if (it < NS) return true;
      bool a = true;
      if (pending >= 0 && !__shfl_sync(0xffffffffu, lane == 0 ? mbar_test(&empty[s], ((it / NS) - 1) & 1) : false, 0))
        flush();
      if (lane == 0) a = mbar_wait(&empty[s], ((it / NS) - 1) & 1, abort);
      return __all_sync(0xffffffffu, a);
    };
    auto bad_page = [&]() { if (isk) bars.bad_piece[w.index & 7] = w.index + 1; };
    while (ok && w.next(p, ln)) {
      const int32_t* table = p.table + w.c.b * p.pt_sb;
      const int L = w.c.s.L, g = w.c.g, b = w.c.b;
      if (box > 0) {
        // lane l holds the run of `box` rows number l % nb of tile l / nb of a batch of 32 / nb tiles
        const int nb = kKeys / box, batch = 32 / nb;
        int row = 0, page = 0, row_n = 0, page_n = 0;
        auto look = [&](int t, int& r, int& pg) {
          const unsigned pos = static_cast<unsigned>(t + lane / nb) * kKeys + lane % nb * box;
          r = -1;
          pg = 0;
          if (t + lane / nb < w.t.a1 && pos < static_cast<unsigned>(L)) {
            r = static_cast<int>(pos % P);
            pg = __ldg(table + pos / P);
          }
        };
        look(w.t.a0, row_n, page_n);
        for (int t = w.t.a0; ok && t < w.t.a1; ++t, ++it) {
          const int k = (t - w.t.a0) % batch;
          if (k == 0) {
            row = row_n;
            page = page_n;
            look(t + batch, row_n, page_n);
          }
          const int s = it % NS;
          ok = acquire(s);
          if (!ok) break;
          const bool mine = lane / nb == k && row >= 0;
          if (mine && (page < 0 || page >= p.num_pages)) {
            bad_page();
            page = p.num_pages;                           // past the pool's end: the box reads as zeros
          }
          const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
          __syncwarp();                                   // a bad page is noted before the tile is announced
          if (lane == 0) mbar_expect_tx(&full[s], static_cast<uint32_t>(boxes) * box * D * 2);
          __syncwarp();
          if (mine) {
            const uint32_t dst = ring + s * TB + lane % nb * box * 128;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) tma_load_4d(map, dst + h * kHalfBytes, &full[s], 64 * h, g, row, page);
          }
        }
      } else {
        const char* pool = static_cast<const char*>(isk ? p.kp : p.vp) + g * p.kv_sh * 2;
        for (int t = w.t.a0; ok && t < w.t.a1; ++t, ++it) {
          // lane l holds the places of rows l, l + 32, l + 64, l + 96
          int64_t off[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const unsigned pos = static_cast<unsigned>(t) * kKeys + i * 32 + lane;
            off[i] = -1;
            if (pos < static_cast<unsigned>(L)) {
              const int page = __ldg(table + pos / P);
              if (page < 0 || page >= p.num_pages) bad_page();
              else off[i] = (page * p.kv_sp + static_cast<int64_t>(pos % P) * p.kv_sr) * 2;
            }
          }
          const int s = it % NS;
          ok = acquire(s);
          if (!ok) break;
          constexpr int CPR = D / 8, RPI = 32 / CPR;      // 16-byte chunks of a row, rows of a step
          const int ch = lane % CPR;
          const uint32_t dst = ring + s * TB + ch / 8 * kHalfBytes;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll 8
            for (int r0 = 0; r0 < 32; r0 += RPI) {
              const int r = r0 + lane / CPR;
              const int64_t o = __shfl_sync(0xffffffffu, off[i], r);
              const int rr = i * 32 + r;
              if (o >= 0) cp_async16(dst + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4), pool + o + ch * 16);
            }
          }
          const int before = pending;
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (before >= 0) {                              // the tile before this one has landed
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[before]);
          }
          pending = s;
        }
      }
      for (int t = w.t.b0; ok && t < w.t.b1; ++t, ++it) {
        const int s = it % NS;
        ok = acquire(s);
        if (!ok) break;
        flush();
        if (lane == 0) {
          const int lo = (w.c.s.ntree - 1 - (t - w.c.s.nprefix)) * kKeys;
          mbar_expect_tx(&full[s], TB);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(map_tree, ring + s * TB + h * kHalfBytes, &full[s], 64 * h, g, lo, b);
        }
      }
    }
    flush();
    // drain: every issued load lands before the CTA can exit
    if (lane == 0)
      for (int j = (it > NS ? it - NS : 0); j < it; ++j) mbar_drain(&full[j % NS], (j / NS) & 1);
    __syncwarp();
  } else if (warp == kWarpTree) {
    // ------------------------------------------------------------ Q and parent[]
    int nq = 0, ntree = 0;
    bool ok = true;
    auto load_q = [&]() -> bool {
      bool a = true;
      if (nq > 0) {
        if (lane == 0) a = mbar_wait(&bars.q_empty, (nq - 1) & 1, abort);
        a = __all_sync(0xffffffffu, a);
      }
      if (!a) return false;
      if (lane == 0) {
        mbar_expect_tx(&bars.q_full, static_cast<uint32_t>(p.rows) * D * 2);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_load_4d(&map_q, base + Sh::kQ + h * kHalfBytes, &bars.q_full, 64 * h, w.c.g * G, w.i0, w.c.b);
      }
      ++nq;
      return true;
    };
    while (ok && w.next(p, ln)) {
      if (w.cnt == 0) continue;
      const bool first = nq == 0;
      if (first) ok = load_q();
      if (ok && w.t.b1 > w.t.b0) {
        const int buf = ntree & 1;
        bool a = true;
        if (ntree >= 2 && lane == 0) a = mbar_wait(&bars.t_empty[buf], ((ntree >> 1) - 1) & 1, abort);
        ok = __all_sync(0xffffffffu, a);
        if (!ok) break;
        const int32_t* par = p.parent + w.c.b * p.par_sb;
        for (int j = lane; j < w.i0 + w.nodes; j += 32) {
          const int pj = par[j];
          spar[buf * kMaxT + j] = j == 0 ? (pj == -1 ? kRootMark : kBadMark)
                                         : ((pj >= 0 && pj < j) ? static_cast<uint16_t>(pj) : kBadMark);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.t_full[buf]);
        ++ntree;
      }
      if (ok && !first) ok = load_q();
    }
    if (lane == 0 && nq > 0) mbar_drain(&bars.q_full, (nq - 1) & 1);
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc_qk = instr_desc(kRows, kKeys, 0, 0);
      const uint32_t idesc_pv = instr_desc(kRows, D, 0, 1);
      CountWalk cs = {ln.first, -1, 0}, cp = cs;          // the pieces of the next S and of the next P V
      int rs = 0, rp = 0;                                 // tiles done in those pieces
      int is = 0, ip = 0;                                 // S and P V issued in all
      bool more_s = next_count(p, ln, cs), more_p = more_s;
      cp = cs;
      auto step = [&](CountWalk& x, int& r, bool& more) {
        if (r >= x.cnt) {
          more = next_count(p, ln, x);
          r = 0;
        }
      };
      uint32_t idle = 0;
      while (more_p) {
        // all tests of a poll are independent: together they cost little more than one
        const bool want_s = more_s && is < ip + 2;
        const bool tk = want_s && mbar_test(&bars.k_full[is % KS], (is / KS) & 1);
        const bool tq = want_s && (rs > 0 || mbar_test(&bars.q_full, cs.queue & 1));
        const bool want_p = ip < is;
        const bool tv = want_p && mbar_test(&bars.v_full[ip % VS], (ip / VS) & 1);
        const bool tp = want_p && mbar_test(&bars.p_full[ip & 1], (ip >> 1) & 1);
        // the first tile of either group overwrites its accumulator, so the last piece's must have been read
        const bool to = want_p && (rp > 1 || cp.queue == 0 || mbar_test(&bars.o_free, (cp.queue - 1) & 1));
        bool did = false;
        if (tk && tq) {
          fence_after();
          const uint32_t sq = base + Sh::kQ, sk = base + Sh::kK + (is % KS) * TB;
          const uint32_t sd = tmem + kColS + (is & 1) * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
            mma_bf16(sd, smem_desc(sq + off, 16, 1024), smem_desc(sk + off, 16, 1024), idesc_qk, kk > 0);
          }
          mma_commit(&bars.k_empty[is % KS]);
          mma_commit(&bars.s_full[is & 1]);
          if (rs == cs.cnt - 1) mma_commit(&bars.q_empty);
          ++is;
          ++rs;
          step(cs, rs, more_s);
          did = true;
        }
        // O_h += P V: P is bf16 pairs over the first 64 columns of its S
        if (tv && tp && to) {
          fence_after();
          const uint32_t sv = base + Sh::kV + (ip % VS) * TB;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts(tmem + kColO + (ip & 1) * 128, tmem + kColS + (ip & 1) * 128 + kk * 8,
                        smem_desc(sv + kk * 2048, kHalfBytes, 1024), idesc_pv, (rp > 1 || kk > 0) ? 1u : 0u);
          mma_commit(&bars.v_empty[ip % VS]);
          mma_commit(&bars.pv_done[ip & 1]);
          ++ip;
          ++rp;
          step(cp, rp, more_p);
          did = true;
        }
        if (did) {
          idle = 0;
        } else if (++idle >= kWaitLimit || ((idle & 255u) == 255u && *abort)) {
          *abort = 1;
          break;
        }
      }
      if (*abort) {
        // what was issued completes before the TMEM is freed
        for (int j = is > 2 ? is - 2 : 0; j < is; ++j) mbar_drain(&bars.s_full[j & 1], (j >> 1) & 1);
        for (int j = ip > 2 ? ip - 2 : 0; j < ip; ++j) mbar_drain(&bars.pv_done[j & 1], (j >> 1) & 1);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warps 0-7
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int row = tid & (kRows - 1), half = tid >> 7;   // half: the warpgroup
    const float sl2 = p.scale * 1.4426950408889634f;      // scores in log2 units
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t scol = trow + kColS + 128u * static_cast<uint32_t>(half);
    const uint32_t ocol = trow + kColO + 128u * static_cast<uint32_t>(half);
    int it0 = 0, ntree = 0;                               // tiles before this piece
    SplitUnit split = {-1, 0, 0, 0, 0};
    bool ok = true;
    PieceWalk& sw = walks[warp];
    sw = w;
    __syncwarp();
    while (true) {
      {
        PieceWalk x = sw;
        __syncwarp();
        if (!x.next(p, ln)) break;
        sw = x;
        __syncwarp();
      }
      const PieceWalk& w = sw;
      const Piece& c = w.c;
      const int rows_here = w.nodes * G;
      const bool live = (warp & 3) * 32 < rows_here;      // the warp has valid rows
      const bool row_valid = row < rows_here;
      const int my_node = w.i0 + row / G;
      const int na = w.t.a1 - w.t.a0, cnt = w.cnt, nodes = c.s.n;
      const int keys0 = c.s.L - w.t.a0 * kKeys;           // prefix keys from the piece's first tile on
      const int lo0 = (c.s.ntree - 1 - (w.t.b0 - na - c.s.nprefix)) * kKeys;
      const int r0 = (half ^ it0) & 1;                    // the group's first tile
      float m_run = -INFINITY, l_run = 0.f;
      bool my_ok = true, nf = false;
      int cur = -2;                                       // walk position on this row's root path (-2: not begun)
      const uint16_t* par = spar + (ntree & 1) * kMaxT;
      for (int r = r0; r < cnt; r += 2) {
        const int it = it0 + r;
        const bool tree = r >= na;
        const int lo = lo0 - r * kKeys;                   // tree tile: its first node
        const int nk = min(kKeys, tree ? nodes - lo : keys0 - r * kKeys);
        const bool full = !tree && nk == kKeys;
        // keys that the row sees
        uint32_t mk[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (tree) {
          if (cur == -2) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars.t_full[ntree & 1], (ntree >> 1) & 1, abort));
            cur = row_valid && ok ? my_node : -1;
          }
          mk[0] = mk[1] = mk[2] = mk[3] = 0u;
          while (cur >= lo) {
            const int k = cur - lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) mk[i] |= (k >> 5) == i ? 1u << (k & 31) : 0u;
            const uint16_t up = par[cur];
            my_ok = my_ok && up != kBadMark;
            cur = up >= kRootMark ? -1 : static_cast<int>(up);
          }
        } else if (!full) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int nh = nk - 32 * i;
            mk[i] = nh >= 32 ? 0xffffffffu : (nh <= 0 ? 0u : ((1u << nh) - 1u));
          }
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars.s_full[half], (it >> 1) & 1, abort));
        fence_after();
        if (live && ok) {
          // Two forms of one computation: a full prefix tile holds its 128
          // scores in registers; the others (one or two per piece) mask them,
          // 32 at a time in loops that are not unrolled, and read them twice:
          // code that runs once per piece is fetched each time, and fetching
          // it costs more than running it.
          float nmu, factor = 1.f;
          bool grow;
          auto take = [&](const float* mx) {              // the tile's maximum into the row's state
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
            const float m_new = fmaxf(m_run, mt);
            grow = m_new > m_run + 8.0f;                  // also the first finite maximum
            if (grow) {
              factor = ex2_approx(m_run - m_new);         // 0 when m_run = -inf
              m_run = m_new;
            }
            nmu = (m_run == -INFINITY) ? 0.f : -m_run;
          };
          // p = 2^(s sl2 - m) as bf16 pairs over the first half of S, behind
          // the columns already read
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (full) {
            float s[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(scol + q * 32, s + q * 32);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 128; ++k) mx[k & 3] = fmaxf(mx[k & 3], s[k]);
            take(mx);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t pk[16];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float a = ex2_approx(fmaf(s[q * 32 + k], sl2, nmu));
                const float b = ex2_approx(fmaf(s[q * 32 + k + 1], sl2, nmu));
                ps[k & 2] += a;
                ps[(k & 2) + 1] += b;
                pk[k / 2] = pack_bf16(a, b);
              }
              tmem_st16u(scol + q * 16, pk);
            }
          } else {
            auto mask = [&](int q) { return q == 0 ? mk[0] : (q == 1 ? mk[1] : (q == 2 ? mk[2] : mk[3])); };
            float s[32];
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              tmem_ld32(scol + q * 32, s);
              tmem_wait_ld();
              const uint32_t m = mask(q);
#pragma unroll
              for (int k = 0; k < 32; ++k) mx[k & 3] = fmaxf(mx[k & 3], ((m >> k) & 1u) ? s[k] : -INFINITY);
            }
            take(mx);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              tmem_ld32(scol + q * 32, s);
              tmem_wait_ld();
              const uint32_t m = mask(q);
              uint32_t pk[16];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float a = ((m >> k) & 1u) ? ex2_approx(fmaf(s[k], sl2, nmu)) : 0.f;
                const float b = ((m >> (k + 1)) & 1u) ? ex2_approx(fmaf(s[k + 1], sl2, nmu)) : 0.f;
                ps[k & 2] += a;
                ps[(k & 2) + 1] += b;
                pk[k / 2] = pack_bf16(a, b);
              }
              tmem_st16u(scol + q * 16, pk);
              tmem_wait_st();
            }
          }
          l_run = l_run * factor + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
          if (__any_sync(0xffffffffu, grow) && r >= 2) {
            // O_h holds the group's tiles before this one (their P V is done:
            // this tile's S was issued behind it): rescale
            fence_after();
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              float o[16];
              tmem_ld16(ocol + q * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= factor;
              tmem_st16(ocol + q * 16, o);
            }
          }
          tmem_wait_st();
        }
        if (!full) {
          // V rows that are no keys are cleared; a tree tile's rows are looked over
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars.v_full[it % VS], (it / VS) & 1, abort));
          uint8_t* v0 = gbase + Sh::kV + (it % VS) * TB + row * 128;
          uint32_t* vbad = bars.vbad[half][(it >> 1) & 1];
          bool hit = false;
          if (ok && (row >= nk || tree)) {
#pragma unroll 4
            for (int ch = 0; ch < D / 8; ++ch) {
              uint4* at = reinterpret_cast<uint4*>(v0 + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (row & 7)) << 4));
              if (row >= nk) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else {
                uint4 x = *at;
                uint32_t e[4] = {x.x, x.y, x.z, x.w};
                bool h = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if ((e[i] & 0x7f80u) == 0x7f80u) { e[i] &= 0xffff0000u; h = true; }
                  if ((e[i] & 0x7f800000u) == 0x7f800000u) { e[i] &= 0xffffu; h = true; }
                }
                if (h) { *at = make_uint4(e[0], e[1], e[2], e[3]); hit = true; }
              }
            }
          }
          if (hit) atomicOr(vbad + (row >> 5), 1u << (row & 31));
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          if (tree) {
            // every warp of the group comes here for every tree tile, after an abort too
            bar_sync(2 + half, 128);
            uint32_t any = 0, seen = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = *reinterpret_cast<volatile uint32_t*>(vbad + i);
              any |= x;
              seen |= x & mk[i];
            }
            if (any) {
              nf = nf || seen;
              bar_sync(2 + half, 128);
              if ((tid & 127) < 4) vbad[tid & 3] = 0;
              bar_sync(2 + half, 128);
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&bars.p_full[half]);
      }
      // ---------------------------------------------------------- output
      // the group's last P V; tiles two apart complete in order, so one phase is enough
      it0 += cnt;
      if (cnt > r0) {
        const int last = it0 - 1 - ((it0 - 1 - half) & 1);
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars.pv_done[half], (last >> 1) & 1, abort));
      }
      // the groups meet: M = max(m_0, m_1), c_h = 2^(m_h - M),
      // O = (c_0 O_0 + c_1 O_1) / (c_0 l_0 + c_1 l_1); group h writes d columns DH h ..
      bars.red_m[half][row] = m_run;
      bars.red_l[half][row] = l_run;
      bars.red_nf[half][row] = nf + 2 * !my_ok;
      fence_before();
      bar_sync(1, kSoftmaxThreads);
      fence_after();
      const float m_0 = bars.red_m[0][row], m_1 = bars.red_m[1][row];
      const float l_0 = bars.red_l[0][row], l_1 = bars.red_l[1][row];
      nf = ((bars.red_nf[0][row] | bars.red_nf[1][row]) & 1) != 0;
      my_ok = ((bars.red_nf[0][row] | bars.red_nf[1][row]) & 2) == 0;
      const float M = fmaxf(m_0, m_1);
      const float c_0 = (m_0 == -INFINITY) ? 0.f : ex2_approx(m_0 - M);
      const float c_1 = (m_1 == -INFINITY) ? 0.f : ex2_approx(m_1 - M);
      // a group whose sum is NaN (a NaN score) makes the row NaN
      const float l_row = c_0 * l_0 + c_1 * l_1 + ((l_0 != l_0 || l_1 != l_1) ? NAN : 0.f);
      const bool have_0 = cnt > (it0 - cnt & 1 ? 1 : 0), have_1 = cnt > (it0 - cnt & 1 ? 0 : 1);   // tiles of group 0, 1
      const bool bad = c.s.bad_len || !my_ok || !ok || bars.bad_piece[w.index & 7] == w.index + 1;
      const bool empty = l_row == 0.f;
      const float inv = bad ? NAN : (empty ? 0.f : 1.f / l_row);
      const float w_0 = c_0 * inv, w_1 = c_1 * inv;
      const bool whole = c.t0 == 0 && c.t1 == c.s.len;
      const int packed = w.i0 * G + row;
      const int which = c.t0 == 0 ? 1 : 0;
      const int64_t slot = part_slot(p, blockIdx.x, which, kRows) + row;
      if (live) {
        __nv_bfloat16* orow = row_valid ? out_row<__nv_bfloat16>(p, c.b, c.g, packed) : nullptr;
#pragma unroll 1
        for (int q = 0; q < DH / 16; ++q) {
          const int col = half * DH + q * 16;
          float v0[16], v1[16];
          if (have_0) tmem_ld16(trow + kColO + col, v0);
          if (have_1) tmem_ld16(trow + kColO + 128 + col, v1);
          tmem_wait_ld();
          if (!row_valid) continue;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            // an accumulator that no tile wrote is not looked at
            v0[e] = (have_0 ? w_0 * v0[e] : 0.f) + (have_1 ? w_1 * v1[e] : 0.f) + (bad ? NAN : 0.f);
          }
          if (nf) {
            // the values that are not finite, of the nodes this row sees
            int j = my_node;
            while (true) {
              const __nv_bfloat16* vs = static_cast<const __nv_bfloat16*>(p.vt) + c.b * p.kt_sb +
                                        static_cast<int64_t>(j) * p.kt_st + static_cast<int64_t>(c.g) * p.kt_sh + col;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = __bfloat162float(vs[e]);
                if (!(fabsf(x) < INFINITY)) v0[e] += x;
              }
              const uint16_t up = par[j];
              if (up >= kRootMark) break;
              j = up;
            }
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint4 x;
              x.x = pack_bf16(v0[8 * e], v0[8 * e + 1]);
              x.y = pack_bf16(v0[8 * e + 2], v0[8 * e + 3]);
              x.z = pack_bf16(v0[8 * e + 4], v0[8 * e + 5]);
              x.w = pack_bf16(v0[8 * e + 6], v0[8 * e + 7]);
              *reinterpret_cast<uint4*>(orow + col + 8 * e) = x;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(p.part_o + slot * D + col + 4 * e) =
                  make_float4(v0[4 * e], v0[4 * e + 1], v0[4 * e + 2], v0[4 * e + 3]);
          }
        }
        if (half == 0 && row_valid) {
          const float lse2 = bad ? NAN : (empty ? -INFINITY : M + log2f(l_row));
          if (!whole) p.part_lse[slot] = lse2;
          else if (p.lse) p.lse[lse_row(p, c.b, c.g, packed)] = lse2 * kLn2;
          if (!my_ok) set_status(p.status, TV_DEV_BAD_PARENT);
        }
      }
      // the accumulators are free for the next piece
      fence_before();
      __syncwarp();
      if (lane == 0 && cnt > 0) mbar_arrive(&bars.o_free);
      if (tid == 0) {
        if (bars.bad_piece[w.index & 7] == w.index + 1) set_status(p.status, TV_DEV_BAD_PAGE);
        if (!ok) set_status(p.status, TV_DEV_TIMEOUT);
      }
      if (w.t.b1 > w.t.b0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.t_empty[ntree & 1]);
        ++ntree;
      }
      if (tid == 0 && c.t0 == 0 && !whole) split = split_of(ln, c, w.i0 * G, rows_here);
      bar_sync(1, kSoftmaxThreads);                       // red_*: read by all
    }
    if (tid == 0) p.splits[blockIdx.x] = split;
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ host side

namespace {

// A dimension of one element has no stride to speak of: any valid one.
int64_t stride_or(int64_t dim, int64_t s) { return dim > 1 ? s : 128; }

bool stride_ok(int64_t dim, int64_t s) { return dim <= 1 || (s > 0 && s % 8 == 0 && s * 2 < (1ll << 40)); }

int page_box(int P) {
  int b = 128;
  while (b >= 8 && P % b != 0) b /= 2;
  return b >= 8 ? b : 0;
}

template <int D>
cudaError_t launch(const PagedAttnParams& p, int grid, int box, const CUtensorMap* m, cudaStream_t stream) {
  constexpr size_t smem = Shape<D>::kBytes + 1024;
  const cudaError_t e = cudaFuncSetAttribute(attn_paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  attn_paged_tc_kernel<D><<<grid, kThreads, smem, stream>>>(m[0], m[1], m[2], m[3], m[4], p, box);
  return cudaGetLastError();
}

}  // namespace

bool attn_paged_tc_supported(const tv_attn_paged_args* a) {
  if (a->dtype != TV_BF16 || (a->d != 64 && a->d != 128)) return false;
  if (a->B == 0 || a->T == 0 || a->T > kMaxT || a->num_pages == 0 || a->max_pages == 0) return false;
  if (!stride_ok(a->Hq, a->q_sh) || !stride_ok(a->T, a->q_st) || !stride_ok(a->B, a->q_sb)) return false;
  if (!stride_ok(a->Hkv, a->kv_sh) || !stride_ok(a->page_size, a->kv_sr) || !stride_ok(a->num_pages, a->kv_sp)) return false;
  if (!stride_ok(a->Hkv, a->kt_sh) || !stride_ok(a->T, a->kt_st) || !stride_ok(a->B, a->kt_sb)) return false;
  if (!stride_ok(a->Hq, a->o_sh) || !stride_ok(a->T, a->o_st) || !stride_ok(a->B, a->o_sb)) return false;
  const uintptr_t al = reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->k_pages) |
                       reinterpret_cast<uintptr_t>(a->v_pages) | reinterpret_cast<uintptr_t>(a->k_tree) |
                       reinterpret_cast<uintptr_t>(a->v_tree) | reinterpret_cast<uintptr_t>(a->out);
  return (al & 15u) == 0 && tcmap::encode_fn() != nullptr;
}

cudaError_t launch_attn_paged_tc(const PagedAttnParams& p, int grid, cudaStream_t stream) {
  CUtensorMap m[5];
  const int box = page_box(p.page_size);
  auto map = [&](CUtensorMap* t, const void* x, int64_t d1, int64_t d2, int64_t d3, int64_t s1, int64_t s2, int64_t s3,
                 int b1, int b2) {
    return tcmap::make_map(t, x, p.d, d1, d2, d3, stride_or(d1, s1), stride_or(d2, s2), stride_or(d3, s3), b1, b2);
  };
  if (!map(&m[0], p.q, p.Hq, p.T, p.B, p.q_sh, p.q_st, p.q_sb, p.G, p.rows / p.G) ||
      !map(&m[3], p.kt, p.Hkv, p.T, p.B, p.kt_sh, p.kt_st, p.kt_sb, 1, kKeys) ||
      !map(&m[4], p.vt, p.Hkv, p.T, p.B, p.kt_sh, p.kt_st, p.kt_sb, 1, kKeys))
    return cudaErrorInvalidValue;
  if (box > 0) {
    if (!map(&m[1], p.kp, p.Hkv, p.page_size, p.num_pages, p.kv_sh, p.kv_sr, p.kv_sp, 1, box) ||
        !map(&m[2], p.vp, p.Hkv, p.page_size, p.num_pages, p.kv_sh, p.kv_sr, p.kv_sp, 1, box))
      return cudaErrorInvalidValue;
  } else {
    m[1] = m[3];
    m[2] = m[4];
  }
  return p.d == 64 ? launch<64>(p, grid, box, m, stream) : launch<128>(p, grid, box, m, stream);
}

}  // namespace tv
