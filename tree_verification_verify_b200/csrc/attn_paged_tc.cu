// tree_verify_attn_paged on the tensor cores (tcgen05 + TMEM + TMA), bf16
// with d = 64 or 128.
//
// A persistent CTA per SM works through its stretch of the line
// (attn_paged.cuh).  A unit's query rows are the G heads of one kv head of
// up to 128 / G nodes (a row tile), or of a team of CTAs' row tiles; its key
// tiles are 128 prefix rows, fetched page by page, then tree nodes 128 at a
// time from the last ones down, masked per row by the row's root path.  The
// prefix's last rows and a small tree share one tile.  Loads, products and
// softmax of consecutive tiles overlap across the borders of units.
//
// What bounds it.  A steady tile takes about 2450 cycles (1.4 us) against 1024
// each of the tensor pipe and the exponentials: with up to 128 rows a sequence
// that is HBM (one sequence of 262144 rows, 16 nodes of 8 heads: 197 us, 5.4
// TB/s; 32 sequences of up to 16 nodes on 512 to 16384 rows: 217 us, 5.3
// TB/s; 64 single tokens on 512 to 8000 rows: 192 us, 5.8 TB/s), with more
// rows what the L2 hands the SMs, about 7 TB/s (two sequences of 65537 to
// 131072 rows, 64 nodes of 4 heads: 246 us, 838 TFLOP/s).  Those are short
// runs at 1965 MHz; in long ones, under the power cap, the second takes 258 us
// and the last 296.  Beside the tiles: 5 to 8 us from the start to the first
// product, 5 us a border between units (256 single tokens on 512 rows: 162 us,
// 85 for their bytes), 6 us for the second kernel; those are most of a small
// call (one token on 700 rows: 16.4 us).
//
// Warp roles (384 threads):
//   warps 0-7  softmax and output: two warpgroups, a thread per query row
//              (TMEM lane), that take the key tiles in turn, so that one
//              group's exponentials run while the other waits for TMEM and
//              barriers (both on halves of the same tile: twice the time
//              a tile, half of it waits).  Warps without a valid row skip
//              the arithmetic (decoding: G of 128 rows are real);
//   warp 8     K tiles, warp 10 V tiles.  Page sizes that are multiples of
//              8 rows: one TMA box per run of rows that both the page and
//              the tile divide into (gcd(page size, 128) rows), a box per
//              lane; the page table is read for several tiles at a time, one
//              batch ahead.  Other page sizes: 16-byte cp.async per row
//              into the same swizzled layout;
//   warp 9     MMA: one thread polls what is ready and issues S = Q K^T up
//              to three tiles ahead or O += P V (P read from TMEM), so
//              neither waits for the other's operands;
//   warp 11    the pieces' descriptions, several ahead of their use (finding
//              one takes a search and four divisions), Q and parent[].  Pieces
//              without a tile are not described; this warp writes their rows.
//              Every described piece has a tile, so the roles are at most a few
//              pieces apart and the ring of descriptions never holds one up
//              (the MMA thread looks for the next S while it still owes P V
//              and has not given the older descriptions back: eight pieces
//              without a tile in a row would stop it for good).
// TMEM: three S buffers and one accumulator O.  The groups share O, and so
// they share each row's reference maximum m: P = 2^(s - m).  The group with
// tile j takes m over from the group with tile j - 1 (a barrier per pair of
// warps that share rows), raises it only when the tile's maximum exceeds it
// by more than 8 (P <= 2^8, exact in O / l) and then rescales O itself, once
// P V of tile j - 1 is done.  (With an accumulator and a maximum per group
// there is room for two S buffers only, and S of a group's next tile has to
// wait for P V of its last one: 3900 cycles a tile with 128 rows when one accumulator took 3000.)  P is
// rounded to bf16 for the product with V (the tensor cores' operand type);
// sums use the unrounded fp32 weights.
//
// V of a tree tile may hold infinities or NaN in nodes that a row does not
// see, and 0 * NaN would reach that row.  The softmax warps look the nodes'
// rows over, put 0 in such places and note the rows; a query row that sees
// one adds those values to its output at the end (an infinity or a NaN takes
// over whatever its weight).  Rows of the last K steps that are no keys are
// cleared; later K steps are not issued.
// Every mbarrier wait is bounded (a failing poll takes 3.2 us, the limit 13 s).
// On expiry the flag `going` falls, which the waits for tiles heed; the roles
// drain what they issued and leave.  The softmax warps meet at block barriers
// within a piece, so they may not leave at different pieces: they walk all
// that warp 11 has described, and when it gives up it says which piece is the
// first that will not be described.  When they are done warp 11 records
// TV_DEV_TIMEOUT and writes NaN into all rows of the CTA's stretch, those that
// were finished among them: nothing of an earlier call is left in the outputs
// or in the partial rows.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <climits>

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
constexpr int kTreeBox = 8;                               // tree nodes of a TMA box
constexpr uint32_t kHalfBytes = kRows * 128;              // 128 rows x 64 bf16
constexpr uint32_t kTmemCols = 512;
constexpr int kSB = 3;                                    // S buffers, 128 columns each
constexpr uint32_t kColS = 0, kColO = kSB * 128;
constexpr uint16_t kRootMark = 0xFFFEu, kBadMark = 0xFFFFu;
constexpr int kRing = 8, kAhead = 3;                      // descriptions kept, and made ahead
constexpr int kLostPieces = 1, kLostProducts = 2;         // PagedAttnParams::lost

// Shared memory: Q, the K and V rings (64 KB and 96 KB: a V tile waits for the
// softmax; the other way round took 6 % longer), two parent[] buffers.
template <int D>
struct Shape {
  static constexpr uint32_t kTile = D / 64 * kHalfBytes;  // bytes of a K, V or Q tile
  static constexpr int kKS = 2 * 128 / D, kVS = 3 * 128 / D;
  static constexpr uint32_t kQ = 0, kK = kTile, kV = kK + kKS * kTile, kPar = kV + kVS * kTile;
  static constexpr uint32_t kBytes = kPar + 2 * kMaxT * 2;
};

// A piece, ready for use: its tiles are na prefix tiles from a0 on, then ntr
// tree tiles whose first nodes are lo0, lo0 - 128, ...
struct Desc {
  int valid;                    // 0: there are no more pieces
  int cnt;                      // na + ntr (at least 1)
  int b, g, i0;                 // sequence, kv head, first node of this CTA's row tile
  int nodes;                    // nodes of the row tile
  int n, L;                     // the sequence's nodes and prefix rows
  int a0, na, ntr, lo0;
  int rem, off;                 // the tree tile's prefix rows, and where its nodes begin
  int bad_len, whole, begins;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[6], v_empty[6];
  uint64_t s_full[kSB], p_full[kSB];                      // S and P buffers
  uint64_t pv_done[2];                                    // P V, by tile parity
  uint64_t dec[4][2];                                     // [warp & 3][group] the group's rows have their reference maximum
  uint64_t o_full, o_free;                                // a piece's O is whole; it has been read
  uint64_t t_full[2], t_empty[2];                         // parent[] buffers
  uint64_t w_full[kRing], w_empty[kRing];                 // piece descriptions
  uint32_t tmem_base;
  int going;                                              // 0 after a wait that ran out
  int end_at;                                             // the first piece that will not be described, once warp 11 gave up
  int bad_piece[8];                                       // piece number + 1 that met a bad page
  uint32_t vbad[2][4][4];                                 // [group][its tree tile & 3] V rows with infinities or NaN
  Desc desc[kRing];
  float m_ref[kRows];                                     // the rows' reference maxima
  float red_m[2][kRows], red_l[2][kRows];
  uint8_t red_nf[2][kRows];
};

// Two fp32 operations in one instruction (sm_100).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Non-blocking tests of five barriers in one go: bit i is set when phase
// (parity >> i) & 1 of b[i] is complete.  One after the other, each test took
// its own 100 to 300 cycles (shared memory is busy with operands and tiles).
__device__ __forceinline__ uint32_t mbar_test5(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3, uint32_t b4,
                                               uint32_t parity) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p<5>;\n\t.reg .u32 q<5>, v<5>;\n\t"
      "and.b32 q0, %6, 1;\n\tbfe.u32 q1, %6, 1, 1;\n\tbfe.u32 q2, %6, 2, 1;\n\t"
      "bfe.u32 q3, %6, 3, 1;\n\tbfe.u32 q4, %6, 4, 1;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p0, [%1], q0;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p1, [%2], q1;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p2, [%3], q2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p3, [%4], q3;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p4, [%5], q4;\n\t"
      "selp.u32 v0, 1, 0, p0;\n\tselp.u32 v1, 2, 0, p1;\n\tselp.u32 v2, 4, 0, p2;\n\t"
      "selp.u32 v3, 8, 0, p3;\n\tselp.u32 v4, 16, 0, p4;\n\t"
      "or.b32 v0, v0, v1;\n\tor.b32 v2, v2, v3;\n\tor.b32 v0, v0, v4;\n\tor.b32 %0, v0, v2;\n\t}"
      : "=r"(r)
      : "r"(b0), "r"(b1), "r"(b2), "r"(b3), "r"(b4), "r"(parity)
      : "memory");
  return r;
}

// Bounded wait on phase `parity`; false when the CTA gives up (going nullptr:
// not asked) or the limit expired (then the flag falls).  Rolled, as
// every loop here that can be: unrolled as the compiler would have it the
// kernel has 144 KB of code, the warps' roles push one another out of the
// instruction cache, and its speed changes by up to half with unrelated edits.
// (With the limit a parameter of the kernel, 64 sequences' single tokens took
// 225 us for 200.)
__device__ __forceinline__ bool wait_for(uint64_t* b, uint32_t parity, volatile int* going, uint32_t limit = kWaitLimit) {
  const uint32_t a = smem_u32(b);
#pragma unroll 1
  for (uint32_t it = 0; it < limit; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if (going != nullptr && (it & 255u) == 255u && *going <= 0) return false;
  }
  if (going != nullptr) *going = 0;
  return false;
}
// After giving up: work already issued completes.
__device__ __forceinline__ void drain(uint64_t* b, uint32_t parity) { wait_for(b, parity, nullptr, kDrainLimit); }

__device__ __forceinline__ void bar_arrive(int id, int n) { asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }
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

// Adds the values that are not finite, of the nodes that the row sees, to
// the thread's columns of its row, which it has just written.
template <int D>
__device__ __forceinline__ void add_nonfinite(const PagedAttnParams& p, const Desc& d, int64_t slot, __nv_bfloat16* orow, int col,
                                           int cols, int node, const uint16_t* par, bool whole) {
  while (true) {
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.vt) + d.b * p.kt_sb + static_cast<int64_t>(node) * p.kt_st +
                             static_cast<int64_t>(d.g) * p.kt_sh;
#pragma unroll 1
    for (int e = col; e < col + cols; ++e) {
      const float x = __bfloat162float(v[e]);
      if (fabsf(x) < INFINITY) continue;
      if (whole) orow[e] = __float2bfloat16(__bfloat162float(orow[e]) + x);
      else p.part_o[slot * D + e] += x;
    }
    const uint16_t up = par[node];
    if (up >= kRootMark) break;
    node = up;
  }
}

// The rows of a piece by one warp, without keys (a unit that has none, or tree
// tiles of later nodes alone) or as NaN.
template <int D>
__device__ __forceinline__ void fill_rows(const PagedAttnParams& p, const Desc& d, int64_t slot, bool nan) {
  const int lane = threadIdx.x & 31;
  const float x = nan ? NAN : 0.f, z = nan ? NAN : -INFINITY;
  const uint32_t xx = pack_bf16(x, x);
#pragma unroll 1
  for (int e = lane; e < d.nodes * p.G * (D / 8); e += 32) {
    const int r = e / (D / 8), col = e % (D / 8) * 8;
    if (d.whole) {
      *reinterpret_cast<uint4*>(out_row<__nv_bfloat16>(p, d.b, d.g, d.i0 * p.G + r) + col) = make_uint4(xx, xx, xx, xx);
    } else {
      float4* o = reinterpret_cast<float4*>(p.part_o + (slot + r) * D + col);
      o[0] = o[1] = make_float4(x, x, x, x);
    }
  }
#pragma unroll 1
  for (int r = lane; r < d.nodes * p.G; r += 32) {
    if (!d.whole) p.part_lse[slot + r] = z;
    else if (p.lse) p.lse[lse_row(p, d.b, d.g, d.i0 * p.G + r)] = z;
  }
}

}  // namespace ptc

using namespace ptc;

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_paged_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_kt,
                     const __grid_constant__ CUtensorMap map_vt, PagedAttnParams p) {
  using Sh = Shape<D>;
  constexpr int KS = Sh::kKS, VS = Sh::kVS;
  constexpr uint32_t TB = Sh::kTile;
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ Bars bars;
  __shared__ Line ln;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.G, box = p.box;
  const int align = box > 0 ? box : 8;
  const int npt = p.rows / p.team / G;                    // nodes of a row tile
  const int member = static_cast<int>(blockIdx.x) % p.team;
  const uint32_t raw = smem_u32(dsmem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;           // 128B swizzle atoms are 1 KB
  uint8_t* gbase = dsmem_raw + (base - raw);
  uint16_t* spar = reinterpret_cast<uint16_t*>(gbase + Sh::kPar);
  volatile int* going = &bars.going;

  if (tid >= 32 && tid < 37) {
    const CUtensorMap* m = tid == 32 ? &map_q : (tid == 33 ? &map_k : (tid == 34 ? &map_v : (tid == 35 ? &map_kt : &map_vt)));
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  // (three threads share this while the first warps wait for the lengths)
  if (lane == 0 && (warp == kWarpK || warp == kWarpV || warp == kWarpTree)) {
    if (warp == kWarpK) {
      for (int s = 0; s < KS; ++s) { mbar_init(&bars.k_full[s], 1); mbar_init(&bars.k_empty[s], 1); }
      for (int s = 0; s < VS; ++s) { mbar_init(&bars.v_full[s], 1); mbar_init(&bars.v_empty[s], 1); }
      mbar_init(&bars.q_full, 1); mbar_init(&bars.q_empty, 1);
      mbar_init(&bars.o_full, 1); mbar_init(&bars.o_free, 8);
    } else if (warp == kWarpV) {
      for (int s = 0; s < kSB; ++s) { mbar_init(&bars.s_full[s], 1); mbar_init(&bars.p_full[s], 4); }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&bars.pv_done[s], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&bars.dec[i][s], 1);
        mbar_init(&bars.t_full[s], 1); mbar_init(&bars.t_empty[s], 8);
      }
      bars.going = 1;
      bars.end_at = INT_MAX;
    } else {
      for (int s = 0; s < kRing; ++s) { mbar_init(&bars.w_full[s], 1); mbar_init(&bars.w_empty[s], 11); }
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (tid < 32) bars.vbad[tid >> 4][tid >> 2 & 3][tid & 3] = 0;
  if (tid < 8) bars.bad_piece[tid] = 0;
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  build_line<kKeys, kPagedTcCost, kThreads>(p, ln, align);              // ends with a CTA barrier
  fence_after();
  const uint32_t tmem = bars.tmem_base;

  // Description k, and its release (every consuming warp once per piece);
  // nullptr past the last one, and when it does not come.  Softmax warps
  // ask whether it will: warp 11 describes it or says that it will not, after
  // three waits of its own at most.  (All roles asking: 256 single tokens 190
  // us for 182.)
  auto desc = [&](int k, bool softmax) -> const Desc* {
    uint64_t* w = &bars.w_full[k % kRing];
    const uint32_t parity = (k / kRing) & 1;
    if (!softmax) {
      if (!wait_for(w, parity, nullptr)) {
        *going = 0;
        return nullptr;
      }
    } else {
#pragma unroll 1
      for (uint32_t n = 0; !wait_for(w, parity, nullptr, 1024); ++n)
        if (n == kWaitLimit / 128 || *static_cast<volatile int*>(&bars.end_at) <= k) {
          *going = 0;
          return nullptr;
        }
    }
    const Desc* d = &bars.desc[k % kRing];
    return d->valid ? d : nullptr;
  };
  auto release = [&](int k) { mbar_arrive(&bars.w_empty[k % kRing]); };

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
    auto announce = [&](int s) {                          // copies that have landed, to the tensor cores
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    };
    auto flush = [&]() {
      if (pending < 0) return;
      cp_async_wait_all();
      announce(pending);
      pending = -1;
    };
    auto acquire = [&](int s) -> bool {                   // the stage is free
      if (it < NS) return true;
      bool a = true;
      // (no stage yet: the last tile is announced now instead of after the next one's copies)
      if (pending >= 0 && !__shfl_sync(0xffffffffu, lane == 0 ? mbar_test(&empty[s], ((it / NS) - 1) & 1) : false, 0))
        flush();
      if (lane == 0) a = wait_for(&empty[s], ((it / NS) - 1) & 1, going);
      return __all_sync(0xffffffffu, a);
    };
    for (int k = 0;; ++k) {
      const Desc* d = desc(k, false);
      if (__any_sync(0xffffffffu, !d)) break;
      const int32_t* table = p.table + d->b * p.pt_sb;
      const int L = d->L, g = d->g, b = d->b, a0 = d->a0, a1 = d->a0 + d->na, cnt = d->cnt;
      const int rem = d->rem, off = d->off, nodes = d->n, lo0 = d->lo0;
      auto bad_page = [&]() { if (isk) bars.bad_piece[k & 7] = k + 1; };
      if (box > 0) {
        // lane l holds the run of `box` rows number l % nb of tile l / nb of
        // a batch of 32 / nb tiles; the tile after the last prefix tile may
        // hold the prefix's last rows
        const int nb = kKeys / box, batch = 32 / nb;
        const int stop = a1 + (rem > 0);
        int row = 0, page = 0, row_n = 0, page_n = 0;
        auto look = [&](int t, int& r, int& pg) {
          const unsigned pos = static_cast<unsigned>(t + lane / nb) * kKeys + lane % nb * box;
          r = -1;
          pg = 0;
          if (t + lane / nb < stop && pos < static_cast<unsigned>(L)) {
            r = static_cast<int>(pos % P);
            pg = __ldg(table + pos / P);
          }
        };
        look(a0, row_n, page_n);
        for (int r = 0; ok && r < cnt; ++r, ++it) {
          const int t = a0 + r, q = r % batch;
          if (q == 0) {
            row = row_n;
            page = page_n;
            look(t + batch, row_n, page_n);
          }
          const int s = it % NS;
          ok = acquire(s);
          if (!ok) break;
          const bool mine = lane / nb == q && row >= 0;
          if (mine && (page < 0 || page >= p.num_pages)) {
            bad_page();
            page = p.num_pages;                           // past the pool's end: the box reads as zeros
          }
          uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, mine))) * box * D * 2;
          // tree nodes: boxes of 8 into rows off, off + 8, ...
          const int lo = lo0 - (t - a1) * kKeys;
          const int tb = t >= a1 ? (min(nodes - lo, kKeys - off) + kTreeBox - 1) / kTreeBox : 0;
          bytes += static_cast<uint32_t>(tb) * kTreeBox * D * 2;
          __syncwarp();                                   // a bad page is noted before the tile is announced
          if (lane == 0) mbar_expect_tx(&full[s], bytes);
          __syncwarp();
          const uint32_t dst = ring + s * TB;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            if (mine) tma_load_4d(map, dst + lane % nb * box * 128 + h * kHalfBytes, &full[s], 64 * h, g, row, page);
            if (lane < tb)
              tma_load_4d(map_tree, dst + (off + lane * kTreeBox) * 128 + h * kHalfBytes, &full[s], 64 * h, g,
                          lo + lane * kTreeBox, b);
          }
        }
      } else {
        const char* pool = static_cast<const char*>(isk ? p.kp : p.vp) + g * p.kv_sh * 2;
        const char* tree = static_cast<const char*>(isk ? p.kt : p.vt) + (b * p.kt_sb + g * p.kt_sh) * 2;
        // pages of rows l, l + 32, ... of the next tile, read a tile ahead
        int pg[4];
        auto look = [&](int t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const unsigned pos = static_cast<unsigned>(t) * kKeys + i * 32 + lane;
            pg[i] = pos < static_cast<unsigned>(L) ? __ldg(table + pos / P) : 0;
          }
        };
        look(a0);
        for (int r = 0; ok && r < cnt; ++r, ++it) {
          // lane l looks up rows l, l + 32, l + 64, l + 96: the offset in its
          // source in units of 16 bytes, the top bit for the tree; all ones: no row
          const int t = a0 + r, lo = lo0 - (t - a1) * kKeys;
          const int np = t < a1 ? kKeys : rem;            // prefix rows (as far as the prefix goes)
          const int s = it % NS;
          constexpr int CPR = D / 8, RPI = 32 / CPR;      // 16-byte chunks of a row, rows of a step
          constexpr uint32_t kTree = 0x80000000u, kNone = 0xffffffffu;
          const int ch = lane % CPR;
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = i * 32 + lane;
            o[i] = kNone;
            const unsigned pos = static_cast<unsigned>(t) * kKeys + x;
            if (x < np && pos < static_cast<unsigned>(L)) {
              if (pg[i] < 0 || pg[i] >= p.num_pages) bad_page();
              else o[i] = static_cast<uint32_t>((pg[i] * p.kv_sp + static_cast<int64_t>(pos % P) * p.kv_sr) / 8);
            } else if (t >= a1 && x >= off && lo + x - off < nodes) {
              o[i] = static_cast<uint32_t>(static_cast<int64_t>(lo + x - off) * p.kt_st / 8) | kTree;
            }
          }
          if (r + 1 < cnt) look(t + 1);
          ok = acquire(s);
          if (!ok) break;
          // (one warp issues 2048 copies a tile: what it does for each counts.
          // With 64-bit offsets, the swizzle worked out each time and the
          // pages read when they are needed: 838 us for 64 sequences' decode
          // over pages of 5 rows, so 430; pages of 16 rows take 200)
          uint32_t at[8 / RPI];                           // the chunk's place in rows r0 + lane / CPR, r0 = 0, RPI, ... 8 - RPI
#pragma unroll
          for (int i = 0; i < 8 / RPI; ++i) {
            const int rr = i * RPI + lane / CPR;
            at[i] = ring + s * TB + ch / 8 * kHalfBytes + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
          }
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const uint32_t oi = i < 2 ? (i == 0 ? o[0] : o[1]) : (i == 2 ? o[2] : o[3]);
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += RPI) {
              const uint32_t y = __shfl_sync(0xffffffffu, oi, r0 + lane / CPR);
              const char* src = (y & kTree ? tree : pool) + static_cast<uint64_t>(y & ~kTree) * 16;
              if (y != kNone) cp_async16(at[r0 / RPI % (8 / RPI)] + (i * 32 + r0 / 8 * 8) * 128, src + ch * 16);
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (pending >= 0) {                             // the tile before this one has landed
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            announce(pending);
          }
          pending = s;
        }
      }
      __syncwarp();
      if (lane == 0) release(k);
    }
    flush();
    // drain: every issued load lands before the CTA can exit
    if (lane == 0)
#pragma unroll 1
      for (int j = (it > NS ? it - NS : 0); j < it; ++j) drain(&full[j % NS], (j / NS) & 1);
    __syncwarp();
  } else if (warp == kWarpTree) {
    // ------------------------------------------------------------ pieces, Q and parent[]
    int nq = 0, ntree = 0, made = 0, pos = ln.first;
    bool ok = true, more = true, failed = false;
    SplitUnit split = {-1, 0, 0, 0, 0};
    auto make = [&]() {                                   // description number `made`
      const int s = made % kRing;
      if (made >= kRing || p.lost == kLostPieces) {
        bool a = true;
        if (lane == 0) {
          if (made >= kRing) a = wait_for(&bars.w_empty[s], ((made / kRing) - 1) & 1, going);
          if (p.lost == kLostPieces && made > 0 && !failed) a = false;
          if (!a) {
            *going = 0;
            *static_cast<volatile int*>(&bars.end_at) = made;
          }
        }
        more = __all_sync(0xffffffffu, a);
        if (!more) return;
      }
      Desc x;
      x.valid = 0;
#pragma unroll 1
      while (!x.valid && pos < ln.last) {
        const Piece c = piece_at<kKeys>(p, ln, pos, align);
        pos = c.next;
        if (c.t0 >= c.t1) continue;
        const int unit_i0 = c.rt * npt * p.team;
        x.whole = c.t0 == 0 && c.t1 == c.s.tiles;
        x.begins = c.t0 == 0;
        if (x.begins && !x.whole) split = split_of(ln, c, unit_i0 * G, min(npt * p.team, c.s.n - unit_i0) * G);
        x.b = c.b; x.g = c.g; x.i0 = unit_i0 + member * npt;
        x.nodes = min(npt, c.s.n - x.i0);
        if (x.nodes <= 0) continue;                       // a team mate's row tile is the last
        x.n = c.s.n; x.L = c.s.L;
        x.bad_len = c.s.bad_len;
        x.a0 = min(c.t0, c.s.nprefix);
        x.na = min(c.t1, c.s.nprefix) - x.a0;
        // tree tiles of later nodes than the row tile's are left out
        const int skip = c.s.ntree > 0 ? c.s.ntree - ((x.i0 + x.nodes - 1) / kKeys + 1) : 0;
        const int b0 = max(c.t0, c.s.nprefix + skip), b1 = min(c.t1, c.s.nprefix + c.s.ntree);
        x.ntr = max(0, b1 - b0);
        x.lo0 = (c.s.ntree - 1 - (b0 - c.s.nprefix)) * kKeys;
        x.rem = x.ntr > 0 ? c.s.rem : 0;
        x.off = x.ntr > 0 ? c.s.off : 0;
        x.cnt = x.na + x.ntr;
        x.valid = x.cnt > 0 && !failed;
        if (!x.valid) fill_rows<D>(p, x, part_slot(p, ln.stretch, x.begins) + member * npt * G, failed || x.bad_len);
      }
      more = x.valid;
      if (failed) return;
      if (lane == 0) {
        bars.desc[s] = x;
        mbar_arrive(&bars.w_full[s]);
      }
      __syncwarp();
      ++made;
    };
    while (true) {
      for (int k = 0;; ++k) {
#pragma unroll 1
        while (more && made <= (k == 0 ? 0 : k + kAhead)) make(); // (the first piece's Q before its successors)
        if (k >= made) break;
        const Desc& d = bars.desc[k % kRing];             // (kept: this warp makes its successor in the ring)
        if (!d.valid) break;
        if (!ok) continue;
        bool a = true;
        if (nq > 0 && lane == 0) a = wait_for(&bars.q_empty, (nq - 1) & 1, going);
        ok = __all_sync(0xffffffffu, a);
        if (!ok) continue;
        if (lane == 0) {
          // rows past the tensor's nodes read as zeros
          mbar_expect_tx(&bars.q_full, static_cast<uint32_t>(npt * G) * D * 2);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(&map_q, base + Sh::kQ + h * kHalfBytes, &bars.q_full, 64 * h, d.g * G, d.i0, d.b);
        }
        ++nq;
        if (d.ntr > 0) {
          const int buf = ntree & 1;
          if (ntree >= 2 && lane == 0) a = wait_for(&bars.t_empty[buf], ((ntree >> 1) - 1) & 1, going);
          ok = __all_sync(0xffffffffu, a);
          if (!ok) continue;
          const int32_t* par = p.parent + d.b * p.par_sb;
#pragma unroll 1
          for (int j = lane; j < d.i0 + d.nodes; j += 32) {
            const int pj = par[j];
            spar[buf * kMaxT + j] = j == 0 ? (pj == -1 ? kRootMark : kBadMark)
                                           : ((pj >= 0 && pj < j) ? static_cast<uint16_t>(pj) : kBadMark);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.t_full[buf]);
          ++ntree;
        }
      }
      if (failed) break;
      if (lane == 0 && nq > 0) drain(&bars.q_full, (nq - 1) & 1);
      // the softmax warps have written their last row
      bar_sync(4, kSoftmaxThreads + 32);
      failed = __any_sync(0xffffffffu, *going == 0);
      if (!failed) break;
      // the other roles that wait for a description that will not come find an end
      if (lane == 0) {
        *static_cast<volatile int*>(&bars.desc[made % kRing].valid) = 0;
        mbar_arrive(&bars.w_full[made % kRing]);
      }
      // the whole stretch again, every row NaN
      pos = ln.first;
      made = 0;
      more = true;
      if (lane == 0) set_status(p.status, TV_DEV_TIMEOUT);
    }
    if (lane == 0 && member == 0) p.splits[ln.stretch] = split;
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc_qk = instr_desc(kRows, kKeys, 0, 0);
      const uint32_t idesc_pv = instr_desc(kRows, D, 0, 1);
      int is = 0, ip = 0;                                 // S and P V issued in all
      int rs = 0, rp = 0;                                 // of those, in the present pieces
      int ks = -1, kp = -1;                               // the present pieces
      const Desc *ds = nullptr, *dp = nullptr;
      int cnt_s = 0, cnt_p = 0;                           // tiles of the present pieces
      int na = 0, keys0 = 0, nodes = 0, lo0 = 0, off = 0; // of the piece of the next P V
      auto next_s = [&]() {
        ds = desc(++ks, false);
        if (ds) cnt_s = ds->cnt;
        rs = 0;
      };
      auto next_p = [&]() {
        if (kp >= 0) release(kp);
        dp = desc(++kp, false);
        if (dp) {
          cnt_p = dp->cnt;
          na = dp->na; keys0 = dp->L - dp->a0 * kKeys; nodes = dp->n; lo0 = dp->lo0; off = dp->off;
        }
        rp = 0;
      };
      next_s();
      next_p();
      if (p.lost == kLostProducts && dp) {
        dp = nullptr;
        *going = 0;
      }
      uint32_t idle = 0;
      while (dp) {
        const uint32_t par = static_cast<uint32_t>((is / KS) & 1) | static_cast<uint32_t>(ks & 1) << 1 |
                             static_cast<uint32_t>((ip / VS) & 1) << 2 | static_cast<uint32_t>((ip / kSB) & 1) << 3 |
                             static_cast<uint32_t>((kp - 1) & 1) << 4;
        const uint32_t got = mbar_test5(smem_u32(&bars.k_full[is % KS]), smem_u32(&bars.q_full), smem_u32(&bars.v_full[ip % VS]),
                                        smem_u32(&bars.p_full[ip % kSB]), smem_u32(&bars.o_free), par);
        const bool want_s = ds && is < ip + kSB, want_p = ip < is;
        bool did = false;
        // O += P V: P is bf16 pairs over the first 64 columns of its S.  The
        // first product of a piece overwrites O, so the last piece's must have been read.
        if (want_p && (got & 12u) == 12u && (rp > 0 || kp == 0 || (got & 16u))) {
          fence_after();
          const uint64_t dv = smem_desc(base + Sh::kV + (ip % VS) * TB, kHalfBytes, 1024);
          const uint32_t od = tmem + kColO, pd = tmem + kColS + (ip % kSB) * 128;
          const int end = rp < na ? min(kKeys, keys0 - rp * kKeys) : off + min(nodes - (lo0 - (rp - na) * kKeys), kKeys - off);
          const int steps = (end + 15) / 16;              // K steps up to the tile's last key
          // (16 rows of V are 2 KB; unrolled for the tiles that count: issued
          // from a loop, a tile's 8 MMAs took 1000 cycles instead of 550)
          if (steps == 8) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) mma_bf16_ts(od, pd + kk * 8, dv + kk * 128, idesc_pv, (rp > 0 || kk > 0) ? 1u : 0u);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < steps; ++kk)
              mma_bf16_ts(od, pd + kk * 8, dv + kk * 128, idesc_pv, (rp > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(&bars.v_empty[ip % VS]);
          mma_commit(&bars.pv_done[ip & 1]);
          ++ip;
          if (++rp == cnt_p) {
            mma_commit(&bars.o_full);
            next_p();
          }
          did = true;
        }
        if (want_s && (got & 1u) && (rs > 0 || (got & 2u))) {
          fence_after();
          const uint64_t dq = smem_desc(base + Sh::kQ, 16, 1024), dk = smem_desc(base + Sh::kK + (is % KS) * TB, 16, 1024);
          const uint32_t sd = tmem + kColS + (is % kSB) * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {           // (16 columns are 32 B, 64 a half tile)
            const uint32_t o = (kk >> 2) * (kHalfBytes >> 4) + (kk & 3) * 2;
            mma_bf16(sd, dq + o, dk + o, idesc_qk, kk > 0);
          }
          mma_commit(&bars.k_empty[is % KS]);
          mma_commit(&bars.s_full[is % kSB]);
          ++is;
          if (++rs == cnt_s) {
            mma_commit(&bars.q_empty);
            next_s();
          }
          did = true;
        }
        if (did) {
          idle = 0;
        } else if (++idle >= kWaitLimit || ((idle & 255u) == 255u && *going == 0)) {
          *going = 0;
          break;
        }
      }
      if (*going == 0) {
        // what was issued completes before the TMEM is freed
#pragma unroll 1
        for (int j = is > kSB ? is - kSB : 0; j < is; ++j) drain(&bars.s_full[j % kSB], (j / kSB) & 1);
#pragma unroll 1
        for (int j = ip > 2 ? ip - 2 : 0; j < ip; ++j) drain(&bars.pv_done[j & 1], (j >> 1) & 1);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warps 0-7
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int row = tid & (kRows - 1), half = tid >> 7;   // half: the warpgroup
    const float sl2 = p.scale * 1.4426950408889634f;      // scores in log2 units
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t ocol = trow + kColO;
    int it0 = 0, ntree = 0, nfix = 0;                     // tiles, tree pieces, the group's tree tiles before this piece
    bool ok = true;
    for (int k = 0;; ++k) {
      const Desc* d = desc(k, true);
      if (!d) break;
      const int my_rows = d->nodes * G;
      const bool live = (warp & 3) * 32 < my_rows;        // the warp has valid rows
      const bool row_valid = row < my_rows;
      const int my_node = d->i0 + row / G;
      const int na = d->na, cnt = d->cnt, nodes = d->n, rem = d->rem, off = d->off, lo0 = d->lo0;
      const int keys0 = d->L - d->a0 * kKeys;             // prefix keys from the piece's first tile on
      float m_run = -INFINITY, l_run = 0.f;               // the maximum that l_run refers to
      bool my_ok = true, nf = false;
      int cur = -2;                                       // walk position on this row's root path (-2: not begun)
      const uint16_t* par = spar + (ntree & 1) * kMaxT;
      for (int r = (half ^ it0) & 1; r < cnt; r += 2) {
        const int it = it0 + r, sb = it % kSB;
        const uint32_t scol = trow + kColS + 128u * static_cast<uint32_t>(sb);
        const bool tree = r >= na;
        const int lo = lo0 - (r - na) * kKeys;            // tree tile: its first node
        // keys [0, np) of the prefix, [off, end) of the tree
        const int np = tree ? rem : min(kKeys, keys0 - r * kKeys);
        const int end = tree ? off + min(nodes - lo, kKeys - off) : np;
        const bool full = np == kKeys;
        // keys that the row sees
        uint32_t mk[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (!full) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int nh = np - 32 * i;
            mk[i] = nh >= 32 ? 0xffffffffu : (nh <= 0 ? 0u : ((1u << nh) - 1u));
          }
        }
        if (tree) {
          if (cur == -2) {
            ok = ok && __all_sync(0xffffffffu, wait_for(&bars.t_full[ntree & 1], (ntree >> 1) & 1, going));
            cur = row_valid && ok ? my_node : -1;
          }
#pragma unroll 1
          while (cur >= lo) {
            const int x = cur - lo + off;
#pragma unroll
            for (int i = 0; i < 4; ++i) mk[i] |= (x >> 5) == i ? 1u << (x & 31) : 0u;
            const uint16_t up = par[cur];
            my_ok = my_ok && up != kBadMark;
            cur = up >= kRootMark ? -1 : static_cast<int>(up);
          }
        }
        ok = ok && __all_sync(0xffffffffu, wait_for(&bars.s_full[sb], (it / kSB) & 1, going));
        fence_after();
        if (live && ok) {
          // S is masked where it lies and read again for the weights, in loops, a
          // quarter of the code of holding it in registers: 256 sequences' single
          // tokens 162 us for 179 with d = 128, 171 for 210 with d = 64; 64
          // sequences' single tokens 193 for 198, trees the same.
          if (!full) {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              const uint32_t w = q < 2 ? (q == 0 ? mk[0] : mk[1]) : (q == 2 ? mk[2] : mk[3]);
              float z[32];
              tmem_ld32(scol + q * 32, z);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) z[x] = ((w >> x) & 1u) ? z[x] : -INFINITY;
              tmem_st16(scol + q * 32, z);
              tmem_st16(scol + q * 32 + 16, z + 16);
            }
            tmem_wait_st();
          }
          float s[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(scol + q * 32, s + q * 32);
          tmem_wait_ld();
          float mx[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) mx[x] = fmaxf(s[x], s[x + 8]);
#pragma unroll
          for (int x = 16; x < 128; x += 2) mx[(x >> 1) & 7] = max3(mx[(x >> 1) & 7], s[x], s[x + 1]);
          const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sl2;
          // the row's reference maximum after the tile before
          float m = -INFINITY;
          if (r > 0) {
            ok = __all_sync(0xffffffffu, wait_for(&bars.dec[warp & 3][half ^ 1], ((it - 1) >> 1) & 1, going));
            m = bars.m_ref[row];
          }
          const float m_new = fmaxf(m, mt);
          const bool grow = m_new > m + 8.0f;             // also the first finite maximum
          if (__any_sync(0xffffffffu, grow) && r > 0 && ok) {
            // O holds the tiles before this one: wait for the last P V, then rescale
            ok = __all_sync(0xffffffffu, wait_for(&bars.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, going));
            fence_after();
            const float factor = grow ? ex2_approx(m - m_new) : 1.f;   // 0 when m = -inf
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              float o[16];
              tmem_ld16(ocol + q * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= factor;
              tmem_st16(ocol + q * 16, o);
            }
            tmem_wait_st();
          }
          if (grow) m = m_new;
          if (grow || r == 0) bars.m_ref[row] = m;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.dec[warp & 3][half]);
          if (m != m_run) {
            l_run = m_run == -INFINITY ? 0.f : l_run * ex2_approx(m_run - m);
            m_run = m;
          }
          const float nmu = (m_run == -INFINITY) ? 0.f : -m_run;
          // p = 2^(s sl2 - m) as bf16 pairs over the first half of S
          float2 ps[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
          const float2 sl = make_float2(sl2, sl2), nm = make_float2(nmu, nmu);
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float z[32];
            uint32_t pk[16];
            tmem_ld32(scol + q * 32, z);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              float2 e = fma2(make_float2(z[x], z[x + 1]), sl, nm);
              e.x = ex2_approx(e.x);
              e.y = ex2_approx(e.y);
              ps[(x >> 1) & 3] = add2(ps[(x >> 1) & 3], e);
              pk[x / 2] = pack_bf16(e.x, e.y);
            }
            tmem_st16u(scol + q * 16, pk);
          }
          const float2 sum = add2(add2(ps[0], ps[1]), add2(ps[2], ps[3]));
          l_run += sum.x + sum.y;
          tmem_wait_st();
        } else if (lane == 0) {
          mbar_arrive(&bars.dec[warp & 3][half]);
        }
        if (!full) {
          // V rows of the K steps that are no keys are cleared, nodes' rows looked over
          ok = ok && __all_sync(0xffffffffu, wait_for(&bars.v_full[it % VS], (it / VS) & 1, going));
          uint8_t* v0 = gbase + Sh::kV + (it % VS) * TB;
          uint32_t* vbad = bars.vbad[half][nfix & 3];
          auto chunk = [&](int x, int ch) {
            return reinterpret_cast<uint4*>(v0 + x * 128 + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (x & 7)) << 4));
          };
          constexpr int CPR = D / 8;
          if (ok) {
            const int top = (end + 15) & ~15;
#pragma unroll 1
            for (int e = tid & 127; e < (top - np) * CPR; e += 128) {
              const int x = np + e / CPR;
              if (!tree || x < off || x >= end) *chunk(x, e % CPR) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (tree) {
#pragma unroll 1
              for (int e = tid & 127; e < (end - off) * CPR; e += 128) {
                const int x = off + e / CPR;
                uint4* at = chunk(x, e % CPR);
                const uint4 v = *at;
                uint32_t u[4] = {v.x, v.y, v.z, v.w};
                bool h = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if ((u[i] & 0x7f80u) == 0x7f80u) { u[i] &= 0xffff0000u; h = true; }
                  if ((u[i] & 0x7f800000u) == 0x7f800000u) { u[i] &= 0xffffu; h = true; }
                }
                if (h) {
                  *at = make_uint4(u[0], u[1], u[2], u[3]);
                  atomicOr(vbad + (x >> 5), 1u << (x & 31));
                }
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          // every warp of the group comes here for every tree tile, whatever has happened
          if (tree) bar_sync(2 + half, 128);
        }
        if (tree) {
          const volatile uint32_t* vbad = bars.vbad[half][nfix & 3];
#pragma unroll
          for (int i = 0; i < 4; ++i) nf = nf || (vbad[i] & mk[i]);
          // the slot after next was last read two tree tiles ago
          if ((tid & 127) < 4) bars.vbad[half][(nfix + 2) & 3][tid & 3] = 0;
          ++nfix;
        }
        fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&bars.p_full[sb]);
      }
      // ---------------------------------------------------------- output
      it0 += cnt;
      ok = ok && __all_sync(0xffffffffu, wait_for(&bars.o_full, k & 1, going));
      // the groups' sums meet at the larger of their maxima, O's reference:
      // out = O / (2^(m_0 - M) l_0 + 2^(m_1 - M) l_1); group h writes half of the columns
      bars.red_m[half][row] = m_run;
      bars.red_l[half][row] = l_run;
      bars.red_nf[half][row] = nf + 2 * !my_ok;
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
      const bool bad = d->bad_len || !my_ok || !ok || bars.bad_piece[k & 7] == k + 1;
      const bool empty = l_row == 0.f;
      const float inv = bad ? NAN : (empty ? 0.f : 1.f / l_row);
      const bool whole = d->whole;
      const int packed = d->i0 * G + row;
      const int64_t slot = part_slot(p, ln.stretch, d->begins ? 1 : 0) + member * npt * G + row;
      if (live) {
        __nv_bfloat16* orow = row_valid ? out_row<__nv_bfloat16>(p, d->b, d->g, packed) : nullptr;
        constexpr int NC = D / 2;                         // columns of a thread
#pragma unroll 1
        for (int q = 0; q < NC / 32; ++q) {
          const int col = half * NC + q * 32;
          float v0[32];
          tmem_ld32(ocol + col, v0);
          tmem_wait_ld();
          if (!row_valid) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            v0[e] = bad ? NAN : (empty ? 0.f : v0[e] * inv);
          if (whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4 x;
              x.x = pack_bf16(v0[8 * e], v0[8 * e + 1]);
              x.y = pack_bf16(v0[8 * e + 2], v0[8 * e + 3]);
              x.z = pack_bf16(v0[8 * e + 4], v0[8 * e + 5]);
              x.w = pack_bf16(v0[8 * e + 6], v0[8 * e + 7]);
              *reinterpret_cast<uint4*>(orow + col + 8 * e) = x;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(p.part_o + slot * D + col + 4 * e) =
                  make_float4(v0[4 * e], v0[4 * e + 1], v0[4 * e + 2], v0[4 * e + 3]);
          }
        }
        if (nf && row_valid && !bad) add_nonfinite<D>(p, *d, slot, orow, half * NC, NC, my_node, par, whole);
        if (half == 0 && row_valid) {
          const float lse2 = bad ? NAN : (empty ? -INFINITY : M + log2f(l_row));
          if (!whole) p.part_lse[slot] = lse2;
          else if (p.lse) p.lse[lse_row(p, d->b, d->g, packed)] = lse2 * kLn2;
          if (!my_ok) set_status(p.status, TV_DEV_BAD_PARENT);
        }
      }
      // O and parent[] are free for the pieces to come
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.o_free);
      if (d->ntr > 0) {
        if (lane == 0) mbar_arrive(&bars.t_empty[ntree & 1]);
        ++ntree;
      }
      if (tid == 0 && bars.bad_piece[k & 7] == k + 1) set_status(p.status, TV_DEV_BAD_PAGE);
      bar_sync(1, kSoftmaxThreads);                       // red_*, m_ref: read by all
      __syncwarp();
      if (lane == 0) release(k);
    }
    bar_arrive(4, kSoftmaxThreads + 32);                  // (warp 11)
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

template <int D>
cudaError_t launch(const PagedAttnParams& p, int grid, const CUtensorMap* m, cudaStream_t stream) {
  constexpr size_t smem = Shape<D>::kBytes + 1024;
  const cudaError_t e = cudaFuncSetAttribute(attn_paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  attn_paged_tc_kernel<D><<<grid, kThreads, smem, stream>>>(m[0], m[1], m[2], m[3], m[4], p);
  return cudaGetLastError();
}

std::atomic<int> g_lost{0};

}  // namespace

void attn_paged_set_lost(int lost) { g_lost = lost; }

int attn_paged_tc_box(int P) {
  int b = 128;
  while (b >= 8 && P % b != 0) b /= 2;
  return b >= 8 ? b : 0;
}

// As many CTAs to a team as a sequence can have row tiles, four at most (then
// the other row tiles read the keys again).  64 nodes of 4 heads, two tiles:
// 249 us, 284 with teams of one.  40 nodes of 8 heads, three: 214, 227 with
// teams of one and 264 with teams of four, whose last CTA has nothing to do.
// 64 nodes of 8 heads, four: 260, 262 with teams of two, 290 of one.
int attn_paged_tc_team(const tv_attn_paged_args* a) {
  const int G = a->Hq / a->Hkv, npt = kRows / G;
  const int tiles = (a->T + npt - 1) / npt;
  return std::min(tiles, 4);
}

bool attn_paged_tc_supported(const tv_attn_paged_args* a) {
  if (a->dtype != TV_BF16 || (a->d != 64 && a->d != 128)) return false;
  if (a->B == 0 || a->T == 0 || a->T > kMaxT || a->num_pages == 0 || a->max_pages == 0) return false;
  if (!stride_ok(a->Hq, a->q_sh) || !stride_ok(a->T, a->q_st) || !stride_ok(a->B, a->q_sb)) return false;
  if (!stride_ok(a->Hkv, a->kv_sh) || !stride_ok(a->page_size, a->kv_sr) || !stride_ok(a->num_pages, a->kv_sp)) return false;
  if (!stride_ok(a->Hkv, a->kt_sh) || !stride_ok(a->T, a->kt_st) || !stride_ok(a->B, a->kt_sb)) return false;
  if (!stride_ok(a->Hq, a->o_sh) || !stride_ok(a->T, a->o_st) || !stride_ok(a->B, a->o_sb)) return false;
  // row by row, a row's place in its pool is 31 bits of 16-byte units
  constexpr int64_t kMost = 1ll << 34;
  const int64_t page = std::max(stride_or(a->num_pages, a->kv_sp), stride_or(a->page_size, a->kv_sr) * a->page_size);
  if (attn_paged_tc_box(a->page_size) == 0 &&
      (page >= kMost / a->num_pages || stride_or(a->T, a->kt_st) >= kMost / a->T))
    return false;
  const uintptr_t al = reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->k_pages) |
                       reinterpret_cast<uintptr_t>(a->v_pages) | reinterpret_cast<uintptr_t>(a->k_tree) |
                       reinterpret_cast<uintptr_t>(a->v_tree) | reinterpret_cast<uintptr_t>(a->out);
  return (al & 15u) == 0 && tcmap::encode_fn() != nullptr;
}

cudaError_t launch_attn_paged_tc(PagedAttnParams& p, int grid, cudaStream_t stream) {
  CUtensorMap m[5];
  p.lost = g_lost;
  const int tile = kRows / p.G * p.G;
  auto map = [&](CUtensorMap* t, const void* x, int64_t d1, int64_t d2, int64_t d3, int64_t s1, int64_t s2, int64_t s3,
                 int b1, int b2) {
    return tcmap::make_map(t, x, p.d, d1, d2, d3, stride_or(d1, s1), stride_or(d2, s2), stride_or(d3, s3), b1, b2);
  };
  if (!map(&m[0], p.q, p.Hq, p.T, p.B, p.q_sh, p.q_st, p.q_sb, p.G, tile / p.G) ||
      !map(&m[3], p.kt, p.Hkv, p.T, p.B, p.kt_sh, p.kt_st, p.kt_sb, 1, kTreeBox) ||
      !map(&m[4], p.vt, p.Hkv, p.T, p.B, p.kt_sh, p.kt_st, p.kt_sb, 1, kTreeBox))
    return cudaErrorInvalidValue;
  if (p.box > 0) {
    if (!map(&m[1], p.kp, p.Hkv, p.page_size, p.num_pages, p.kv_sh, p.kv_sr, p.kv_sp, 1, p.box) ||
        !map(&m[2], p.vp, p.Hkv, p.page_size, p.num_pages, p.kv_sh, p.kv_sr, p.kv_sp, 1, p.box))
      return cudaErrorInvalidValue;
  } else {
    m[1] = m[3];
    m[2] = m[4];
  }
  return p.d == 64 ? launch<64>(p, grid, m, stream) : launch<128>(p, grid, m, stream);
}

}  // namespace tv
