// tree_verify_attn_paged on CUDA cores: fp32, and the shapes the tensor-core
// kernel does not take.
//
// A CTA works through its stretch of the line (attn_paged.cuh) piece by
// piece, in key tiles of 64: K and V rows are staged in shared memory as
// fp32 and used by the R packed (node, head) rows of the tile, four rows to
// a warp.  With few rows (decoding: R = 4) the warps split the tile's keys
// instead, WK ways, each with an online softmax of its own that is combined
// at the end of the piece, so every warp has work at every shape.
//   S    a lane takes 64 / (32 WK) keys (or 32 WK / 64 lanes share one key's
//        d); per 16 bytes of K it does 16 FMAs (4 rows);
//   P V  a lane takes d / 32 columns; per V load it does 4 rows.
// Bound by the shared-memory reads of that arithmetic where rows are many (16
// sequences of 8 nodes of 4 heads on 512 to 4096 rows, fp32: 246 us, 19
// TFLOP/s), by the latencies of start, tiles and merge where they are few (3
// sequences of 15 nodes on 97 to 1009 rows: 16.6 us).  bf16 with d = 32 on the
// first of these: 124 us.  A tree of 3000 nodes of 8 heads, bf16, d = 128: 1.55
// ms, since every row tile goes through all tiles of earlier nodes.
#include <algorithm>

#include "attn_paged.cuh"

namespace tv {

using namespace paged;

namespace simt {

constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kKeys = 64;
constexpr int kRowsPerWarp = 4;

template <int D>
constexpr int kStride = D + 4;                     // rows of K 16 bytes apart in the banks

template <int D, int WK>
constexpr size_t smem_bytes() {
  return sizeof(float) * ((kRowsPerWarp * kWarps / WK) * D + kKeys * kStride<D> + kKeys * D +
                          kWarps * kRowsPerWarp * (kKeys / WK));
}

// 4 consecutive elements as fp32.
__device__ __forceinline__ float4 ld4(const float* s) { return __ldg(reinterpret_cast<const float4*>(s)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* s) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(s));
  const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&u.x);
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&u.y);
  return make_float4(__low2float(a), __high2float(a), __low2float(b), __high2float(b));
}
template <typename T>
__device__ __forceinline__ float4 ld4_any(const T* s, bool vec) {
  if (vec) return ld4(s);
  return make_float4(to_f32(s[0]), to_f32(s[1]), to_f32(s[2]), to_f32(s[3]));
}

}  // namespace simt

using namespace simt;

template <typename T, int D, int WK>
__global__ void __launch_bounds__(kThreads)
attn_paged_simt_kernel(PagedAttnParams p, int vec) {
  constexpr int WR = kWarps / WK;                  // warps along the rows
  constexpr int R = kRowsPerWarp * WR;             // rows of a tile
  constexpr int KW = kKeys / WK;                   // keys of a warp
  constexpr int KPL = KW >= 32 ? KW / 32 : 1;      // keys of a lane
  constexpr int LPK = KW >= 32 ? 1 : 32 / KW;      // lanes of a key
  constexpr int DL = D / 32;
  constexpr int KS = kStride<D>;
  extern __shared__ __align__(16) float smem_f[];
  __shared__ Line ln;
  __shared__ int64_t koff[2][kKeys];               // element offset of a key's row; -1: no key
  __shared__ uint64_t vis[R];                      // tree tile: keys that the row sees
  __shared__ int s_cur[R];                         // walk position on the row's root path
  __shared__ int s_bad, s_badrow[R];
  float* qs = smem_f;                              // [R][D]
  float* ks = qs + R * D;                          // [64][D + 4]
  float* vs = ks + kKeys * KS;                     // [64][D]
  float* ps = vs + kKeys * D;                      // [warp][4][KW]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp / WK, wk = warp % WK;
  const int G = p.G;
  build_line<kKeys, kPagedSimtCost, kThreads>(p, ln, 0);
  SplitUnit split = {-1, 0, 0, 0, 0};

  for (int pos = ln.first; pos < ln.last;) {
    const Piece c = piece_at<kKeys>(p, ln, pos, 0);
    pos = c.next;
    if (c.t0 >= c.t1) continue;
    const int n = c.s.n, L = c.s.L;
    const int packed0 = c.rt * R;
    const int rows = min(R, n * G - packed0);
    const int node_hi = (packed0 + rows - 1) / G;  // last node of the tile
    const int32_t* par = p.parent + c.b * p.par_sb;
    const int32_t* table = p.table + c.b * p.pt_sb;
    __syncthreads();                               // the last piece's shared memory is free
    for (int e = tid; e < R * D / 4; e += kThreads) {
      const int r = e / (D / 4), dd = (e % (D / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int node = (packed0 + r) / G, head = c.g * G + (packed0 + r) % G;
        v = ld4_any(static_cast<const T*>(p.q) + c.b * p.q_sb + static_cast<int64_t>(node) * p.q_st +
                        static_cast<int64_t>(head) * p.q_sh + dd, vec & 1);
        v.x *= p.scale; v.y *= p.scale; v.z *= p.scale; v.w *= p.scale;
      }
      *reinterpret_cast<float4*>(qs + r * D + dd) = v;
    }
    if (tid < R) {
      s_cur[tid] = (tid < rows) ? (packed0 + tid) / G : -1;
      s_badrow[tid] = 0;
    }
    if (tid == 0) s_bad = 0;
    float m[4], l[4], acc[4][DL];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY; l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < DL; ++e) acc[r][e] = 0.f;
    }
    // where key k of tile t lies; tree tiles run from the last one down
    auto locate = [&](int t, int k) -> int64_t {
      if (t < c.s.nprefix) {
        const unsigned j = static_cast<unsigned>(t) * kKeys + k, P = p.page_size;
        if (j >= static_cast<unsigned>(L)) return -1;
        const int page = table[j / P];
        if (page < 0 || page >= p.num_pages) { s_bad = 1; return -1; }
        return page * p.kv_sp + static_cast<int64_t>(j % P) * p.kv_sr + c.g * p.kv_sh;
      }
      const int j = (c.s.ntree - 1 - (t - c.s.nprefix)) * kKeys + k;
      return j < n ? c.b * p.kt_sb + static_cast<int64_t>(j) * p.kt_st + c.g * p.kt_sh : -1;
    };
    const int tend = min(c.t1, c.s.nprefix + c.s.ntree);
    __syncthreads();                               // s_bad is reset before any key is located
    if (tid < kKeys && c.t0 < tend) koff[c.t0 & 1][tid] = locate(c.t0, tid);
    for (int t = c.t0; t < tend; ++t) {
      const bool tree = t >= c.s.nprefix;
      const int lo = tree ? (c.s.ntree - 1 - (t - c.s.nprefix)) * kKeys : 0;
      __syncthreads();                             // koff of tile t; ks, vs free
      if (tid < kKeys && t + 1 < tend) koff[(t + 1) & 1][tid] = locate(t + 1, tid);
      if (tree && lo > node_hi) continue;          // later nodes than any of this row tile
      const T* kb = static_cast<const T*>(tree ? p.kt : p.kp);
      const T* vb = static_cast<const T*>(tree ? p.vt : p.vp);
#pragma unroll 4
      for (int e = tid; e < kKeys * D / 4; e += kThreads) {
        const int k = e / (D / 4), dd = (e % (D / 4)) * 4;
        const int64_t off = koff[t & 1][k];
        float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
        if (off >= 0) {
          kv = ld4_any(kb + off + dd, vec & 2);
          vv = ld4_any(vb + off + dd, vec & 2);
        }
        *reinterpret_cast<float4*>(ks + k * KS + dd) = kv;
        *reinterpret_cast<float4*>(vs + k * D + dd) = vv;
      }
      if (tree && tid < R) {
        // the row's ancestors among nodes lo .. lo + 63; nodes fall along the
        // path, so the walk goes on where the tile above left it
        uint64_t v = 0;
        int cur = s_cur[tid];
        while (cur >= lo) {
          if (cur < lo + kKeys) v |= 1ull << (cur - lo);
          const int up = par[cur];
          if (cur == 0) {
            if (up != -1) s_badrow[tid] = 1;
            cur = -1;
          } else if (up < 0 || up >= cur) {
            s_badrow[tid] = 1;
            cur = -1;
          } else {
            cur = up;
          }
        }
        s_cur[tid] = cur;
        vis[tid] = v;
      }
      __syncthreads();
      if (wr * 4 < rows) {
        // S: 4 rows x this lane's keys
        float s[4][KPL];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < KPL; ++i) s[r][i] = 0.f;
        const int key0 = wk * KW + lane / LPK;
        const int d0 = (lane % LPK) * (D / LPK);
#pragma unroll 4
        for (int dd = 0; dd < D / LPK; dd += 4) {
          float4 kv[KPL];
#pragma unroll
          for (int i = 0; i < KPL; ++i)
            kv[i] = *reinterpret_cast<const float4*>(ks + (key0 + i * 32) * KS + d0 + dd);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(qs + (wr * 4 + r) * D + d0 + dd);
#pragma unroll
            for (int i = 0; i < KPL; ++i)
              s[r][i] = fmaf(qv.x, kv[i].x, fmaf(qv.y, kv[i].y, fmaf(qv.z, kv[i].z, fmaf(qv.w, kv[i].w, s[r][i]))));
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < KPL; ++i) {
#pragma unroll
            for (int o = 1; o < LPK; o <<= 1) s[r][i] += __shfl_xor_sync(0xffffffffu, s[r][i], o);
            const int k = key0 + i * 32;
            const bool ok = tree ? ((vis[wr * 4 + r] >> k) & 1ull) != 0 : koff[t & 1][k] >= 0;
            if (!ok) s[r][i] = -INFINITY;
            mx = fmaxf(mx, s[r][i]);
          }
          mx = warp_max(mx);
          const float mn = fmaxf(m[r], mx);
          const float base = mn == -INFINITY ? 0.f : mn;   // no key yet: every weight is 0
          const float corr = expf(m[r] - base);
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < KPL; ++i) {
            float e = expf(s[r][i] - base);
            // (a key that the row sees has some weight: fp32's least, so that V shows if it is not finite)
            if (tree && e == 0.f && s[r][i] > -INFINITY) e = 0x1p-149f;
            if (lane % LPK == 0) {
              ps[(warp * 4 + r) * KW + lane / LPK + i * 32] = e;
              sum += e;
            }
          }
          l[r] = l[r] * corr + warp_sumf(sum);
          m[r] = mn;
#pragma unroll
          for (int e = 0; e < DL; ++e) acc[r][e] *= corr;
        }
        __syncwarp();
        // O += P V over this warp's keys
        for (int j = 0; j < KW; j += 4) {
          float pr[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *reinterpret_cast<float4*>(pr[r]) = *reinterpret_cast<const float4*>(ps + (warp * 4 + r) * KW + j);
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            float v[DL];
            const float* src = vs + (wk * KW + j + jj) * D + lane * DL;
            if (DL == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
            else if (DL == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
            else v[0] = src[0];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // a tree key that the row does not see weighs nothing, whatever V holds
              if (tree && pr[r][jj] == 0.f) continue;
#pragma unroll
              for (int e = 0; e < DL; ++e) acc[r][e] = fmaf(pr[r][jj], v[e], acc[r][e]);
            }
          }
        }
      }
    }
    __syncthreads();                               // ks, vs: the warps' results
    float* ro = ks;                                // [warp][4][D]
    float* rm = vs;                                // [warp][4] maxima, then sums
    if (WK > 1) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int e = 0; e < DL; ++e) ro[(warp * 4 + r) * D + lane * DL + e] = acc[r][e];
        if (lane == 0) { rm[warp * 4 + r] = m[r]; rm[kWarps * 4 + warp * 4 + r] = l[r]; }
      }
      __syncthreads();
    }
    const bool whole = c.t0 == 0 && c.t1 == c.s.tiles;
    const int which = c.t0 == 0 ? 1 : 0;
    const int64_t slot0 = part_slot(p, blockIdx.x, which);
    // the WK warps of a row share its rows' output
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = wr * 4 + r;
      if (row >= rows || (WK > 1 && r % WK != wk)) continue;
      float M = m[r], den = l[r], o[DL];
#pragma unroll
      for (int e = 0; e < DL; ++e) o[e] = acc[r][e];
      if (WK > 1) {
        M = -INFINITY; den = 0.f;
#pragma unroll
        for (int e = 0; e < DL; ++e) o[e] = 0.f;
        for (int w = 0; w < WK; ++w) M = fmaxf(M, rm[(wr * WK + w) * 4 + r]);
        const float base = M == -INFINITY ? 0.f : M;
        for (int w = 0; w < WK; ++w) {
          const int x = (wr * WK + w) * 4 + r;
          const float f = expf(rm[x] - base);
          den += f * rm[kWarps * 4 + x];
#pragma unroll
          for (int e = 0; e < DL; ++e) o[e] = fmaf(f, ro[x * D + lane * DL + e], o[e]);
        }
      }
      const bool bad = c.s.bad_len || s_bad || s_badrow[row];
      const bool empty = den == 0.f;
      const float inv = bad ? NAN : (empty ? 0.f : 1.f / den);
      const float lse = bad ? NAN : (empty ? -INFINITY : M + logf(den));
      if (whole) {
        T* dst = out_row<T>(p, c.b, c.g, packed0 + row) + lane * DL;
#pragma unroll
        for (int e = 0; e < DL; ++e) dst[e] = static_cast<T>(empty && !bad ? 0.f : o[e] * inv);
        if (lane == 0 && p.lse) p.lse[lse_row(p, c.b, c.g, packed0 + row)] = lse;
      } else {
#pragma unroll
        for (int e = 0; e < DL; ++e) p.part_o[(slot0 + row) * D + lane * DL + e] = empty && !bad ? 0.f : o[e] * inv;
        if (lane == 0) p.part_lse[slot0 + row] = bad ? NAN : lse * 1.4426950408889634f;
      }
    }
    if (tid == 0 && s_bad) set_status(p.status, TV_DEV_BAD_PAGE);
    if (tid < rows && s_badrow[tid]) set_status(p.status, TV_DEV_BAD_PARENT);
    if (c.t0 == 0 && !whole) split = split_of(ln, c, packed0, rows);
  }
  if (tid == 0) p.splits[blockIdx.x] = split;
}

// A warp per row of a split unit:
//   M = max lse, w = 2^(lse - M), out = sum w o / sum w, lse = M + log2 sum w
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_paged_merge_kernel(PagedAttnParams p) {
  constexpr int DL = D / 32;
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kWarps + (threadIdx.x >> 5);
#if defined(__CUDA_ARCH__)
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the first kernel's rows are there
#endif
  const SplitUnit u = p.splits[c0];
  if (u.c1 < 0 || r >= u.rows) return;
  // The pieces in order, U of them in flight (the first lies in the second
  // slot of its stretch, the others in the first), under a running maximum.
  constexpr int U = 16;
  float M = -INFINITY, den = 0.f, acc[DL];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < DL; ++e) acc[e] = 0.f;
  for (int k0 = c0; k0 <= u.c1; k0 += U) {
    float o[U][DL], v[U];
    float m = M;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (k0 + i > u.c1) break;
      const int64_t s = part_slot(p, k0 + i, k0 + i == c0) + r;
      v[i] = p.part_lse[s];
      const float* src = p.part_o + s * D + lane * DL;
      if (DL == 4) *reinterpret_cast<float4*>(o[i]) = *reinterpret_cast<const float4*>(src);
      else if (DL == 2) *reinterpret_cast<float2*>(o[i]) = *reinterpret_cast<const float2*>(src);
      else o[i][0] = src[0];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (k0 + i > u.c1) break;
      bad |= v[i] != v[i];
      m = fmaxf(m, v[i]);
    }
    if (m == -INFINITY) continue;                          // no keys so far
    const float f = exp2f(M - m);
    den *= f;
#pragma unroll
    for (int e = 0; e < DL; ++e) acc[e] *= f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (k0 + i > u.c1) break;
      const float w = exp2f(v[i] - m);
      den += w;
      // (a piece without keys has 0 there; one whose weight is below fp32's range still shows what is not finite)
#pragma unroll
      for (int e = 0; e < DL; ++e) acc[e] = fmaf(w, o[i][e], acc[e]);
    }
    M = m;
  }
  const float inv = bad ? NAN : (den > 0.f ? 1.f / den : 0.f);
  const int packed = u.packed0 + r;
  T* o = out_row<T>(p, u.b, u.g, packed) + lane * DL;
#pragma unroll
  for (int e = 0; e < DL; ++e) o[e] = static_cast<T>(bad ? NAN : acc[e] * inv);
  if (lane == 0 && p.lse)
    p.lse[lse_row(p, u.b, u.g, packed)] = bad ? NAN : (den > 0.f ? (M + log2f(den)) * kLn2 : -INFINITY);
}

namespace {

template <typename T, int D, int WK>
cudaError_t launch(const PagedAttnParams& p, int grid, int vec, cudaStream_t stream) {
  constexpr size_t smem = smem_bytes<D, WK>();
  const cudaError_t e = cudaFuncSetAttribute(attn_paged_simt_kernel<T, D, WK>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  attn_paged_simt_kernel<T, D, WK><<<grid, kThreads, smem, stream>>>(p, vec);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rows(const PagedAttnParams& p, int grid, int vec, cudaStream_t stream) {
  switch (p.rows) {
    case 4: return launch<T, D, 8>(p, grid, vec, stream);
    case 8: return launch<T, D, 4>(p, grid, vec, stream);
    case 16: return launch<T, D, 2>(p, grid, vec, stream);
    default: return launch<T, D, 1>(p, grid, vec, stream);
  }
}

template <typename T>
cudaError_t launch_d(const PagedAttnParams& p, int grid, int vec, cudaStream_t stream) {
  switch (p.d) {
    case 32: return launch_rows<T, 32>(p, grid, vec, stream);
    case 64: return launch_rows<T, 64>(p, grid, vec, stream);
    default: return launch_rows<T, 128>(p, grid, vec, stream);
  }
}

}  // namespace

// Rows of a tile: four to a warp, no more warps along the rows than a
// sequence's rows fill.
int attn_paged_simt_rows(int64_t rows) { return rows > 16 ? 32 : (rows > 8 ? 16 : (rows > 4 ? 8 : 4)); }

namespace {

template <typename T, int D>
cudaError_t merge(const PagedAttnParams& p, int grid, cudaStream_t stream) {
  // The launch may overlap the first kernel's tail: every CTA waits for that kernel to end
  const int most = static_cast<int>(std::min(static_cast<int64_t>(p.rows), static_cast<int64_t>(p.T) * p.G));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (most + kWarps - 1) / kWarps);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_paged_merge_kernel<T, D>, p);
}

template <typename T>
cudaError_t merge_d(const PagedAttnParams& p, int grid, cudaStream_t stream) {
  switch (p.d) {
    case 32: return merge<T, 32>(p, grid, stream);
    case 64: return merge<T, 64>(p, grid, stream);
    default: return merge<T, 128>(p, grid, stream);
  }
}

}  // namespace

cudaError_t launch_attn_paged_merge(const PagedAttnParams& p, int grid, cudaStream_t stream) {
  if (grid == 1) return cudaSuccess;                       // nothing is split
  return p.dtype == TV_BF16 ? merge_d<__nv_bfloat16>(p, grid, stream) : merge_d<float>(p, grid, stream);
}

int attn_paged_simt_ctas(int, int d) { return d == 128 ? 2 : 4; }

cudaError_t launch_attn_paged_simt(const PagedAttnParams& p, int grid, cudaStream_t stream) {
  // 4-element loads (16 bytes of fp32, 8 of bf16) where bases and strides allow: bit 0 q, bit 1 K/V
  const int64_t w = p.dtype == TV_BF16 ? 8 : 16, es = p.dtype == TV_BF16 ? 2 : 4;
  auto ok = [&](const void* x) { return reinterpret_cast<uintptr_t>(x) % w == 0; };
  auto st = [&](int64_t s) { return s * es % w == 0; };
  int vec = 0;
  if (ok(p.q) && st(p.q_sb) && st(p.q_st) && st(p.q_sh)) vec |= 1;
  if (ok(p.kp) && ok(p.vp) && ok(p.kt) && ok(p.vt) && st(p.kv_sp) && st(p.kv_sr) && st(p.kv_sh) && st(p.kt_sb) &&
      st(p.kt_st) && st(p.kt_sh))
    vec |= 2;
  return p.dtype == TV_BF16 ? launch_d<__nv_bfloat16>(p, grid, vec, stream) : launch_d<float>(p, grid, vec, stream);
}

}  // namespace tv
