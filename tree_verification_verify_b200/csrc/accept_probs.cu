// tree_accept_probs: the acceptance walk from given probabilities and given
// uniforms.
//
// One thread-block cluster per sequence walks its tree from the root.  With
// probabilities given, a child's test needs two numbers, p(x) and q(x); the
// kernel fetches them for every node at once at the start.  Only a rejection
// (the residual's sum) or a sample (the inverse CDF) reads a row, so a walk
// costs its few row passes and not a pass per node.
//
// After k rejections at a node the residual is (p - a_k q)^+ / N_k with
//   a_0 = 0, N_0 = 1;  a_{k+1} = a_k + N_k,  N_{k+1} = sum (p - a_{k+1} q)^+
// (when that sum is 0 nothing changes): one multiply-add per element and
// pass whatever k is, and every residual is computed from p and q, not from
// the last one's rounded values.  The child test r(x) / q(x) > u becomes
// u q(x) N < (p(x) - a q(x))^+.
//
// A row pass: the row is cut into consecutive chunks, one per warp of the
// cluster, in order; each warp copies its chunk of p and q into shared memory
// (cp.async, all of it in flight at once) and sums it from there, so the
// second rejection at a node and the final sample read nothing again.  Sums
// are fp64 (a vocabulary of fp32 terms beside a threshold).  Warps' sums meet
// in shared memory, CTAs' sums over distributed shared memory.  A sample
// finds its CTA and warp by the prefix of those sums and scans that warp's
// chunk again.  All CTAs of a cluster hold the same state and take the same
// branches.  The loops over a chunk are kept short and rolled: a walk runs
// them a few times only, and fetching unrolled code took longer than running
// it (a pass of 1200 elements a warp, loads and sums unrolled by 5 steps:
// 6.6 us).
// Bound by the chain of those latencies, not by bytes: one sequence of 5
// nodes over V = 32000 takes 10 to 11 us; 8 sequences of up to 16 nodes over
// V = 152064 17.5 us, 32 of them 38 to 40 (34 to 36 where the rows lie in the
// L2), since a CTA with its rows fills an SM and 256 CTAs are two waves.
// Deterministic trees, p alone: 8.6 and 21 us.  (Two CTAs an SM that hold p
// alone and read q anew each pass: 30 us for 34 there, but 41 for 34 with 128
// sequences over V = 32000, all with rows in the L2.)
#include <cooperative_groups.h>

#include <algorithm>

#include "tv_common.cuh"

namespace cg = cooperative_groups;

namespace tv {

namespace accp {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxC = 8;
constexpr size_t kMaxSmem = 220 * 1024;

struct Params {
  int B, T, V;
  const float* p; int64_t tp_sb, tp_st;
  const float* q; int64_t dp_sb, dp_st;
  const int32_t* tok; int64_t tok_sb;
  const int32_t* par; int64_t par_sb;
  const int32_t* n_nodes;
  const double* u_child;
  const double* u_sample;
  int32_t* n_acc;
  int32_t* acc;
  int32_t* out;
  uint32_t* status;
  int vec;                     // rows start on 16 bytes
  int rows_at;                 // byte offset of the row buffers in dynamic shared memory
  int chunk;                   // elements of a warp's chunk (a multiple of 128)
  int cap;                     // elements of it that shared memory holds at a time (a multiple of 128)
};

__device__ __forceinline__ bool prob_ok(float x) { return x >= 0.f && x < INFINITY; }
__device__ __forceinline__ bool uni_ok(double u) { return u >= 0.0 && u < 1.0; }

// Weight of an element in the residual (a, .): the caller scales by 1 / N.
__device__ __forceinline__ double weight(float p, float q, double a) {
  const double w = fma(-a, static_cast<double>(q), static_cast<double>(p));
  return w > 0.0 ? w : 0.0;
}

// The row passes convert V elements a pass, and the conversion unit takes 16
// a clock and SM (10 k clocks a pass of 152064 elements on 8 CTAs).  A
// non-negative fp32's bits, moved to the exponent and fraction fields of a
// double, are exactly its value times 2^-896 (zero and subnormal values
// included): two integer instructions.  Sums stay in that scale, where the
// smallest double still is 2^-178 of a probability of 1.
// Values are taken as bits with -0 made 0, so that a probability is valid
// exactly when they are below infinity's: a pass keeps their maximum.
constexpr double kUnscale = 0x1p896;
constexpr uint32_t kInvalid = 0x7f800000u;
__device__ __forceinline__ uint32_t prob_bits(float x) { return __float_as_uint(x + 0.f); }
__device__ __forceinline__ double scaled(uint32_t u) {
  return __hiloint2double(static_cast<int>(u >> 3), static_cast<int>(u << 29));
}
__device__ __forceinline__ double weight_scaled(uint32_t p, uint32_t q, double a) {
  const double w = fma(-a, scaled(q), scaled(p));
  return __double2hiint(w) < 0 ? 0.0 : w;          // (-0 too)
}

}  // namespace accp

using namespace accp;

__device__ __forceinline__ void cp_async16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

template <bool SAMPLED>        // SPECSAMPLE, else SPECEXEC
__global__ void __launch_bounds__(kThreads) accept_probs_kernel(Params P) {
  extern __shared__ __align__(16) unsigned char dyn[];
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = P.T, V = P.V;
  __shared__ double s_warp[2][kWarps];           // [pass parity]
  __shared__ double s_cta[2][kMaxC];
  __shared__ int s_pick[2];
  double* s_u = reinterpret_cast<double*>(dyn);  // [T] u_child
  int* s_par = reinterpret_cast<int*>(s_u + (SAMPLED ? T : 0));   // [T] parent, -2 when malformed
  int* s_tok = s_par + T;                        // [T] token, -1 when outside [0, V)
  float* s_px = reinterpret_cast<float*>(s_tok + T);              // [T] p, q of the node's token in its parent's rows
  float* s_qx = s_px + (SAMPLED ? T : 0);

  const int n = P.n_nodes ? P.n_nodes[b] : T;
  int32_t* acc = P.acc + static_cast<int64_t>(b) * T;
  int32_t* out = P.out + static_cast<int64_t>(b) * (T + 1);
  if (n <= 0 || n > T) {                         // the whole cluster leaves
    if (rank == 0) {
      for (int i = tid; i < T; i += kThreads) acc[i] = -1;
      for (int i = tid; i < T + 1; i += kThreads) out[i] = -1;
      if (tid == 0) {
        P.n_acc[b] = 0;
        if (n != 0) set_status(P.status, TV_DEV_BAD_LEN);
      }
    }
    return;
  }
  if (C > 1) cl.barrier_arrive();                // peers' shared memory is written to once they all run
  const int32_t* par = P.par + b * P.par_sb;
  const int32_t* tok = P.tok + b * P.tok_sb;
  const float* prow0 = P.p + b * P.tp_sb;
  const float* qrow0 = SAMPLED ? P.q + b * P.dp_sb : nullptr;
  uint32_t bits = 0;
  for (int j = tid; j < n; j += kThreads) {
    int pj = par[j];
    int x = j == 0 ? 0 : tok[j];
    if (j == 0) {
      if (pj != -1) bits |= TV_DEV_BAD_PARENT;
      pj = -2;
    } else if (pj < 0 || pj >= j) {
      bits |= TV_DEV_BAD_PARENT;
      pj = -2;
    }
    if (j > 0 && (x < 0 || x >= V)) {
      bits |= TV_DEV_BAD_TOKEN;
      x = -1;
    }
    s_par[j] = pj;
    s_tok[j] = x;
    if (SAMPLED) {
      const bool ask = pj >= 0 && x >= 0;
      s_px[j] = ask ? __ldg(prow0 + static_cast<int64_t>(pj) * P.tp_st + x) : 0.f;
      s_qx[j] = ask ? __ldg(qrow0 + static_cast<int64_t>(pj) * P.dp_st + x) : 0.f;
      s_u[j] = P.u_child[static_cast<int64_t>(b) * T + j];
    }
  }
  if (rank == 0) set_status(P.status, bits);
  __syncthreads();
  if (C > 1) cl.barrier_wait();

  int pass = 0;
  const int gw = rank * kWarps + warp;
  const int e0 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(gw) * P.chunk));
  const int e1 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(e0) + P.chunk));
  const bool vec = P.vec != 0;
  float* buf_p = reinterpret_cast<float*>(dyn + P.rows_at) + static_cast<size_t>(warp) * P.cap;   // [warp][cap]
  float* buf_q = buf_p + static_cast<size_t>(kWarps) * P.cap;
  int held_p = -1, held_q = -1;                  // rows whose whole chunk is in shared memory
  // elements [es, ee) of a row into this warp's buffer, zeros up to a whole step
  auto copy_in = [&](const float* row, int es, int ee, float* buf) {
    if (vec) {
#pragma unroll 1
      for (int e = es + lane * 4; e + 3 < ee; e += 128) cp_async16(buf + (e - es), row + e);
    }
#pragma unroll 1
    for (int e = (vec ? es + ((ee - es) & ~3) : es) + lane; e < ee; e += 32) cp_async4(buf + (e - es), row + e);
    const int pad = (ee - es + 127) & ~127;
    for (int e = ee - es + lane; e < pad; e += 32) buf[e] = 0.f;
  };
  // f(es, ee) for the pieces [es, ee) of row c's chunk, each in shared memory
  // from element 0 of the buffers on (f true ends the walk)
  auto pieces = [&](int c, bool with_q, auto f) {
    for (int es = e0; es < e1; es += P.cap) {
      const int ee = min(e1, es + P.cap);
      const bool get_p = held_p != c, get_q = with_q && held_q != c;
      __syncwarp();
      if (get_p) copy_in(prow0 + static_cast<int64_t>(c) * P.tp_st, es, ee, buf_p);
      if (get_q) copy_in(qrow0 + static_cast<int64_t>(c) * P.dp_st, es, ee, buf_q);
      if (get_p || get_q) asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      if (f(es, ee)) return;
    }
    const bool whole = e1 - e0 <= P.cap;
    held_p = whole ? c : -1;
    if (with_q) held_q = whole ? c : -1;
  };
  // bits of 4 elements of the buffers
  auto four = [](const float* buf, int o) {
    const float4 x = *reinterpret_cast<const float4*>(buf + o);
    return make_uint4(prob_bits(x.x), prob_bits(x.y), prob_bits(x.z), prob_bits(x.w));
  };
  // sum of the weights of row c's residual a; NaN when the row holds an
  // invalid probability.  The parts stay in s_warp / s_cta [pass & 1].
  auto row_sum = [&](int c, double a) -> double {
    double s0 = 0.0, s1 = 0.0, s2 = 0.0, s3 = 0.0;
    uint32_t top = 0;
    const bool with_q = SAMPLED && a > 0.0;
    pieces(c, with_q, [&](int es, int ee) {
#pragma unroll 2
      for (int o = lane * 4; o < ee - es; o += 128) {
        const uint4 pv = four(buf_p, o), qv = with_q ? four(buf_q, o) : make_uint4(0u, 0u, 0u, 0u);
        top = max(max(max(top, pv.x), max(pv.y, pv.z)), max(max(pv.w, qv.x), max(max(qv.y, qv.z), qv.w)));
        s0 += weight_scaled(pv.x, qv.x, a);
        s1 += weight_scaled(pv.y, qv.y, a);
        s2 += weight_scaled(pv.z, qv.z, a);
        s3 += weight_scaled(pv.w, qv.w, a);
      }
      return false;
    });
    double s = warp_sum(top >= kInvalid ? static_cast<double>(NAN) : ((s0 + s1) + (s2 + s3)) * kUnscale);
    ++pass;
    if (lane == 0) s_warp[pass & 1][warp] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += s_warp[pass & 1][w];
    if (C > 1) {
      if (tid < C) cl.map_shared_rank(&s_cta[pass & 1][0], tid)[rank] = s;
      cl.sync();
      s = 0.0;
      for (int k = 0; k < C; ++k) s += s_cta[pass & 1][k];
    } else if (tid == 0) {
      s_cta[pass & 1][0] = s;
    }
    return s;
  };
  // The inverse-CDF sample over the parts that row_sum(c, a) left: the
  // smallest t with cum_t > target.  Returns it in the warp whose chunk
  // holds it, -1 in the others.
  auto find = [&](int c, double a, double target) -> int {
    // [lo, hi): this warp's stretch of the cumulative sum.  Neighbours
    // compute their common border by the same additions, so exactly one
    // warp holds any target below the sum; at or past it (rounding) the last
    // chunk with weight takes it.
    double base = 0.0, lo = 0.0;
    for (int k = 0; k < rank; ++k) base += s_cta[pass & 1][k];
    for (int w = 0; w < warp; ++w) lo += s_warp[pass & 1][w];
    const double mine = s_warp[pass & 1][warp];
    const double hi = base + (lo + mine);
    double before = base + lo, after = 0.0;
    for (int w = warp + 1; w < kWarps; ++w) after += s_warp[pass & 1][w];
    for (int k = rank + 1; k < C; ++k) after += s_cta[pass & 1][k];
    if (!(mine > 0.0 && target >= before && (target < hi || after == 0.0))) return -1;
    // Lane l takes the l-th run of consecutive elements, so one scan over the
    // lanes finds the run, and the whole warp then goes through that one run.
    const bool with_q = SAMPLED && a > 0.0;
    auto at = [&](int o) -> double {
      return weight_scaled(prob_bits(buf_p[o]), with_q ? prob_bits(buf_q[o]) : 0u, a) * kUnscale;
    };
    int last = -1, hit_at = -1;
    pieces(c, with_q, [&](int es, int ee) {
      const int run = ((ee - es + 31) / 32) | 1;   // odd: the lanes' reads fall in 32 banks
      double mine_sum = 0.0;
      for (int o = lane * run; o < min(ee - es, (lane + 1) * run); ++o) mine_sum += at(o);
      const double incl = warp_incl_scan(mine_sum);
      const unsigned over = __ballot_sync(0xffffffffu, mine_sum > 0.0 && before + incl > target);
      const unsigned some = __ballot_sync(0xffffffffu, mine_sum > 0.0);
      if (some == 0u) return false;
      // the run that holds the target, or (rounding, or it lies in a later piece) the last one with weight
      const int l = over ? __ffs(over) - 1 : 31 - __clz(some);
      double c0 = before + __shfl_sync(0xffffffffu, incl - mine_sum, l);
      for (int o0 = l * run; o0 < min(ee - es, (l + 1) * run); o0 += 32) {
        const int o = o0 + lane;
        const double w = o < min(ee - es, (l + 1) * run) ? at(o) : 0.0;
        const double in = warp_incl_scan(w);
        const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && c0 + in > target);
        const unsigned pos = __ballot_sync(0xffffffffu, w > 0.0);
        if (pos) last = es + o0 + 31 - __clz(pos);
        if (hit) {
          hit_at = es + o0 + __ffs(hit) - 1;
          return true;
        }
        c0 += __shfl_sync(0xffffffffu, in, 31);
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
      return over != 0u;
    });
    return hit_at >= 0 ? hit_at : last;
  };
  // first child of c after node `from` (every warp by itself)
  auto next_child = [&](int c, int from) -> int {
    for (int j0 = from + 1; j0 < n; j0 += 32) {
      const int j = j0 + lane;
      const unsigned m = __ballot_sync(0xffffffffu, j < n && s_par[j] == c);
      if (m) return j0 + __ffs(m) - 1;
    }
    return -1;
  };

  int cur = 0, count = 0;
  bool fault = false;
  while (true) {
    int nxt = -1;
    double a = 0.0, N = 1.0, have = -1.0;        // have: the residual whose parts row_sum left
    if (SAMPLED) {
      for (int j = next_child(cur, cur); j >= 0; j = next_child(cur, j)) {
        if (s_tok[j] < 0) continue;
        const float px = s_px[j], qx = s_qx[j];
        const double u = s_u[j];
        if (!prob_ok(px) || !prob_ok(qx) || !uni_ok(u)) { fault = true; break; }
        if (u * static_cast<double>(qx) * N < weight(px, qx, a)) { nxt = j; break; }
        const double S = row_sum(cur, a + N);
        if (S != S) { fault = true; break; }
        have = a + N;
        if (S > 0.0) {
          a = have;
          N = S;
        }
      }
    }
    if (fault) break;
    if (nxt < 0) {
      const double u = P.u_sample[static_cast<int64_t>(b) * T + cur];
      if (!uni_ok(u)) { fault = true; break; }
      if (have != a) N = row_sum(cur, a);
      if (!(N > 0.0)) { fault = true; break; }   // NaN, or no positive entry
      const int x = find(cur, a, u * N);
      if (SAMPLED) {
        if (x >= 0 && lane == 0) out[count] = x;
        break;
      }
      // every CTA learns the sample
      if (x >= 0 && lane == 0)
        for (int k = 0; k < C; ++k) cl.map_shared_rank(&s_pick[pass & 1], k)[0] = x;
      cl.sync();
      const int t = s_pick[pass & 1];
      for (int j = next_child(cur, cur); j >= 0; j = next_child(cur, j))
        if (s_tok[j] == t) { nxt = j; break; }
      if (nxt < 0) {
        if (rank == 0 && tid == 0) out[count] = t;
        break;
      }
    }
    if (rank == 0 && tid == 0) {
      acc[count] = nxt;
      out[count] = s_tok[nxt];
    }
    ++count;
    cur = nxt;
  }
  if (rank == 0) {
    for (int i = count + tid; i < T; i += kThreads) acc[i] = -1;
    for (int i = count + tid; i < T + 1; i += kThreads)
      if (i > count || fault) out[i] = -1;
    if (tid == 0) {
      P.n_acc[b] = count;
      if (fault) set_status(P.status, TV_DEV_NONFINITE);
    }
  }
  if (C > 1) cl.sync();                          // peers may still read or post sums here
}

int num_sms();

cudaError_t launch_accept_probs(const tv_accept_probs_args* a, bool sampled, cudaStream_t stream) {
  Params p;
  p.B = a->B; p.T = a->T; p.V = a->V;
  p.p = a->target_probs; p.tp_sb = a->tp_sb; p.tp_st = a->tp_st;
  p.q = sampled ? a->draft_probs : nullptr; p.dp_sb = a->dp_sb; p.dp_st = a->dp_st;
  p.tok = a->draft_tokens; p.tok_sb = a->tok_sb;
  p.par = a->parent; p.par_sb = a->parent_sb;
  p.n_nodes = a->n_nodes;
  p.u_child = a->u_child; p.u_sample = a->u_sample;
  p.n_acc = a->n_accepted; p.acc = a->accepted_nodes; p.out = a->out_tokens;
  p.status = a->dev_status;
  auto rows16 = [](const float* x, int64_t sb, int64_t st) {
    return reinterpret_cast<uintptr_t>(x) % 16 == 0 && sb % 4 == 0 && st % 4 == 0;
  };
  p.vec = rows16(p.p, p.tp_sb, p.tp_st) && (!sampled || rows16(p.q, p.dp_sb, p.dp_st));
  // CTAs of a cluster: as many as keep the GPU full, each with at least one
  // step of every warp
  int c = kMaxC;
  while (c > 1 && (static_cast<int64_t>(a->B) * c > 2 * num_sms() || a->V < c * kThreads * 4)) c /= 2;
  const int64_t per = (static_cast<int64_t>(a->V) + c * kWarps - 1) / (c * kWarps);
  p.chunk = static_cast<int>((per + 127) / 128 * 128);
  // the whole chunk in shared memory where it fits (V up to about 200000 at
  // 8 CTAs), else pieces of it
  const size_t nodes = (static_cast<size_t>(a->T) * (sampled ? 24 : 8) + 15) / 16 * 16;
  const size_t per_elt = static_cast<size_t>(kWarps) * (sampled ? 8 : 4);
  const int fit = static_cast<int>((kMaxSmem - nodes) / per_elt) / 128 * 128;
  p.cap = std::min(p.chunk, fit);
  p.rows_at = static_cast<int>(nodes);
  const size_t smem = nodes + static_cast<size_t>(p.cap) * per_elt;
  auto kernel = sampled ? accept_probs_kernel<true> : accept_probs_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a->B) * c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tv
