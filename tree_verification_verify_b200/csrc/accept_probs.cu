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
// cluster, in order; lanes take four elements a step, sums are fp64 (a
// vocabulary of fp32 terms beside a threshold).  Warps' sums meet in shared
// memory, CTAs' sums over distributed shared memory.  A sample finds its CTA
// and warp by the prefix of those sums and scans that warp's chunk again.
// All CTAs of a cluster hold the same state and take the same branches.
#include <cooperative_groups.h>

#include "tv_common.cuh"

namespace cg = cooperative_groups;

namespace tv {

namespace accp {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxC = 8;
constexpr int kMaxT = 4096;

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
  int chunk;                   // elements of a warp's chunk (a multiple of 128)
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
constexpr double kUnscale = 0x1p896;
__device__ __forceinline__ double scaled(float x) {
  const uint32_t u = __float_as_uint(x);
  return __hiloint2double(static_cast<int>((u >> 3) & 0x0fffffffu), static_cast<int>(u << 29));   // (-0 is 0)
}
__device__ __forceinline__ double weight_scaled(float p, float q, double a) {
  const double w = fma(-a, scaled(q), scaled(p));
  return __double2hiint(w) < 0 ? 0.0 : w;          // (-0 too)
}

}  // namespace accp

using namespace accp;

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

  int pass = 0;
  const int gw = rank * kWarps + warp;
  const int e0 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(gw) * P.chunk));
  const int e1 = static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(e0) + P.chunk));
  const bool vec = P.vec != 0;
  // sum of the weights of row c's residual a; NaN when the row holds an
  // invalid probability.  The parts stay in s_warp / s_cta [pass & 1].
  auto row_sum = [&](int c, double a) -> double {
    const float* pr = prow0 + static_cast<int64_t>(c) * P.tp_st;
    const float* qr = SAMPLED && a > 0.0 ? qrow0 + static_cast<int64_t>(c) * P.dp_st : nullptr;
    double s0 = 0.0, s1 = 0.0, s2 = 0.0, s3 = 0.0;
    bool bad = false;
    if (qr) {
#pragma unroll 4
      for (int e = e0 + lane * 4; e < e1; e += 128) {
        const float4 pv = load4(pr, e, e1, vec, 0.f), qv = load4(qr, e, e1, vec, 0.f);
        bad |= !(prob_ok(pv.x) && prob_ok(pv.y) && prob_ok(pv.z) && prob_ok(pv.w));
        bad |= !(prob_ok(qv.x) && prob_ok(qv.y) && prob_ok(qv.z) && prob_ok(qv.w));
        s0 += weight_scaled(pv.x, qv.x, a);
        s1 += weight_scaled(pv.y, qv.y, a);
        s2 += weight_scaled(pv.z, qv.z, a);
        s3 += weight_scaled(pv.w, qv.w, a);
      }
    } else {
#pragma unroll 4
      for (int e = e0 + lane * 4; e < e1; e += 128) {
        const float4 pv = load4(pr, e, e1, vec, 0.f);
        bad |= !(prob_ok(pv.x) && prob_ok(pv.y) && prob_ok(pv.z) && prob_ok(pv.w));
        s0 += scaled(pv.x);
        s1 += scaled(pv.y);
        s2 += scaled(pv.z);
        s3 += scaled(pv.w);
      }
    }
    double s = warp_sum(bad ? static_cast<double>(NAN) : ((s0 + s1) + (s2 + s3)) * kUnscale);
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
    const float* pr = prow0 + static_cast<int64_t>(c) * P.tp_st;
    const float* qr = SAMPLED && a > 0.0 ? qrow0 + static_cast<int64_t>(c) * P.dp_st : nullptr;
    int last = -1;
    for (int es = e0; es < e1; es += 128) {
      const int e = es + lane * 4;
      float4 pv = make_float4(0.f, 0.f, 0.f, 0.f), qv = pv;
      if (e < e1) pv = load4(pr, e, e1, vec, 0.f);
      if (e < e1 && qr) qv = load4(qr, e, e1, vec, 0.f);
      const double w0 = weight(pv.x, qv.x, a), w1 = weight(pv.y, qv.y, a);
      const double w2 = weight(pv.z, qv.z, a), w3 = weight(pv.w, qv.w, a);
      const double incl = warp_incl_scan((w0 + w1) + (w2 + w3));
      const double c0 = before + (incl - ((w0 + w1) + (w2 + w3)));
      int hit = -1;
      if (w3 > 0.0 && c0 + w0 + w1 + w2 + w3 > target) hit = e + 3;
      if (w2 > 0.0 && c0 + w0 + w1 + w2 > target) hit = e + 2;
      if (w1 > 0.0 && c0 + w0 + w1 > target) hit = e + 1;
      if (w0 > 0.0 && c0 + w0 > target) hit = e;
      const unsigned m = __ballot_sync(0xffffffffu, hit >= 0);
      if (m) return __shfl_sync(0xffffffffu, hit, __ffs(m) - 1);
      const int pos = w3 > 0.0 ? e + 3 : (w2 > 0.0 ? e + 2 : (w1 > 0.0 ? e + 1 : (w0 > 0.0 ? e : -1)));
      const unsigned z = __ballot_sync(0xffffffffu, pos >= 0);
      if (z) last = __shfl_sync(0xffffffffu, pos, 31 - __clz(z));
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return last;
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
  const size_t smem = static_cast<size_t>(a->T) * (sampled ? 24 : 8);
  auto kernel = sampled ? accept_probs_kernel<true> : accept_probs_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxT * 24);
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
