// Selections of many nodes at once (csa_attend_tree): the topk largest scores of every node's visible columns, ties to
// the lower column, in ascending order.
//
// The register kernel of indexer.cu gives a query 1024 threads: the lowest latency for a few queries, but one block
// per SM, its barriers and histogram rounds exposed.  With more nodes than SMs a block of 256 threads holding its keys
// in shared memory lets four or five nodes share an SM and cover each other's waits: 512 nodes of 8.2K columns take
// 22 us instead of 38.  Radix select over digits of 11, 11 and 10 bits, then one ascending pass.
#include "kernels.h"
#include "tree.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBins = 2048;

__device__ __forceinline__ int warp_incl(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

__global__ void __launch_bounds__(kThreads) k_tree_topk_many(const float* __restrict__ scores, int cap, int T,
                                                             const int32_t* __restrict__ parent,
                                                             const int32_t* __restrict__ pos,
                                                             const int32_t* __restrict__ n_rows, int ratio, int topk,
                                                             int32_t* __restrict__ sel, TreeNode* __restrict__ nodes,
                                                             int32_t* err) {
  pdl_trigger();
  extern __shared__ uint32_t keys[];  // [cap + T]
  __shared__ int hist[kBins];
  __shared__ int wtot[kWarps], w_gt[kWarps], w_eq[kWarps];
  __shared__ NodeView sv;
  __shared__ int s_ok, s_bin, s_need, s_count;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, q = blockIdx.x;
  // the committed columns are known from the position alone: their scores are requested first
  const int n = max(0, min(cap, pos[q / T] / ratio));
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  pdl_wait();
  const float* sc = scores + (size_t)q * (cap + T);
  constexpr int kU = 8;
  float f[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) f[u] = tid + u * kThreads < n ? __ldg(sc + tid + u * kThreads) : 0.f;
  if (wid == 0) {
    NodeView v;
    const bool ok = node_view(v, parent, T, pos, n_rows, cap, ratio, q, err);
    if (lane == 0) {
      sv = v;
      s_ok = ok;
      TreeNode r{};
      r.nsel = -1;
      if (ok) {
        r.mask = v.mask; r.closers = v.closers; r.p = v.p; r.p0 = v.p0; r.n = v.n;
        r.nsel = min(topk, v.n + __popcll(v.closers));
      }
      nodes[q] = r;
    }
  }
  __syncthreads();
  if (!s_ok) return;
  int32_t* out = sel + (size_t)q * topk;
  const int nvis = n + __popcll(sv.closers);
  if (nvis <= topk) {
    for (int k = tid; k < topk; k += kThreads) out[k] = k < n ? k : (k < nvis ? n + tree_node_at(sv.closers, k - n) : -1);
    return;
  }
  // ---- keys into shared memory, the first digit's counts with them.  A key is at least 1; a column that the node does
  // not see has key 0 and is in no count.
  for (int c0 = 0; c0 < n; c0 += kU * kThreads) {
    float g[kU];
    const int c1 = c0 + kU * kThreads;
#pragma unroll
    for (int u = 0; u < kU; ++u) g[u] = c1 + tid + u * kThreads < n ? __ldg(sc + c1 + tid + u * kThreads) : 0.f;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = c0 + tid + u * kThreads;
      if (c < n) {
        const uint32_t k = max(ord_key(f[u]), 1u);
        keys[c] = k;
        atomicAdd(&hist[k >> 21], 1);
      }
      f[u] = g[u];
    }
  }
  if (tid < T) {
    const bool seen = (sv.closers >> tid) & 1;
    const uint32_t k = seen ? max(ord_key(__ldg(sc + n + tid)), 1u) : 0u;
    keys[n + tid] = k;
    if (seen) atomicAdd(&hist[k >> 21], 1);
  }
  const int ncol = n + T;
  uint32_t prefix = 0, mask = 0;
  int need = topk;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t dmask = pass == 2 ? 1023u : 2047u;
    if (pass > 0) {
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int c = tid; c < ncol; c += kThreads) {
        const uint32_t k = keys[c];
        if (k && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & dmask], 1);
      }
    }
    __syncthreads();
    // bins in descending order, eight a thread: the one where the count reaches `need`
    int b[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      b[i] = hist[kBins - 1 - (8 * tid + i)];
      sum += b[i];
    }
    const int incl_w = warp_incl(sum);
    if (lane == 31) wtot[wid] = incl_w;
    __syncthreads();
    int before = incl_w - sum;
    for (int w = 0; w < wid; ++w) before += wtot[w];
    if (before < need && need <= before + sum) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < need && need <= before + b[i]) {
          s_bin = kBins - 1 - (8 * tid + i);
          s_need = need - before;
          s_count = b[i];
        }
        before += b[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    need = s_need;
    mask |= dmask << shift;
    // the bin holds exactly the keys still needed: the later digits decide nothing (the same answer everywhere)
    if (s_count == need) break;
    __syncthreads();  // (s_bin is rewritten only after everyone has read it)
  }
  // ---- ascending pass: warp w takes a contiguous share; counts of the keys above and equal first
  const int per = (((ncol + kWarps - 1) / kWarps) + 31) & ~31;
  const int lo = wid * per, hi = min(ncol, lo + per);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int c0 = lo; c0 < hi; c0 += 32) {
    const uint32_t k = c0 + lane < hi ? keys[c0 + lane] : 0u;
    gt += (k & mask) > prefix;
    eq += k != 0 && (k & mask) == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    w_gt[wid] = gt;
    w_eq[wid] = eq;
  }
  __syncthreads();
  int eq_rank = 0, slot = 0;
  for (int w = 0; w < wid; ++w) {
    slot += w_gt[w];
    eq_rank += w_eq[w];
  }
  slot += min(eq_rank, need);
  const unsigned lt = (1u << lane) - 1u;
#pragma unroll 2
  for (int c0 = lo; c0 < hi; c0 += 32) {
    const uint32_t k = c0 + lane < hi ? keys[c0 + lane] : 0u;
    const bool is_eq = k != 0 && (k & mask) == prefix;
    const unsigned eqb = __ballot_sync(0xffffffffu, is_eq);
    const bool take = (k & mask) > prefix || (is_eq && eq_rank + __popc(eqb & lt) < need);
    const unsigned tb = __ballot_sync(0xffffffffu, take);
    if (take) {
      const int o = slot + __popc(tb & lt);
      if (o < topk) out[o] = c0 + lane;
    }
    slot += __popc(tb);
    eq_rank += __popc(eqb);
  }
}

}  // namespace

bool topk_tree_many_fits(int Q, int cap, int T, int sms) {
  return Q > sms && (size_t)(cap + T) * sizeof(uint32_t) <= 64 * 1024;  // at least three blocks an SM
}

cudaError_t launch_topk_tree_many(const Dims& L, const float* scores, int B, int T, const int32_t* parent, int cap,
                                  const int32_t* n_rows, const int32_t* pos, int32_t* sel, TreeNode* nodes,
                                  int32_t* err, cudaStream_t s) {
  const size_t smem = (size_t)(cap + T) * sizeof(uint32_t);
  cudaFuncSetAttribute(k_tree_topk_many, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
  CSA_LAUNCH(k_tree_topk_many, dim3(B * T), dim3(kThreads), smem, s, scores, cap, T, parent, pos, n_rows, L.ratio,
             L.topk, sel, nodes, err);
  return cudaGetLastError();
}

}  // namespace csa
