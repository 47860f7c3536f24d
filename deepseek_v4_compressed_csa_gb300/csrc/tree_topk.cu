// Selections by blocks of 256 threads (csa_attend_tree): the topk largest scores of every node's visible columns, ties to
// the lower column, in ascending order.
//
// The register kernel of indexer.cu gives a query 1024 threads: the lowest latency for a few queries, but one block
// per SM, its barriers and histogram rounds exposed.  With more nodes than SMs a block of 256 threads holding its keys
// in shared memory lets four or five nodes share an SM and cover each other's waits: 512 nodes of 8.2K columns take
// 17 us instead of 38.  With few nodes it leaves room on its SM for the attention's CTA (topk_tree_small_blocks).  Radix select over digits of 11, 11 and 10 bits, then one ascending pass.  Bound by its
// instructions, some seventy for every 32 columns (the ascending pass alone took 35 with a rank per column, and 22 us).
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

__global__ void __launch_bounds__(kThreads) k_tree_topk(const float* __restrict__ scores, int cap, int T,
                                                             const int32_t* __restrict__ parent,
                                                             const int32_t* __restrict__ pos,
                                                             const int32_t* __restrict__ n_rows, int ratio, int topk,
                                                             int32_t* __restrict__ sel, TreeNode* __restrict__ nodes,
                                                             int32_t* err) {
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
  pdl_trigger();  // (indexer.cu, TopkTree)
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
  // ---- ascending pass.  A lane collects the verdicts on 32 consecutive columns as two bit masks, by ballots of its warp;
  // then one scan over the masks' counts gives every lane its place, and it writes the columns of its bits.
  const int words = (ncol + 31) >> 5;
  int gt_before = 0, eq_before = 0;  // of the words of earlier rounds
  for (int w0 = 0; w0 < words; w0 += kThreads) {
    uint32_t m_gt = 0, m_eq = 0;
    const int first = w0 + 32 * wid, here = min(32, words - first);  // this warp's words
#pragma unroll 4
    for (int i = 0; i < here; ++i) {
      const int c = (first + i) * 32 + lane;
      const uint32_t k = c < ncol ? keys[c] : 0u, d = k & mask;
      const uint32_t g = __ballot_sync(0xffffffffu, d > prefix), e = __ballot_sync(0xffffffffu, k != 0 && d == prefix);
      if (lane == i) {
        m_gt = g;
        m_eq = e;
      }
    }
    const int n_gt = __popc(m_gt), n_eq = __popc(m_eq);
    const int i_gt = warp_incl(n_gt), i_eq = warp_incl(n_eq);
    __syncthreads();  // (the previous round's totals have been read)
    if (lane == 31) {
      w_gt[wid] = i_gt;
      w_eq[wid] = i_eq;
    }
    __syncthreads();
    int gt = gt_before + i_gt - n_gt, eq = eq_before + i_eq - n_eq;
    for (int w = 0; w < kWarps; ++w) {
      if (w < wid) {
        gt += w_gt[w];
        eq += w_eq[w];
      }
      gt_before += w_gt[w];
      eq_before += w_eq[w];
    }
    int left = max(0, min(n_eq, need - eq));  // of the equal ones, the lowest columns
    uint32_t take = m_gt;
    for (uint32_t r = m_eq; left > 0; --left, r &= r - 1) take |= r & (~r + 1);
    const int c0 = (first + lane) * 32;
    for (int o = gt + min(eq, need); take != 0 && o < topk; ++o, take &= take - 1) out[o] = c0 + __ffs(take) - 1;
  }
}

}  // namespace

// More nodes than SMs: up to 64 KB of keys, at least three blocks an SM.  Few nodes, whose attention takes several CTAs
// each: up to 33 KB, since a block of 1024 threads fills its SM's registers and keeps the attention's CTA, which fetches
// queries and window rows ahead, away from it (8 nodes of 2K columns: selection and attention 20.8 us, with the register
// kernel 23.8; of 8K 23.5 and 24.4; of 15K 26.8 and 26.2).  In between the register kernel (64 nodes of 8K columns: 35
// us, here 41).
bool topk_tree_small_blocks(int Q, int cap, int T, int sms) {
  const size_t bytes = (size_t)(cap + T) * sizeof(uint32_t);
  return (Q > sms && bytes <= 64 * 1024) || (4 * Q <= sms && bytes <= 33 * 1024);
}

cudaError_t launch_topk_tree_small(const Dims& L, const float* scores, int B, int T, const int32_t* parent, int cap,
                                  const int32_t* n_rows, const int32_t* pos, int32_t* sel, TreeNode* nodes,
                                  int32_t* err, cudaStream_t s) {
  const size_t smem = (size_t)(cap + T) * sizeof(uint32_t);
  allow_smem<64 * 1024>(k_tree_topk);
  CSA_LAUNCH(k_tree_topk, dim3(B * T), dim3(kThreads), smem, s, scores, cap, T, parent, pos, n_rows, L.ratio,
             L.topk, sel, nodes, err);
  return cudaGetLastError();
}

}  // namespace csa
