// Device helpers for a tree of drafted tokens.
//
// A tree of at most 64 nodes per sequence is its parent array: parent[i] in [0, i) for a child, -1 for a child of
// the last committed token, below -1 for an unused slot.  Because a parent always has the lower index, the set of
// a node's ancestors and itself, as a 64-bit mask, lists the node's path in order: the bit of rank k is the
// path's node at depth k.  Every kernel derives the masks it needs from the parent array itself (a walk of
// depth(i) steps in registers or shared memory, hidden behind its first loads), so no plan has to be built, kept
// or invalidated when a tree changes from step to step.
#pragma once
#include "common.cuh"

namespace csa {

constexpr int kTreeMax = 64;
constexpr int kTreeNone = -2;

// A committed length that every node's position, and the one behind it, fit on in 32 bits.
__device__ __forceinline__ bool tree_pos_ok(int p0) { return p0 >= 0 && p0 <= INT32_MAX - kTreeMax; }

// Parent of node i as the walks use it: kTreeNone for an unused slot or (bad set) a parent that is not below i.
__device__ __forceinline__ int tree_parent(const int32_t* __restrict__ parent, int T, int i, bool& bad) {
  if (i >= T) return kTreeNone;
  const int p = __ldg(parent + i);
  if (p >= i) {
    bad = true;
    return kTreeNone;
  }
  return p < -1 ? kTreeNone : p;
}

// One warp, every lane: the path mask of node i of a tree (0: unused slot, or a path through one, which sets bad).
// The parent row is held in two registers a lane; the walk is two shuffles a step.
__device__ __forceinline__ uint64_t tree_path_warp(const int32_t* __restrict__ parent, int T, int i, bool& bad) {
  const int lane = threadIdx.x & 31;
  bool ignore = false;
  const int lo = tree_parent(parent, T, lane, ignore), hi = tree_parent(parent, T, lane + 32, ignore);
  uint64_t mask = 0;
  int a = i;
  bool first = true;
  while (a >= 0) {
    const int pl = __shfl_sync(0xffffffffu, lo, a & 31), ph = __shfl_sync(0xffffffffu, hi, a & 31);
    const int up = a < 32 ? pl : ph;
    mask |= 1ull << a;
    if (up == kTreeNone) {
      // node i is an unused slot (no error unless its parent is out of range), or an ancestor of it is
      if (!first || (i < T && __ldg(parent + i) >= i)) bad = true;
      return 0;
    }
    first = false;
    a = up;
  }
  return mask;
}

// Whole block (at least 64 threads): every node's path mask into shared memory; returns whether the array is
// consistent (the same answer in every thread).  par: 64 ints of shared memory.
__device__ __forceinline__ bool tree_masks_block(const int32_t* __restrict__ parent, int T, uint64_t* masks, int* par) {
  const int i = threadIdx.x;
  bool bad = false;
  if (i < kTreeMax) par[i] = tree_parent(parent, T, i, bad);
  __syncthreads();
  if (i < kTreeMax) {
    uint64_t m = 0;
    int a = i;
    while (a >= 0) {
      m |= 1ull << a;
      const int up = par[a];
      if (up == kTreeNone) {
        if (a != i) bad = true;
        m = 0;
        break;
      }
      a = up;
    }
    masks[i] = m;
  }
  return __syncthreads_or(bad) == 0;
}

// The path's node at depth k (k < popcount of the mask).
__device__ __forceinline__ int tree_node_at(uint64_t mask, int k) {
  for (int s = 0; s < k; ++s) mask &= mask - 1;
  return __ffsll((long long)mask) - 1;
}

// The nodes of a path that complete a window, when the path starts at position p0.
__device__ __forceinline__ uint64_t tree_closers(uint64_t mask, int p0, int ratio) {
  uint64_t c = 0;
  int left = ratio - 1 - p0 % ratio;  // steps to the next node that completes one
  while (mask) {
    const uint64_t bit = mask & (~mask + 1);
    if (left == 0) {
      c |= bit;
      left = ratio;
    }
    --left;
    mask ^= bit;
  }
  return c;
}

// ---------------------------------------------------------------- a node's view of its sequence
struct NodeView {
  uint64_t mask, closers;  // the path; its nodes that complete a window
  int b, i, p0, p, n;      // sequence, node, committed length, the node's position, committed rows
};
// One warp, every lane; false: an unused slot, or a state error (reported by lane 0).
__device__ __forceinline__ bool node_view(NodeView& v, const int32_t* parent, int T_, const int32_t* pos,
                                          const int32_t* n_rows, int cap, int ratio, int q, int32_t* err) {
  v.b = q / T_;
  v.i = q - v.b * T_;
  v.p0 = pos[v.b];
  v.n = n_rows[v.b];
  bool bad = false;
  v.mask = tree_path_warp(parent + (size_t)v.b * T_, T_, v.i, bad);
  const bool state = !tree_pos_ok(v.p0) || v.n != v.p0 / ratio || v.n > cap;
  if ((bad || (state && v.mask)) && (threadIdx.x & 31) == 0) atomicOr(err, CSA_DEV_STATE);
  if (state || v.mask == 0) return false;
  v.p = v.p0 + __popcll(v.mask) - 1;
  v.closers = tree_closers(v.mask, v.p0, ratio);
  return true;
}

}  // namespace csa
