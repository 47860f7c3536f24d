// Attention of a tree's nodes on the 5th-generation tensor cores (bf16, 64 query heads over one 512-dim latent, K = V,
// RoPE on the last 64 dims): a persistent CTA per SM walks its share of the nodes, each over its own keys - selected
// (or all) committed rows, rows that its path completes, window tokens, its path's tokens - in tiles of 128.
//
// Definition: include/csa.h, csa_attend_tree; the records in `nodes` come from the selection (indexer.cu) or from
// k_tree_nodes (tree.cu).
//
// Per tile of 128 keys the tensor pipe needs 32 products of 128 x 64 x 16 for S^T = K Q^T and, with the probabilities
// as two bf16 parts (P_hi = bf16(P), P_lo = bf16(P - P_hi): the product keeps ~16 bits of P, so that the output's error
// is its one rounding), 24 of 128 x 128 x 16 and 16 of 128 x 64 x 16 for O^T += V^T [P_hi | P_lo]^T.  At N = 64 and 128
// a product takes 48 and 64 clocks (it waits for shared memory below N = 128): 1536 + 2304 clocks a tile.  Shared memory
// holds one tile (128 KB), the query block (64 KB) and P (32 KB), tensor memory the two halves of O^T and S^T, so S^T
// of the next tile cannot be formed while a tile's softmax runs; the design keeps that gap and everything else short:
//   loaders (warps 9-15)  fill a tile in four pairs of 64-dim boxes: a pair of the next tile is refilled as soon as the
//     PV products of the current tile have read it.  Consecutive committed rows (no selection) are TMA boxes; of 128
//     selected committed rows four warps fetch 56 by tile::gather4, 28 requests each (a warp issues one every ~75 clocks
//     whatever its threads do, and the copy engine takes ~14 clocks for one), three warps the others by cp.async, which
//     the products' own use of shared memory slows to ~28 B a clock: all rows by seven gathering warps take 117.5 us
//     where this takes 115.3, 56 to 96 gathered rows much the same;
//     tiles of mixed sources (window, path, the selection's end) are cp.async by address.
//   MMA (warp 8)  one thread; descriptors are a base plus a constant: built from addresses every time they cost it
//     ~90 clocks a product, twice what the tensor pipe takes.
//   softmax (warps 0-7)  thread = (key row, 32 heads).  The reference that exponents are taken against is the head's
//     sink: it is in the denominator anyway, needs no maximum over the tile, and any logit within 2^64 of it is exact
//     in fp32's range.  A tile with a larger logit raises the reference to its column maximum (and rescales O^T and the
//     sums); a logit far below the sink gives zero, as it should.  Sums stay per thread until the node's last tile.
//   epilogue (warps 0-7)  O^T / Z, rotated back, rounded once, through the P buffer (free then) to TMA stores: a thread
//     holds one dim of 32 heads, and its 2-byte stores straight to memory cost 7 us a node.  Transposing by stmatrix or by
//     shuffles instead changes nothing (within 1 us for the 512 nodes below), plain 16-byte stores out of the buffer cost
//     3 us: the next node's first tile, whose rows take 3.5K clocks to land, hides all but 2.4K of its 7.5K clocks.
// 512 nodes of 640 keys, 512 of them selected: 98 us beside 17 for the selection; 128 nodes of 1.9K consecutive keys
// each: 64 us, 5.7K clocks a tile of the 3.8K that its products take.
//
// Few nodes with long lists (kSplit): a cluster of S CTAs per node, each its run of the tiles, the parts of O^T joined
// through distributed shared memory.  S is the largest of 8, 4, 2 whose clusters all run at once and that leaves two
// tiles to each CTA (one tile each gains nothing over the join): 8 nodes over 8.2K rows take 48 us instead of 196, 64
// over 2K 44 instead of 59.  The same for the nodes left over after whole rounds of the SMs saves 2 us at 512
// nodes, which its bookkeeping costs again: those stay a CTA each.
#include <atomic>

#include "kernels.h"
#include "tc.cuh"
#include "tree.cuh"

namespace csa {

namespace {

constexpr int kPR = 128;                 // keys per tile
constexpr int kAD = 512;                 // latent dims
constexpr int kAH = 64;                  // heads
constexpr int kBox = kPR * 128;          // 64 dims x 128 rows (16 KB)
constexpr int kQBox = kAH * 128;         // 64 dims x 64 heads (8 KB)
constexpr int kPPart = kPR * 128;        // P^T part: 128 keys x 64 heads, MN-major (16 KB)
constexpr int kSoft = 256;               // warps 0-7
constexpr int kHalf = kSoft / 2;         // threads of one head half
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp0 = 9, kLoadWarps = 7;  // sixteen warps in all, 128 registers a thread
constexpr int kThreads = 32 * (kLoadWarp0 + kLoadWarps);
constexpr int kGatherWarps = 4, kGatherRows = 56;  // of a selected tile: the copy engine's share, the others by cp.async
constexpr int kGatherLanes = kGatherRows / 2 / kGatherWarps;                          // requests of a warp for a pair
constexpr int kCopyInstr = (kPR - kGatherRows) / 2 / (kLoadWarps - kGatherWarps);     // row pairs of a copying warp
static_assert(kGatherLanes * kGatherWarps * 2 == kGatherRows && kCopyInstr <= 16, "whole shares");
constexpr int kTmemCols = 512;
constexpr uint32_t kColO3 = 384;         // O^T tile 3 (hi + lo in one accumulator); tiles 0-2: 128 m, hi | lo
constexpr uint32_t kColS = 448;          // S^T
constexpr float kRaiseAt = 64.f;         // log2 headroom over the reference
constexpr int kMaxSplit = 8;
constexpr int kBarAll = 3;               // named barriers: 1, 2 the halves, 3 all softmax warps

constexpr int kOffQ = 8 * kBox;
constexpr int kOffP = kOffQ + 8 * kQBox;
constexpr int kOffRed = kOffP + 2 * kPPart;   // [4 lane quarters][64 heads]
constexpr int kOffRef = kOffRed + 4 * 64 * 4; // [64] negated reference per head (log2 units)
constexpr int kOffInv = kOffRef + 64 * 4;     // [64] 1 / Z
constexpr int kOffBars = kOffInv + 64 * 4;
constexpr int kNumBars = 15;
constexpr int kOffTmem = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffTmem + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory per block");

struct TaArgs {
  const __nv_bfloat16* pool;   // [B, cap, 512]
  const __nv_bfloat16* ring;   // [B, Wr, 512]
  const __nv_bfloat16* kv;     // [B, T, 512] the nodes' latent rows
  const __nv_bfloat16* rows;   // [B, T, 512] the rows that they complete
  const int32_t* sel;          // [Q, topk] columns, or null: every visible one
  const TreeNode* nodes;       // [Q]
  const float* sink;
  const float* inv_freq;
  __nv_bfloat16* out;          // [Q, 64, 512]
  int Q, T, cap, topk, W, Wr;
  int S;                       // kSplit: CTAs of the cluster that shares a query
  float scale2;                // softmax scale * log2(e)
  int32_t* err;
};

__device__ __forceinline__ int node_keys(const TaArgs& a, const TreeNode& r) {
  return r.nsel < 0 ? 0 : r.nsel + min(a.W, r.p + 1);
}

// Address of key k (< node_keys) of query q; col: its column where a selection says (k < r.nsel, a.sel).
__device__ __forceinline__ const __nv_bfloat16* key_row(const TaArgs& a, const TreeNode& r, int q, int k, int col) {
  const size_t b = q / a.T;
  if (k < r.nsel) {
    const int c = a.sel ? col : (k < r.n ? k : r.n + tree_node_at(r.closers, k - r.n));
    return c < r.n ? a.pool + (b * a.cap + c) * kAD : a.rows + (b * a.T + (c - r.n)) * kAD;
  }
  const int t = r.p - min(a.W, r.p + 1) + 1 + (k - r.nsel);
  return t < r.p0 ? a.ring + (b * a.Wr + t % a.Wr) * kAD : a.kv + (b * a.T + tree_node_at(r.mask, t - r.p0)) * kAD;
}

// The keys [k0, k1) among a query's that this CTA takes: all, or (kSplit) its run of the tiles.
template <bool kSplit>
__device__ __forceinline__ void key_range(const TaArgs& a, int keys, int& k0, int& k1) {
  k0 = 0;
  k1 = keys;
  if constexpr (kSplit) {
    const int tiles = (keys + kPR - 1) / kPR, rank = blockIdx.x % a.S;
    k0 = min(keys, (int)((long long)tiles * rank / a.S) * kPR);
    k1 = min(keys, (int)((long long)tiles * (rank + 1) / a.S) * kPR);
  }
}

// 2^x by the hardware approximation (relative error ~2^-22; results below 2^-126 flush to zero)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(tc::smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Reduce 32 columns over the 32 lanes of a warp; lane L returns column L.
template <bool kMax>
__device__ __forceinline__ float reduce_scatter32(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int st = 0; st < 5; ++st) {
    const int half = 16 >> st;
    const bool upper = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = upper ? v[i] : v[i + half];
      const float keep = upper ? v[i + half] : v[i];
      const float recv = __shfl_xor_sync(0xffffffffu, send, half);
      v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  return v[0];
}

// The softmax warps: the joined output of query qi.  CTA r of the cluster takes dims [512 r / S, 512 (r + 1) / S) of
// every head, four a thread, from the S parts in rank order.  Parts are relative to references of their own: the largest
// one is the common one.  (A part without keys has a sum of zero and no O^T.)  table: S x 64 floats.
__device__ __forceinline__ void join_parts(const TaArgs& a, const uint8_t* rows, const float* nref, const float* sums,
                                           float* table, int qi) {
  const int tid = threadIdx.x, per = kAD / a.S / 4, d = kAD / a.S * (blockIdx.x % a.S) + 4 * (tid % per);
  if (tid < kAH) {  // each part's factor of head tid
    float ref[kMaxSplit], sum[kMaxSplit], top = -INFINITY;
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s) {
      if (s >= a.S) break;
      ref[s] = -tc::ld_cluster_f32(tc::cluster_map(nref + tid, s));
      sum[s] = tc::ld_cluster_f32(tc::cluster_map(sums + tid, s));
      top = fmaxf(top, ref[s]);
    }
    float Z = exp2f(__ldg(a.sink + tid) * 1.4426950408889634f - top);
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s) {
      if (s >= a.S) break;
      ref[s] = sum[s] == 0.f ? 0.f : exp2f(ref[s] - top);
      Z = fmaf(ref[s], sum[s], Z);
    }
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s) {
      if (s >= a.S) break;
      table[s * kAH + tid] = ref[s] / Z;
    }
  }
  float c0 = 1.f, s0 = 0.f, c1 = 1.f, s1 = 0.f;
  const bool turned = d >= kAD - 64;
  if (turned) {
    const int p = a.nodes[qi].p, i = (d - (kAD - 64)) >> 1;
    rope_cs(p, a.inv_freq, i, &c0, &s0);
    rope_cs(p, a.inv_freq, i + 1, &c1, &s1);
  }
  tc::named_bar(kBarAll, kSoft);
  const float* part = reinterpret_cast<const float*>(rows) + d;
  constexpr int kU = 8;  // heads in flight a thread
  const int step = kSoft / per;
  for (int h0 = tid / per; h0 < kAH; h0 += kU * step) {
    float4 o[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < a.S; ++s) {
      float4 v[kU];
      float f[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        const int h = h0 + k * step;
        f[k] = h < kAH ? table[s * kAH + h] : 0.f;
        if (f[k] != 0.f) v[k] = tc::ld_cluster_f4(tc::cluster_map(part + h * kAD, s));
      }
#pragma unroll
      for (int k = 0; k < kU; ++k)
        if (f[k] != 0.f)
          o[k] = make_float4(fmaf(f[k], v[k].x, o[k].x), fmaf(f[k], v[k].y, o[k].y), fmaf(f[k], v[k].z, o[k].z),
                             fmaf(f[k], v[k].w, o[k].w));
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int h = h0 + k * step;
      if (h >= kAH) break;
      float4 y = o[k];
      if (turned)
        y = make_float4(fmaf(y.x, c0, y.y * s0), fmaf(-y.x, s0, y.y * c0), fmaf(y.z, c1, y.w * s1),
                        fmaf(-y.z, s1, y.w * c1));
      uint2 pk;
      __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&pk);
      b[0] = __floats2bfloat162_rn(y.x, y.y);
      b[1] = __floats2bfloat162_rn(y.z, y.w);
      *reinterpret_cast<uint2*>(a.out + ((size_t)qi * kAH + h) * kAD + d) = pk;
    }
  }
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    k_tc_tree_attend(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_out,
                     const __grid_constant__ CUtensorMap tm_pool, const __grid_constant__ CUtensorMap tm_row,
                     const __grid_constant__ TaArgs a) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* rows = smem;
  uint8_t* qbuf = smem + kOffQ;
  uint8_t* pbuf = smem + kOffP;
  float* red = reinterpret_cast<float*>(smem + kOffRed);
  float* nref = reinterpret_cast<float*>(smem + kOffRef);
  float* invz = reinterpret_cast<float*>(smem + kOffInv);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* q_full = bars + 0;     // query block landed (TMA)
  uint64_t* q_empty = bars + 1;    // the query's last score product retired
  uint64_t* rows_full = bars + 2;  // [4] box pair m of the tile landed (one arrival per loader warp)
  uint64_t* box_free = bars + 6;   // [4] PV of dims 128 m .. retired: pair m may take the next tile
  uint64_t* s_full = bars + 10;    // S^T of the tile in tensor memory
  uint64_t* p_full = bars + 11;    // P written, S^T read
  uint64_t* pv_done = bars + 12;   // PV of the tile retired
  uint64_t* o_free = bars + 13;    // the query's output read out of tensor memory
  uint64_t* drain = bars + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmem);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tc::mbar_init(q_full, 1);
    tc::mbar_init(q_empty, 1);
    for (int m = 0; m < 4; ++m) {
      tc::mbar_init(rows_full + m, kLoadWarps);
      tc::mbar_init(box_free + m, 1);
    }
    tc::mbar_init(s_full, 1);
    tc::mbar_init(p_full, kSoft / 32);
    tc::mbar_init(pv_done, 1);
    tc::mbar_init(o_free, kSoft / 32);
    tc::mbar_init(drain, 1);
    tc::fence_mbar_init();
    tc::tma_prefetch(&tm_q);
    tc::tma_prefetch(&tm_out);
    tc::tma_prefetch(&tm_pool);
    tc::tma_prefetch(&tm_row);
  }
  pdl_wait();
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool failed = false;
  int joins = -1;  // kSplit, softmax warps: the query whose parts the cluster joins
  const int q_first = kSplit ? blockIdx.x / a.S : blockIdx.x, q_step = kSplit ? gridDim.x / a.S : gridDim.x;

  if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (tc::elect_one()) {
      constexpr uint32_t id_qk = tc::idesc_bf16(128, 64);
      constexpr uint32_t id_pv2 = tc::idesc_bf16(128, 128, true, true);
      constexpr uint32_t id_pv1 = tc::idesc_bf16(128, 64, true, true);
      const uint64_t kd = tc::sdesc_kmajor_sw128(tc::smem_u32(rows)), qd = tc::sdesc_kmajor_sw128(tc::smem_u32(qbuf));
      const uint64_t vd = tc::sdesc_mnmajor_sw128(tc::smem_u32(rows), kBox, 1024);
      const uint64_t pd = tc::sdesc_mnmajor_sw128(tc::smem_u32(pbuf), kPPart, 1024);
      uint32_t nq = 0, nt = 0;
      for (int qi = q_first; qi < a.Q && !failed; qi += q_step) {
        int first, keys;
        key_range<kSplit>(a, node_keys(a, a.nodes[qi]), first, keys);
        if (first == keys) continue;
        if (!tc::mbar_wait(q_full, nq & 1)) { failed = true; break; }
        for (int k0 = first; k0 < keys; k0 += kPR, ++nt) {
          const uint32_t par = nt & 1;
          // S^T = K Q^T, pair by pair as the rows land
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (failed || !tc::mbar_wait(rows_full + m, par)) { failed = true; break; }
            tc::fence_after_sync();
#pragma unroll
            for (int k = 8 * m; k < 8 * m + 8; ++k)
              tc::mma_bf16(tmem + kColS, kd + (((k >> 2) * kBox + (k & 3) * 32) >> 4),
                           qd + (((k >> 2) * kQBox + (k & 3) * 32) >> 4), id_qk, k > 0);
          }
          if (failed) break;
          tc::mma_commit(s_full);
          const bool last = k0 + kPR >= keys;
          if (last) tc::mma_commit(q_empty);
          if (!tc::mbar_wait(p_full, par)) { failed = true; break; }
          if (k0 == first && nq > 0 && !tc::mbar_wait(o_free, (nq - 1) & 1)) { failed = true; break; }
          tc::fence_after_sync();
          // O^T += V^T P^T: dims 128 m .., tiles 0-2 with both parts side by side, tile 3 with the parts in turn.  The
          // last tile's products stop at its last 16 keys.
          const uint32_t acc = k0 > first;
          if (!last || keys - k0 > kPR - 16) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint64_t ad = vd + ((2 * m * kBox + kk * 2048) >> 4), bd = pd + ((kk * 2048) >> 4);
                if (m < 3) {
                  tc::mma_bf16(tmem + 128 * m, ad, bd, id_pv2, kk > 0 ? 1u : acc);
                } else {
                  tc::mma_bf16(tmem + kColO3, ad, bd, id_pv1, kk > 0 ? 1u : acc);
                  tc::mma_bf16(tmem + kColO3, ad, bd + (kPPart >> 4), id_pv1, 1u);
                }
              }
              tc::mma_commit(box_free + m);
            }
          } else {
            const int steps = (keys - k0 + 15) >> 4;
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
#pragma unroll 1
              for (int kk = 0; kk < steps; ++kk) {
                const uint64_t ad = vd + ((2 * m * kBox + kk * 2048) >> 4), bd = pd + ((kk * 2048) >> 4);
                if (m < 3) {
                  tc::mma_bf16(tmem + 128 * m, ad, bd, id_pv2, kk > 0 ? 1u : acc);
                } else {
                  tc::mma_bf16(tmem + kColO3, ad, bd, id_pv1, kk > 0 ? 1u : acc);
                  tc::mma_bf16(tmem + kColO3, ad, bd + (kPPart >> 4), id_pv1, 1u);
                }
              }
              tc::mma_commit(box_free + m);
            }
          }
          tc::mma_commit(pv_done);
        }
        ++nq;
      }
      // retire every MMA before tensor memory is released
      tc::mma_commit(drain);
      if (!tc::mbar_wait(drain, 0)) failed = true;
    }
  } else if (warp >= kLoadWarp0) {
    // ------------------------------------------------------------ loaders
    // By address: warp w's instruction k of a pair copies 256 bytes of rows 2 i and 2 i + 1, i = w + 7 k (i < 64), a
    // half warp each; lane l holds the address of row 2 (w + 7 (l % 16)) + l / 16, so that one shuffle hands a half its
    // row.  By gather: lane l of warp w < kGatherWarps requests box j % 2 of a pair and the four rows 4 (j / 2) .. of it,
    // j = w + kGatherWarps l; the other warps copy the rows behind those, as by address (lane l holds the pool row).
    // Nothing that takes long stands between a tile's copies: while tile i is copied, the columns of tile i + 2 are
    // being read, the rows of tile i + 1 are on their way into L2 (its columns have arrived), and the next node's
    // record is in registers.
    constexpr int kInstr = (64 + kLoadWarps - 1) / kLoadWarps;  // 10
    const int w = warp - kLoadWarp0;
    const uint32_t r_base = tc::smem_u32(rows) + ((lane >> 3) & 1) * kBox;
    const int c = lane & 15;
    const int my_row = c < kInstr && w + kLoadWarps * c < 64 ? 2 * (w + kLoadWarps * c) + (lane >> 4) : kPR;
    const bool gathers = w < kGatherWarps;
    const int j = w + kGatherWarps * lane;  // this lane's gather of a pair (lane < kGatherLanes)
    const int copy0 = kGatherRows / 2 + w - kGatherWarps;  // a copying warp's row pairs: copy0 + 2 k ..
    const int copy_row = 2 * (copy0 + (kLoadWarps - kGatherWarps) * c) + (lane >> 4);  // (c < kCopyInstr) this lane's
    struct Tile {  // a tile of the walk: query, first key, the end of the CTA's keys of the query, its record
      int qi, k0, keys;
      bool first;  // kSplit: of the query's tiles here
      TreeNode rec;
    };
    TreeNode ahead;  // the record of the query after the walk's
    auto start_query = [&](Tile& t, int qi) {  // the first query from qi on that has keys here; `ahead` is qi's record
      for (; qi < a.Q; qi += q_step) {
        t.rec = ahead;
        ahead = a.nodes[min(qi + q_step, a.Q - 1)];
        key_range<kSplit>(a, node_keys(a, t.rec), t.k0, t.keys);
        if (t.keys > t.k0) break;
      }
      t.qi = qi;
      if constexpr (kSplit) t.first = true;
    };
    auto advance = [&](Tile& t) {
      if (t.qi >= a.Q) return;
      t.k0 += kPR;
      if constexpr (kSplit) t.first = false;
      if (t.k0 >= t.keys) start_query(t, t.qi + q_step);
    };
    struct Columns {  // of this lane's row, of its gather's rows (a copying warp: g[0], of the row it copies), of the
      int own, g[4], last;  // tile's last row
    };
    auto columns = [&](const Tile& t, Columns& x) {
      if (t.qi >= a.Q || !a.sel) return;
      const int32_t* p = a.sel + (size_t)t.qi * a.topk + t.k0;
      const int n = t.rec.nsel - t.k0;
      if (my_row < min(n, kPR)) x.own = __ldg(p + my_row);
      if (n >= kPR) {
        x.last = __ldg(p + kPR - 1);
        if (!gathers) {
          if (c < kCopyInstr) x.g[0] = __ldg(p + copy_row);
        } else if (lane < kGatherLanes) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x.g[e] = __ldg(p + 4 * (j >> 1) + e);
        }
      }
    };
    enum { kByAddress, kByBox, kByGather };
    auto tile_mode = [&](const Tile& t, const Columns& x) {
      if (!a.sel) return t.k0 + kPR <= t.rec.n ? kByBox : kByAddress;
      return t.k0 + kPR <= t.rec.nsel && x.last < t.rec.n ? kByGather : kByAddress;  // (columns ascend)
    };
    auto address = [&](const Tile& t, int mode, int col) -> const __nv_bfloat16* {
      if (t.qi >= a.Q || my_row >= kPR || t.k0 + my_row >= t.keys || mode == kByBox) return nullptr;
      const __nv_bfloat16* p = key_row(a, t.rec, t.qi, t.k0 + my_row, col);
#pragma unroll
      for (int e = 0; e < 8; ++e) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 64 * e));
      return p;
    };
    ahead = a.nodes[q_first];  // (the grid has at most Q clusters)
    Tile cur, nxt;
    Columns col{};
    start_query(cur, q_first);
    columns(cur, col);
    int mode = cur.qi < a.Q ? tile_mode(cur, col) : kByAddress;
    const __nv_bfloat16* ptr = address(cur, mode, col.own);
    int g0 = col.g[0], g1 = col.g[1], g2 = col.g[2], g3 = col.g[3];
    nxt = cur;
    advance(nxt);
    columns(nxt, col);
    // the warp's cp.async copies of pair m have been issued: those of the pair before are waited for and reported
    auto copied = [&](int m) {
      tc::cp_async_commit();
      if (m >= 1) {
        tc::cp_async_wait_group<1>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(rows_full + m - 1);
      }
    };
    uint32_t nq = 0, nt = 0;
    for (; cur.qi < a.Q && !failed; ++nt) {
      if (kSplit ? cur.first : cur.k0 == 0) {
        if (w == 0 && lane == 0) {
          // the query block, once the previous query's last score product has retired
          if (nq > 0 && !tc::mbar_wait(q_empty, (nq - 1) & 1)) failed = true;
          if (!failed) {
            tc::mbar_arrive_expect_tx(q_full, 8 * kQBox);
            for (int m = 0; m < 8; ++m) tc::tma_load_2d(qbuf + m * kQBox, &tm_q, q_full, 64 * m, cur.qi * kAH);
          }
        }
        ++nq;
      }
      const uint32_t par = (nt - 1) & 1;  // phase of the previous tile's releases
      const int pairs = (min(kPR, (cur.keys - cur.k0 + 15) & ~15)) >> 1;  // row pairs that the products read
      const long long mine = reinterpret_cast<long long>(ptr);
      const int how = mode, row0 = (cur.qi / a.T) * a.cap;
      const int box_row = row0 + cur.k0, a0 = row0 + g0, a1 = row0 + g1, a2 = row0 + g2, a3 = row0 + g3;
      // the next tile's rows into L2, the columns of the one after it
      cur = nxt;
      if (cur.qi < a.Q) mode = tile_mode(cur, col);
      ptr = address(cur, mode, col.own);
      g0 = col.g[0]; g1 = col.g[1]; g2 = col.g[2]; g3 = col.g[3];
      advance(nxt);
      columns(nxt, col);
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        if (nt > 0 && !failed && !tc::mbar_wait(box_free + m, par)) failed = true;
        if (__any_sync(0xffffffffu, failed)) { failed = true; break; }
        if (how == kByBox) {
          if (lane == 0 && w == 0) {
            tc::mbar_arrive_expect_tx(rows_full + m, 2 * kBox);
            tc::tma_load_2d(rows + 2 * m * kBox, &tm_pool, rows_full + m, 128 * m, box_row);
            tc::tma_load_2d(rows + (2 * m + 1) * kBox, &tm_pool, rows_full + m, 128 * m + 64, box_row);
          } else if (lane == 0) {
            tc::mbar_arrive(rows_full + m);
          }
          continue;
        }
        if (how == kByGather) {
          if (gathers) {
            if (lane == 0) tc::mbar_arrive_expect_tx(rows_full + m, kGatherLanes * 512);
            __syncwarp();
            if (lane < kGatherLanes)
              tc::tma_gather4(rows + (2 * m + (j & 1)) * kBox + (j >> 1) * 512, &tm_row, rows_full + m,
                              64 * (2 * m + (j & 1)), a0, a1, a2, a3);
            continue;
          }
#pragma unroll
          for (int k = 0; k < kCopyInstr; ++k) {
            const int pool_row = __shfl_sync(0xffffffffu, a0, k + (lane & 16));
            const int r = 2 * (copy0 + (kLoadWarps - kGatherWarps) * k) + (lane >> 4);
            tc::cp_async16(r_base + 2 * m * kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           a.pool + (size_t)pool_row * kAD + 128 * m + 8 * c, 16u);
          }
          copied(m);
          continue;
        }
        const __nv_bfloat16* src[kInstr];
#pragma unroll
        for (int k = 0; k < kInstr; ++k)
          src[k] = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(0xffffffffu, mine, k + (lane & 16)));
#pragma unroll
        for (int k = 0; k < kInstr; ++k) {
          const int i = w + kLoadWarps * k, r = 2 * i + (lane >> 4);
          tc::cp_async16_if(i < pairs, r_base + 2 * m * kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                        src[k] ? src[k] + 128 * m + 8 * c : a.pool, src[k] ? 16u : 0u);
        }
        copied(m);
      }
      if (failed) break;
      if (how == kByBox || (how == kByGather && gathers)) continue;
      tc::cp_async_wait_group<0>();
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(rows_full + 3);
    }
    tc::cp_async_wait_all();
    // after a failed wait the bulk copies in flight are given their time (the products wait for them otherwise)
    if (failed && lane == 0) {
      if (nq > 0 && w == 0) tc::mbar_wait(q_full, (nq - 1) & 1);
      for (int m = 0; m < 4; ++m) tc::mbar_wait(rows_full + m, nt & 1);
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ softmax and epilogue
    const int quad = warp & 3, half = warp >> 2, hb = 32 * half, row = 32 * quad + lane;
    const int bar = 1 + half;
    const uint32_t ts = tmem + ((uint32_t)(32 * quad) << 16) + hb;  // this warp's lanes, this half's columns
    const float4* nr4 = reinterpret_cast<const float4*>(nref + hb);
    const float2 sc2 = make_float2(a.scale2, a.scale2);
    // a head's reference before any raise: its sink (kept finite: a sink of -inf raises on the first tile)
    const float z2 = __ldg(a.sink + hb + lane) * 1.4426950408889634f;
    const float ref0 = fminf(fmaxf(z2, -3e38f), 3e38f);
    uint8_t* stage = pbuf + half * kPPart;  // the epilogue's: two buffers of 32 heads x 128 dims
    uint8_t* pdst = pbuf + (row >> 3) * 1024 + (row & 7) * 128;
    uint32_t nq = 0, nt = 0;
    int p_next = a.nodes[q_first].p, nsel_next = a.nodes[q_first].nsel;
    for (int qi = q_first; qi < a.Q && !failed; qi += q_step) {
      const int p = p_next, all_keys = nsel_next < 0 ? 0 : nsel_next + min(a.W, p + 1);
      // the next record is on its way while this node is worked on
      const TreeNode* next = a.nodes + min(qi + q_step, a.Q - 1);
      p_next = next->p;
      nsel_next = next->nsel;
      if (all_keys == 0) continue;
      int first, keys;
      key_range<kSplit>(a, all_keys, first, keys);
      // the previous query's stores have read the P buffer, its 1 / Z has been used
      if (quad == 0 && lane == 0) bulk_wait_read<0>();
      if (quad == 0) nref[hb + lane] = -ref0;
      tc::named_bar(kBarAll, kSoft);
      float2 l[16];
#pragma unroll
      for (int h = 0; h < 16; ++h) l[h] = make_float2(0.f, 0.f);
      for (int k0 = first; k0 < keys; k0 += kPR, ++nt) {
        if (!tc::mbar_wait(s_full, nt & 1)) failed = true;
        tc::fence_after_sync();
        const bool live = k0 + row < keys;
        float2 x[16];  // scores over the reference (log2 units), then probabilities
        float mx = -INFINITY;
        auto scores = [&]() {
          uint32_t u[32];
          tc::tmem_ld32(ts + kColS, u);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 r = nr4[i];
            x[2 * i] = __ffma2_rn(make_float2(__uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1])), sc2,
                                  make_float2(r.x, r.y));
            x[2 * i + 1] = __ffma2_rn(make_float2(__uint_as_float(u[4 * i + 2]), __uint_as_float(u[4 * i + 3])), sc2,
                                      make_float2(r.z, r.w));
          }
        };
        // fp32 for the sums (left in x), two bf16 parts of P^T (MN-major) for the PV products
        auto probabilities = [&]() {
          if (!live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = make_float2(-INFINITY, -INFINITY);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 e = make_float2(ex2(x[4 * j + k].x), ex2(x[4 * j + k].y));
              x[4 * j + k] = e;
              const __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
              hi[k] = *reinterpret_cast<const uint32_t*>(&h);
              const __nv_bfloat162 d = __floats2bfloat162_rn(e.x - __uint_as_float(hi[k] << 16),
                                                             e.y - __uint_as_float(hi[k] & 0xffff0000u));
              lo[k] = *reinterpret_cast<const uint32_t*>(&d);
            }
            const int off = ((4 * half + j) ^ (row & 7)) << 4;
            *reinterpret_cast<uint4*>(pdst + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(pdst + kPPart + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          tc::fence_proxy_async_smem();
        };
        scores();
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fmaxf(x[i].x, x[i].y));
        probabilities();
        // The tile's probabilities stand unless a logit was above the headroom: the question goes round once they are
        // written, when the half's warps have to meet anyway (a failed wait goes round with it).
        if (tc::named_bar_any(bar, kHalf, failed || (live && mx > kRaiseAt))) {
          if (tc::named_bar_any(bar, kHalf, failed)) {
            failed = true;
            break;
          }
          // the reference of such a head becomes the tile's column maximum; the sums and O^T are rescaled
          float v[32];
          {
            uint32_t u[32];
            tc::tmem_ld32(ts + kColS, u);
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 32; ++h) v[h] = live ? __uint_as_float(u[h]) * a.scale2 : -INFINITY;
          }
          red[quad * 64 + hb + lane] = reduce_scatter32<true>(v);
          tc::named_bar(bar, kHalf);
#pragma unroll
          for (int h = 0; h < 32; ++h) {  // v: the factor of head h
            const float m = fmaxf(fmaxf(red[hb + h], red[64 + hb + h]), fmaxf(red[128 + hb + h], red[192 + hb + h]));
            const float old = -nref[hb + h];
            v[h] = m > old + kRaiseAt ? exp2f(old - m) : 1.f;
          }
          tc::named_bar(bar, kHalf);
          if (quad == 0) {
            const float m = fmaxf(fmaxf(red[hb + lane], red[64 + hb + lane]),
                                  fmaxf(red[128 + hb + lane], red[192 + hb + lane]));
            if (m > -nref[hb + lane] + kRaiseAt) nref[hb + lane] = -m;
          }
          tc::named_bar(bar, kHalf);
#pragma unroll
          for (int h = 0; h < 16; ++h) l[h] = __fmul2_rn(l[h], make_float2(v[2 * h], v[2 * h + 1]));
          if (k0 > first) {  // every earlier PV product has retired (S^T was issued after it)
#pragma unroll 1
            for (int g = 0; g < 7; ++g) {
              const uint32_t ta = ts + (g < 6 ? 64 * g : kColO3);
              uint32_t o[32];
              tc::tmem_ld32(ta, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < 32; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * v[h]);
              tc::tmem_st32(ta, o);
            }
            tc::tmem_wait_st();
          }
          scores();
          probabilities();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full);
#pragma unroll
        for (int h = 0; h < 16; ++h) l[h] = __fadd2_rn(l[h], x[h]);
      }
      // ---- the output: 1 / Z per head, then O^T dim by dim.  After a failed wait a half comes here at once: the barrier
      // of all softmax warps below is where both learn of it and leave together.
      if (!failed) {
        float v[32];
#pragma unroll
        for (int h = 0; h < 16; ++h) {
          v[2 * h] = l[h].x;
          v[2 * h + 1] = l[h].y;
        }
        red[quad * 64 + hb + lane] = reduce_scatter32<false>(v);
      }
      tc::named_bar(bar, kHalf);
      if (quad == 0 && !failed) {
        const int h = hb + lane;
        const float sum = (red[h] + red[64 + h]) + (red[128 + h] + red[192 + h]);
        invz[h] = kSplit ? sum : 1.0f / (exp2f(z2 + nref[h]) + sum);
      }
      // inverse RoPE of this thread's dim of tile 3 (dims 448-511 are lane quarters 2 and 3)
      float rc = 1.f, rs = 0.f;
      if (quad >= 2) rope_cs(p, a.inv_freq, (32 * quad + lane - 64) >> 1, &rc, &rs);
      if (!failed && (!kSplit || first < keys) && !tc::mbar_wait(pv_done, (nt - 1) & 1)) failed = true;
      // both halves: P is no longer read, the buffers may take outputs
      if (tc::named_bar_any(kBarAll, kSoft, failed)) {
        failed = true;
        break;
      }
      tc::fence_after_sync();
      if constexpr (kSplit) {
        // The CTA's part of O^T into its own shared memory, [64 heads][512 dims] over the key rows (the last products
        // have retired), its sums and references beside it.
        float* part = reinterpret_cast<float*>(rows) + hb * kAD + row;
#pragma unroll 1
        for (int m = 0; m < 4 && first < keys; ++m) {
          uint32_t u[32];
          tc::tmem_ld32(ts + (m < 3 ? 128 * m : kColO3), u);
          tc::tmem_wait_ld();
          if (m < 3) {
            uint32_t u2[32];
            tc::tmem_ld32(ts + 128 * m + 64, u2);
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 32; ++h) u[h] = __float_as_uint(__uint_as_float(u[h]) + __uint_as_float(u2[h]));
          }
#pragma unroll
          for (int h = 0; h < 32; ++h) part[h * kAD + 128 * m] = __uint_as_float(u[h]);
        }
        joins = qi;
        break;  // (a cluster has one query)
      }
      const float4* iz4 = reinterpret_cast<const float4*>(invz + hb);
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        uint8_t* buf = stage + (m & 1) * 8192;  // [2 boxes of 64 dims][32 heads][128 B], 128-byte swizzle
        uint32_t u[32];
        tc::tmem_ld32(ts + (m < 3 ? 128 * m : kColO3), u);
        tc::tmem_wait_ld();
        float o[32];
        if (m < 3) {
          uint32_t u2[32];
          tc::tmem_ld32(ts + 128 * m + 64, u2);
          tc::tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 32; ++h) o[h] = __uint_as_float(u[h]) + __uint_as_float(u2[h]);
        } else {
#pragma unroll
          for (int h = 0; h < 32; ++h) o[h] = __uint_as_float(u[h]);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(o_free);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 z = iz4[i];
          o[4 * i] *= z.x;
          o[4 * i + 1] *= z.y;
          o[4 * i + 2] *= z.z;
          o[4 * i + 3] *= z.w;
        }
        if (m == 3 && quad >= 2) {
#pragma unroll
          for (int h = 0; h < 32; ++h) {
            const float partner = __shfl_xor_sync(0xffffffffu, o[h], 1);
            o[h] = (lane & 1) ? fmaf(-partner, rs, o[h] * rc) : fmaf(o[h], rc, partner * rs);
          }
        }
        if (m >= 2) {  // the buffer's previous store has been read
          if (quad == 0 && lane == 0) bulk_wait_read<1>();
          tc::named_bar(bar, kHalf);
        }
        // dim 32 quad + lane of the tile: box quad / 2, 16-byte chunk (dim % 64) / 8
        const int d = (row & 63);
        uint8_t* dst = buf + (quad >> 1) * 4096 + (d & 7) * 2;
#pragma unroll
        for (int h = 0; h < 32; ++h)
          *reinterpret_cast<__nv_bfloat16*>(dst + h * 128 + (((d >> 3) ^ (h & 7)) << 4)) = __float2bfloat16_rn(o[h]);
        tc::fence_proxy_async_smem();
        tc::named_bar(bar, kHalf);
        if (quad == 0 && lane == 0) {
          tma_store_2d(&tm_out, buf, 128 * m, qi * kAH + hb);
          tma_store_2d(&tm_out, buf + 4096, 128 * m + 64, qi * kAH + hb);
          bulk_commit();
        }
      }
      ++nq;
    }
    if (quad == 0 && lane == 0) bulk_wait_all();  // shared memory is read, the output written
  }
  if constexpr (kSplit) {
    __syncwarp();
    tc::cluster_sync();  // the parts are written
    if (joins >= 0) join_parts(a, rows, nref, invz, reinterpret_cast<float*>(pbuf), joins);
    __syncwarp();
    tc::cluster_sync();  // ... and read
  }
  if (failed) atomicOr(a.err, tc::kErrTimeout);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// Clusters of S CTAs, one CTA an SM, that run at once (a property of the device: asked once for each).
int clusters(int S) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxSplit + 1];  // 0: not asked yet, else 1 + n
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
  int n = known[dev][S].load(std::memory_order_relaxed) - 1;
  if (n < 0) {
    allow_smem<kSmem>(k_tc_tree_attend<true>);
    n = max_clusters(k_tc_tree_attend<true>, kThreads, kSmem, S);
    known[dev][S].store(n + 1, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace

cudaError_t launch_tc_attend_tree(const Dims& L, const TreeAttend& t, const int32_t* sel, int32_t* err,
                                  cudaStream_t s) {
  int sms = 0, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  TaArgs a{};
  a.pool = static_cast<const __nv_bfloat16*>(t.pool);
  a.ring = static_cast<const __nv_bfloat16*>(t.window);
  a.kv = static_cast<const __nv_bfloat16*>(t.kv);
  a.rows = static_cast<const __nv_bfloat16*>(t.rows);
  a.sel = sel; a.nodes = t.ws.nodes; a.sink = t.sink; a.inv_freq = t.inv_freq;
  a.Q = t.B * t.T; a.T = t.T; a.cap = t.cap; a.topk = L.topk; a.W = L.W; a.Wr = L.Wr;
  a.scale2 = L.scale * 1.4426950408889634f;
  a.err = err;
  CUtensorMap tq, to, tp, tr;
  if (!make_tmap_2d_bf16(&tq, t.q, (uint64_t)a.Q * kAH, kAD, kAD * 2, 64) ||
      !make_tmap_2d_bf16(&to, t.out, (uint64_t)a.Q * kAH, kAD, kAD * 2, 32) ||
      !make_tmap_2d_bf16(&tp, t.pool, (uint64_t)t.B * t.cap, kAD, kAD * 2, kPR) ||
      !make_tmap_2d_bf16(&tr, t.pool, (uint64_t)t.B * t.cap, kAD, kAD * 2, 1))
    return cudaErrorInvalidValue;
  a.out = static_cast<__nv_bfloat16*>(t.out);
  const long long tiles = ((t.scores ? L.topk : (long long)t.cap + t.T) + L.W + kPR - 1) / kPR;
  for (a.S = kMaxSplit; a.S > 1; a.S /= 2)
    if (tiles >= 2 * a.S && a.Q <= clusters(a.S)) {
      allow_smem<kSmem>(k_tc_tree_attend<true>);
      const cudaError_t e = launch_pdl_cluster(k_tc_tree_attend<true>, dim3(a.Q * a.S), dim3(kThreads), kSmem, s, a.S,
                                               tq, to, tp, tr, a);
      return e != cudaSuccess ? e : cudaGetLastError();
    }
  allow_smem<kSmem>(k_tc_tree_attend<false>);
  CSA_LAUNCH(k_tc_tree_attend<false>, dim3(min(a.Q, sms)), dim3(kThreads), kSmem, s, tq, to, tp, tr, a);
  return cudaGetLastError();
}

}  // namespace csa
