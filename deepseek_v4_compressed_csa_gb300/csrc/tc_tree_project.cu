// Projections of a tree's drafted tokens on the 5th-generation tensor cores (bf16): for one or both pools of a layer
//   proj[tok][o] = sum_k W[o][k] x[tok][k],  W = [wkv ; wgate], rounded once,
// written to the nodes' entries of the draft buffers (unused slots are left as they were).
//
// C^T = W x^T: M = 128 output features per tile, N <= 256 tokens, the hidden axis streamed by TMA in 64-wide blocks.
// A draft has tens to hundreds of tokens: too few tiles to fill the GPU with whole sums (20 feature tiles for the
// Flash pools), so the hidden axis is split over the S CTAs of a cluster.  They add their parts through distributed
// shared memory: each CTA leaves its fp32 part in its own shared memory (the stage buffers, free by then), and CTA r
// sums the S parts, in split order, of N / S tokens and writes them.  No partial sum goes to memory and no second
// pass reads one.  Both pools are one grid.  Bound by the weights' stream (21 MB for both Flash pools) for few tokens
// (8 tokens: 8.6 us with the pooling behind it, six splits; four took 1.6 us longer, seven 6.5, since their clusters do
// not all run at once, and products issued by a thread that a lane number chose, not elect.sync, 2.1), by the tiles' way
// into shared memory for many (512 tokens: 23.5 us with the pooling; 48 KB of weights and tokens for 512 clocks of
// products).
#include <atomic>

#include "kernels.h"
#include "tc.cuh"
#include "tree.cuh"

namespace csa {

namespace {

constexpr int kThreads = 320;       // warp 0 TMA, warp 1 MMA and TMEM, warps 2-9 accumulators out; all add
constexpr int kABytes = 128 * 128;  // 128 features x 64 values
constexpr int kMaxStages = 8, kMaxSplit = 8;
constexpr int kMaxSmem = 1024 + 200 * 1024;

struct TpArgs {
  __nv_bfloat16* proj[2];
  int Ld[2], m_tiles[2];
  int ntok, T, N, n_tiles, S, kblk, stages;
  const int32_t* parent;
  const int32_t* pos;
  int32_t* err;
};

// Tokens [c0, c1) of the tile: S parts added in split order, one warp per token, four features a lane.  Twelve to
// sixteen remote loads in flight a lane: one token at a time costs the latency of its parts each time (5 us for 512
// tokens).
template <int S>
__device__ __forceinline__ void add_parts(const float* part, int c0, int c1, const uint8_t* live, __nv_bfloat16* out,
                                          int stride) {
  constexpr int kWarps = kThreads / 32, U = S > 4 ? 2 : 12 / S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int c = c0 + warp; c < c1; c += U * kWarps) {
    float4 v[U][S];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float* at = part + min(c + k * kWarps, c1 - 1) * 128 + 4 * lane;
#pragma unroll
      for (int s = 0; s < S; ++s)
        v[k][s] = S > 1 ? tc::ld_cluster_f4(tc::cluster_map(at, s)) : *reinterpret_cast<const float4*>(at);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float4 t = v[k][0];
#pragma unroll
      for (int s = 1; s < S; ++s) {
        t.x += v[k][s].x;
        t.y += v[k][s].y;
        t.z += v[k][s].z;
        t.w += v[k][s].w;
      }
      const int at = c + k * kWarps;
      if (at >= c1 || !live[at]) continue;
      uint2 pk;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&pk);
      h[0] = __floats2bfloat162_rn(t.x, t.y);
      h[1] = __floats2bfloat162_rn(t.z, t.w);
      *reinterpret_cast<uint2*>(out + (size_t)at * stride) = pk;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    k_tc_tree_project(const __grid_constant__ CUtensorMap tm_wkv0, const __grid_constant__ CUtensorMap tm_wg0,
                      const __grid_constant__ CUtensorMap tm_wkv1, const __grid_constant__ CUtensorMap tm_wg1,
                      const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ TpArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full;
  __shared__ uint32_t tmem_slot;
  __shared__ uint8_t live[256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = a.N, stage_bytes = kABytes + N * 128;
  const int split = blockIdx.x % a.S, tile = blockIdx.x / a.S;
  const int n = tile % a.n_tiles;
  int m = tile / a.n_tiles;
  const int pool = m >= a.m_tiles[0];
  if (pool) m -= a.m_tiles[0];
  const int Ld = a.Ld[pool];
  const bool gate = m * 128 >= Ld;
  const CUtensorMap* wmap = pool ? (gate ? &tm_wg1 : &tm_wkv1) : (gate ? &tm_wg0 : &tm_wkv0);
  const int wrow = m * 128 - (gate ? Ld : 0);
  const int k0 = a.kblk * split / a.S, nk = a.kblk * (split + 1) / a.S - k0;
  const uint32_t tcols = N <= 32 ? 32 : (N <= 64 ? 64 : (N <= 128 ? 128 : 256));
  const int first = min(a.stages, nk);
  if (warp == 0 && tc::elect_one()) {
    for (int s = 0; s < a.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(&acc_full, 1);
    tc::fence_mbar_init();
    tc::tma_prefetch(wmap);
    tc::tma_prefetch(&tm_x);
    // the ring's first fill before the programmatic wait: weights and tokens are inputs of the step
    for (int kb = 0; kb < first; ++kb) {
      uint8_t* st = smem + kb * stage_bytes;
      tc::mbar_arrive_expect_tx(&full[kb], stage_bytes);
      tc::tma_load_2d(st, wmap, &full[kb], (k0 + kb) * 64, wrow);
      tc::tma_load_2d(st + kABytes, &tm_x, &full[kb], (k0 + kb) * 64, n * N);
    }
  }
  pdl_wait();
  pdl_trigger();  // (not before: the pooling reads the tree and the positions ahead of its own wait)
  if (warp == 1) {
    tc::tmem_alloc(&tmem_slot, tcols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  bool failed = false;

  if (warp == 0) {
    if (tc::elect_one()) {
      for (int kb = first; kb < nk; ++kb) {
        const int s = kb % a.stages;
        if (!tc::mbar_wait(&empty[s], ((kb / a.stages) & 1) ^ 1)) { failed = true; break; }
        uint8_t* st = smem + s * stage_bytes;
        tc::mbar_arrive_expect_tx(&full[s], stage_bytes);
        tc::tma_load_2d(st, wmap, &full[s], (k0 + kb) * 64, wrow);
        tc::tma_load_2d(st + kABytes, &tm_x, &full[s], (k0 + kb) * 64, n * N);
      }
    }
  } else if (warp == 1) {
    if (tc::elect_one()) {
      const uint32_t idesc = tc::idesc_bf16(128, N);
      const uint64_t base = tc::sdesc_kmajor_sw128(tc::smem_u32(smem));
      int s = 0;
      uint32_t phase = 0;
#pragma unroll 1
      for (int kb = 0; kb < nk; ++kb) {
        if (!tc::mbar_wait(&full[s], phase)) { failed = true; break; }
        tc::fence_after_sync();
        const uint64_t ad = base + ((uint32_t)(s * stage_bytes) >> 4), bd = ad + (kABytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // (32 bytes further: two descriptor address units)
          tc::mma_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, (kb > 0 || k > 0) ? 1u : 0u);
        tc::mma_commit(&empty[s]);
        if (++s == a.stages) { s = 0; phase ^= 1; }
      }
      tc::mma_commit(&acc_full);  // every MMA, and so every load, has retired when this completes
    }
  } else {
    // which of the tile's tokens are nodes (the walk stands behind the products)
    for (int c = threadIdx.x - 64; c < N; c += kThreads - 64) {
      const int tok = n * N + c, b = tok / a.T;
      bool ok = tok < a.ntok && tree_pos_ok(a.pos[min(b, (a.ntok - 1) / a.T)]);
      if (ok) {
        const int32_t* row = a.parent + (size_t)b * a.T;
        for (int i = tok - b * a.T; i >= 0;) {
          const int p = __ldg(row + i);
          if (p >= i || p < -1) { ok = false; break; }
          i = p;
        }
      }
      live[c] = ok;
    }
  }
  // (the other roles' threads wait here: the accumulator is complete for everyone)
  if (!tc::mbar_wait(&acc_full, 0)) failed = true;
  tc::fence_after_sync();
  float* part = reinterpret_cast<float*>(smem);  // [N][128]
  const int nt = min(N, a.ntok - n * N);         // the tile's tokens
  if (warp >= 2) {
    const int quarter = warp & 3;
    for (int c0 = warp < 6 ? 0 : 32; c0 < nt; c0 += 64) {
      uint32_t u[32];
      tc::tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + c0, u);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) part[(c0 + i) * 128 + quarter * 32 + lane] = __uint_as_float(u[i]);
    }
  }
  tc::fence_before_sync();
  if (a.S > 1) tc::cluster_sync();
  else __syncthreads();
  // this CTA's tokens of the tile
  const int c0 = nt * split / a.S, c1 = nt * (split + 1) / a.S;
  __nv_bfloat16* out = a.proj[pool] + (size_t)n * N * 2 * Ld + m * 128 + 4 * lane;
  switch (a.S) {
    case 1: add_parts<1>(part, c0, c1, live, out, 2 * Ld); break;
    case 2: add_parts<2>(part, c0, c1, live, out, 2 * Ld); break;
    case 3: add_parts<3>(part, c0, c1, live, out, 2 * Ld); break;
    case 4: add_parts<4>(part, c0, c1, live, out, 2 * Ld); break;
    case 5: add_parts<5>(part, c0, c1, live, out, 2 * Ld); break;
    case 6: add_parts<6>(part, c0, c1, live, out, 2 * Ld); break;
    case 7: add_parts<7>(part, c0, c1, live, out, 2 * Ld); break;
    default: add_parts<8>(part, c0, c1, live, out, 2 * Ld); break;
  }
  if (failed) atomicOr(a.err, tc::kErrTimeout);
  if (a.S > 1) tc::cluster_sync();  // the parts stay in place until the others have read them
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, tcols);
}

struct Plan {
  int N, n_tiles, S, stages, smem;
};

// Clusters of S CTAs, one CTA an SM, that run at once (a property of the device: asked once for each).
int clusters(int S) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxSplit + 1];  // 0: not asked yet, else 1 + n
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
  int n = known[dev][S].load(std::memory_order_relaxed) - 1;
  if (n < 0) {
    allow_smem<kMaxSmem>(k_tc_tree_project);
    n = max_clusters(k_tc_tree_project, kThreads, kMaxSmem, S);
    known[dev][S].store(n + 1, std::memory_order_relaxed);
  }
  return n;
}

// Tokens per tile and splits: the pair whose slowest CTA needs the fewest tensor clocks (an MMA of 128 x N x 16 takes
// max(32 + N / 4, N / 2) of them: up to N = 128 it waits for shared memory), with all clusters running at once; a
// tile costs about 6000 clocks beside its products (launch, first fill, the parts' exchange).
Plan plan(int m_tiles, int ntok, int kblk, int sms) {
  Plan best{};
  long best_cost = -1;
  int most[kMaxSplit + 1];  // clusters of S at once
  for (int S = 2; S <= kMaxSplit; ++S) most[S] = clusters(S);
  for (int N = 32; N <= 256; N += 32) {
    const int n_tiles = (ntok + N - 1) / N;
    for (int S = 1; S <= kMaxSplit && S <= kblk; ++S) {
      const long tiles = (long)m_tiles * n_tiles;
      if (S > 1 && tiles > most[S]) break;  // (fewer still of a larger cluster)
      const long waves = S > 1 ? 1 : (tiles + sms - 1) / sms;
      const long mma = max(32 + N / 4, N / 2);
      const long cost = waves * (6000 + (long)((kblk + S - 1) / S) * 4 * mma);
      if (best_cost < 0 || cost < best_cost || (cost == best_cost && S < best.S)) {
        best_cost = cost;
        best.N = N;
        best.n_tiles = n_tiles;
        best.S = S;
      }
    }
  }
  const int stage = kABytes + best.N * 128;
  best.stages = max(2, min(kMaxStages, (200 * 1024) / stage));
  best.smem = 1024 + max(best.stages * stage, best.N * 128 * 4);
  return best;
}

}  // namespace

bool tc_tree_project_supported(const Dims& L, int d) {
  return L.dtype == CSA_BF16 && L.X % 64 == 0 && (L.lanes * d) % 128 == 0;
}

cudaError_t launch_tc_tree_project(const Dims& L, const TreeCompress* pools, int npool, const void* x, int B, int T,
                                   const int32_t* parent, const int32_t* pos, int32_t* err, cudaStream_t s) {
  int sms = 0, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  TpArgs a{};
  CUtensorMap tw[2], tg[2], tx;
  int m_tiles = 0;
  for (int k = 0; k < npool; ++k) {
    const csa_compressor* c = pools[k].comp;
    a.Ld[k] = L.lanes * c->d;
    a.m_tiles[k] = 2 * a.Ld[k] / 128;
    a.proj[k] = static_cast<__nv_bfloat16*>(pools[k].proj);
    m_tiles += a.m_tiles[k];
    if (!make_tmap_2d_bf16(&tw[k], c->wkv, a.Ld[k], L.X, (uint64_t)L.X * 2, 128) ||
        !make_tmap_2d_bf16(&tg[k], c->wgate, a.Ld[k], L.X, (uint64_t)L.X * 2, 128))
      return cudaErrorInvalidValue;
  }
  if (npool == 1) {
    tw[1] = tw[0];
    tg[1] = tg[0];
  }
  const Plan p = plan(m_tiles, B * T, L.X / 64, sms);
  if (!make_tmap_2d_bf16(&tx, x, (uint64_t)B * T, L.X, (uint64_t)L.X * 2, p.N)) return cudaErrorInvalidValue;
  a.ntok = B * T; a.T = T; a.N = p.N; a.n_tiles = p.n_tiles; a.S = p.S; a.kblk = L.X / 64; a.stages = p.stages;
  a.parent = parent; a.pos = pos; a.err = err;
  allow_smem<kMaxSmem>(k_tc_tree_project);
  const dim3 grid(m_tiles * p.n_tiles * p.S);
  const cudaError_t e =
      p.S > 1 ? launch_pdl_cluster(k_tc_tree_project, grid, dim3(kThreads), p.smem, s, p.S, tw[0], tg[0], tw[1], tg[1],
                                   tx, a)
              : launch_pdl(k_tc_tree_project, grid, dim3(kThreads), p.smem, s, tw[0], tg[0], tw[1], tg[1], tx, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
