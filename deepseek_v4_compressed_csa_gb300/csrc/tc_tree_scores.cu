// Index scores of a tree's nodes on the 5th-generation tensor cores (Hi = 64 heads of Di = 128 dims; keys in bf16, or
// fp8 rows: kFp8).
//
// score[i][j] = sum_h w_ih ReLU(iq_ih . key_j), w = iw Di^-1/2 Hi^-1/2, for the committed keys of the node's sequence
// and the index rows of its tree (definition: include/csa.h, csa_index_scores_tree).
//
// The product is computed transposed, S^T = K Q^T: M = 128 key rows per tile (TMEM lane = key row), N = 4 nodes x 64
// heads, K = 128.  An epilogue thread then owns one key row and reduces the heads by itself.  Four nodes of a
// sequence share every key tile: a tile (32 KB) costs eight 128 x 256 x 16 products (~1024 tensor clocks), which is
// slower than fetching it from L2, so the kernel is bound by the tensor pipe for four nodes or more and by the key
// stream for fewer.  The tree's own rows are one more tile per group (T <= 64 rows of the draft buffer), masked by
// the path: they need no launch of their own.
//
// Work: the (sequence, group of 4 nodes, tile) triples that exist, in that order, cut into equal runs, one per CTA
// (one CTA per SM).  Each CTA finds its run by a scan over the sequences' row counts, so ragged batches stay
// balanced.  Ten warps: 0 TMA (a ring of three key tiles, two query blocks of 64 KB), 1 MMA (two accumulators of 256
// columns), 2-9 epilogue: two warps per TMEM lane quarter, two nodes each.  Of shared memory's 128 bytes a clock the
// products take 96 and the key tiles 32, so the epilogue stays away from it: a warp keeps its 128 head weights in
// registers, two bf16 to each (read from shared memory for every tile they cost 256 of a tile's clocks, and 60 us
// became what 512 nodes over 8.2K rows took).
//
// fp8 rows (fp8_row.cuh): k_tree_quant_iq brings the queries into the same form, and the heads' scales and the 1/128 of
// the rotation into their weights; the product is one of E4M3 codes, four of 128 x 256 x 32 a tile in half the clocks.
// The row's scale comes after the heads' sum (it is not negative, so that ReLU lets it through).  The epilogue is the
// longer part then: its weights are fp32, too many for registers (72 us), so sixteen warps of one node each read them
// from shared memory, which has the room: 58 us for 512 nodes over 8.2K rows (61 with eight warps of two nodes), where
// the bf16 keys take 47; the fp8 rows' gain is their memory.
#include "fp8_row.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tree.cuh"

namespace csa {

namespace {

constexpr int kRows = 128;               // key rows per tile
constexpr int kG = 4;                    // nodes per group
constexpr int kN = 64 * kG;
constexpr int kQSlots = 2, kAcc = 2;

template <bool kFp8>
struct TsCfg {
  static constexpr int kNodes = kFp8 ? 1 : 2;     // per epilogue warp
  static constexpr int kChunk = kFp8 ? 32 : 64;   // accumulator columns in registers at a time
  static constexpr int kEpiWarps = 4 * kG / kNodes;
  static constexpr int kThreads = 32 * (2 + kEpiWarps);
  static constexpr int kKeyBytes = kRows * (kFp8 ? 128 : 256);  // fp8: one box of 128 codes; bf16: two of 64 dims
  static constexpr int kTileBytes = kKeyBytes + (kFp8 ? kRows * 16 : 0);  // fp8: bytes 128-143 of each row, its scale
  static constexpr int kQBytes = kN * (kFp8 ? 128 : 256);
  static constexpr int kStages = kFp8 ? 6 : 3;
  static constexpr int kOffK = kQSlots * kQBytes;
  static constexpr int kOffScale = kOffK + kStages * kKeyBytes;
  static constexpr int kOffW = kOffK + kStages * kTileBytes;  // fp8: each epilogue warp's 64 head weights
  static constexpr int kOffBars = kOffW + (kFp8 ? kEpiWarps * 64 * 4 : 0);
  static constexpr int kNumBars = 2 * kStages + 2 * kQSlots + 2 * kAcc + 1;
  static constexpr int kOffRun = kOffBars + kNumBars * 8;  // the CTA's run: b, group, tile, count; TMEM address
  static constexpr int kSmem = kOffRun + 32 + 1024;
  static_assert(kSmem <= 232448, "shared memory per block");
};

struct TsArgs {
  const __nv_bfloat16* iw;  // [B, T, 64]
  const float* w8;          // fp8: [B, T, 64] head weights with the query's scale and the 1/128
  const int32_t* parent;
  const int32_t* pos;
  const int32_t* n_rows;
  float wscale;
  int B, T, cap, ratio, groups;  // groups: of kG nodes, per sequence
  float* scores;                 // [B, T, cap + T]
  int32_t* err;
};

// Tiles of a group of sequence b: its committed rows and one of the tree's rows; 0 when the state is inconsistent.
__device__ __forceinline__ int seq_tiles(const TsArgs& a, int b) {
  const int p0 = __ldg(a.pos + b), n = __ldg(a.n_rows + b);
  if (!tree_pos_ok(p0) || n != p0 / a.ratio || n > a.cap) return 0;
  return (n + kRows - 1) / kRows + 1;
}

// Walks the CTA's run group by group: tiles t .. t + cnt - 1 of group g of sequence b, of `tiles` in all.
struct Walk {
  int b, g, t, tiles, left, cnt;
  __device__ __forceinline__ void start(const TsArgs& a, const int* run) {
    b = run[0];
    g = run[1];
    t = run[2];
    left = run[3];
    tiles = left > 0 ? seq_tiles(a, b) : 0;
    cnt = min(left, tiles - t);
  }
  __device__ __forceinline__ void next(const TsArgs& a) {
    left -= cnt;
    if (left <= 0) return;
    t = 0;
    if (++g == a.groups) {
      g = 0;
      do tiles = seq_tiles(a, ++b);
      while (tiles == 0 && b < a.B - 1);
    }
    cnt = min(left, tiles);
  }
};

template <bool kFp8>
__global__ void __launch_bounds__(TsCfg<kFp8>::kThreads, 1)
    k_tc_tree_scores(const __grid_constant__ CUtensorMap tm_keys, const __grid_constant__ CUtensorMap tm_rows,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_key_scales,
                     const __grid_constant__ CUtensorMap tm_row_scales, TsArgs a) {
  using C = TsCfg<kFp8>;
  constexpr int kStages = C::kStages, kTileBytes = C::kTileBytes, kKeyBytes = C::kKeyBytes, kQBytes = C::kQBytes;
  constexpr int kEpiWarps = C::kEpiWarps, kNodes = C::kNodes;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = smem;
  uint8_t* kbuf = smem + C::kOffK;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;
  uint64_t* q_empty = q_full + kQSlots;
  uint64_t* acc_full = q_empty + kQSlots;
  uint64_t* acc_empty = acc_full + kAcc;
  uint64_t* drain = acc_empty + kAcc;
  int* run = reinterpret_cast<int*>(smem + C::kOffRun);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(run + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], kFp8 ? 1 + kEpiWarps : 1);  // its products retired; fp8: its scales read
    }
    for (int s = 0; s < kQSlots; ++s) {
      tc::mbar_init(&q_full[s], 1);
      tc::mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < kAcc; ++s) {
      tc::mbar_init(&acc_full[s], 1);
      tc::mbar_init(&acc_empty[s], kEpiWarps);
    }
    tc::mbar_init(drain, 1);
    tc::fence_mbar_init();
    tc::tma_prefetch(&tm_keys);
    tc::tma_prefetch(&tm_rows);
    tc::tma_prefetch(&tm_q);
    if (kFp8) {
      tc::tma_prefetch(&tm_key_scales);
      tc::tma_prefetch(&tm_row_scales);
    }
  }
  pdl_wait();
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, kAcc * kN);
    tc::tmem_relinquish();
  }
  if (warp == 0) {
    // The CTA's run.  Lane l sums the items of a contiguous share of the sequences; the lane whose share holds the
    // run's first item walks its share for it.
    const int per = (a.B + 31) / 32, b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int tiles = seq_tiles(a, b);
      mine += (long long)tiles * a.groups;
      if (tiles == 0 && blockIdx.x == 0) {  // reported once, and only where there is a node
        bool used = false;
        for (int i = 0; i < a.T; ++i) used |= __ldg(a.parent + (size_t)b * a.T + i) >= -1;
        if (used) atomicOr(a.err, CSA_DEV_STATE);
      }
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    const long long x0 = total * blockIdx.x / gridDim.x, x1 = total * (blockIdx.x + 1) / gridDim.x;
    if (lane == 0) run[3] = (int)(x1 - x0);
    long long at = incl - mine;
    if (x0 < x1 && x0 >= at && x0 < incl) {
      for (int b = b0; b < b1; ++b) {
        const int tiles = seq_tiles(a, b);
        const long long here = (long long)tiles * a.groups;
        if (x0 < at + here) {
          run[0] = b;
          run[1] = (int)((x0 - at) / tiles);
          run[2] = (int)((x0 - at) % tiles);
          break;
        }
        at += here;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool failed = false;
  Walk w;
  w.start(a, run);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA
    if (tc::elect_one()) {
      int stage = 0, nq = 0;
      uint32_t phase = 0, used = 0, par = 0, q_used = 0, q_par = 0;
      for (; w.left > 0 && !failed; w.next(a), ++nq) {
        const int slot = nq % kQSlots;
        const uint32_t ph = (nq / kQSlots) & 1;
        if (!tc::mbar_wait(&q_empty[slot], ph ^ 1)) { failed = true; break; }
        const int qrow = (w.b * a.T + w.g * kG) * 64;
        tc::mbar_arrive_expect_tx(&q_full[slot], kQBytes);
        tc::tma_load_2d(qbuf + slot * kQBytes, &tm_q, &q_full[slot], 0, qrow);
        if (!kFp8) tc::tma_load_2d(qbuf + slot * kQBytes + kQBytes / 2, &tm_q, &q_full[slot], 64, qrow);
        q_used |= 1u << slot;
        q_par = (q_par & ~(1u << slot)) | (ph << slot);
        for (int t = w.t; t < w.t + w.cnt; ++t) {
          if (!tc::mbar_wait(&empty[stage], phase ^ 1)) { failed = true; break; }
          const bool tree = t == w.tiles - 1;
          const CUtensorMap* tm = tree ? &tm_rows : &tm_keys;
          const int row = tree ? w.b * a.T : w.b * a.cap + t * kRows;
          uint8_t* dst = kbuf + stage * kKeyBytes;
          tc::mbar_arrive_expect_tx(&full[stage], kTileBytes);
          tc::tma_load_2d(dst, tm, &full[stage], 0, row);
          if (kFp8)
            tc::tma_load_2d(smem + C::kOffScale + stage * kRows * 16, tree ? &tm_row_scales : &tm_key_scales,
                            &full[stage], 128, row);
          else
            tc::tma_load_2d(dst + kKeyBytes / 2, tm, &full[stage], 64, row);
          used |= 1u << stage;
          par = (par & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      // every load issued must land before the CTA may exit
      for (int s = 0; s < kStages; ++s)
        if (((used >> s) & 1) && !tc::mbar_wait(&full[s], (par >> s) & 1)) failed = true;
      for (int s = 0; s < kQSlots; ++s)
        if (((q_used >> s) & 1) && !tc::mbar_wait(&q_full[s], (q_par >> s) & 1)) failed = true;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    // (one elected thread; descriptors as a base plus constants: what this thread does between two tiles' products is
    // time that the tensor pipe may stand still)
    if (tc::elect_one()) {
      constexpr uint32_t idesc = kFp8 ? tc::idesc_e4m3(kRows, kN) : tc::idesc_bf16(kRows, kN);
      const uint64_t kd = tc::sdesc_kmajor_sw128(tc::smem_u32(kbuf)), qd = tc::sdesc_kmajor_sw128(tc::smem_u32(qbuf));
      int stage = 0, acc = 0, nq = 0;
      uint32_t phase = 0, acc_ph = 0;
      for (; w.left > 0 && !failed; w.next(a), ++nq) {
        const int slot = nq % kQSlots;
        if (!tc::mbar_wait(&q_full[slot], (nq / kQSlots) & 1)) { failed = true; break; }
        const uint64_t bd = qd + slot * (kQBytes >> 4);
#pragma unroll 1
        for (int j = 0; j < w.cnt; ++j) {
          if (!tc::mbar_wait(&full[stage], phase) || !tc::mbar_wait(&acc_empty[acc], acc_ph ^ 1)) {
            failed = true;
            break;
          }
          tc::fence_after_sync();
          const uint64_t ad = kd + stage * (kKeyBytes >> 4);
          const uint32_t d = tmem + acc * kN;
          if constexpr (kFp8) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc::mma_f8(d, ad + 2 * kk, bd + 2 * kk, idesc, kk > 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc::mma_bf16(d, ad + (((kk >> 2) * (kKeyBytes / 2) + (kk & 3) * 32) >> 4),
                           bd + (((kk >> 2) * (kQBytes / 2) + (kk & 3) * 32) >> 4), idesc, kk > 0);
          }
          tc::mma_commit(&empty[stage]);
          tc::mma_commit(&acc_full[acc]);
          if (++acc == kAcc) { acc = 0; acc_ph ^= 1; }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        tc::mma_commit(&q_empty[slot]);
      }
      tc::mma_commit(drain);  // every MMA retires before tensor memory is released
      if (!tc::mbar_wait(drain, 0)) failed = true;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const int q0 = ((warp - 2) >> 2) * kNodes;  // this warp's first node of the group
    int acc = 0, stage = 0;
    uint32_t acc_ph = 0, phase = 0;
    uint64_t closers[kNodes] = {};
    bool live[kNodes] = {};
    uint32_t wt[kNodes][32];  // head weights 2 i (low half) and 2 i + 1 as bf16 (fp8: in shared memory)
    float* wbuf = reinterpret_cast<float*>(smem + C::kOffW) + (warp - 2) * 64;
    const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + q0 * 64;
    for (; w.left > 0; w.next(a)) {
      const int n = a.n_rows[w.b], stride = a.cap + a.T;
      float* out = a.scores + ((size_t)w.b * a.T + w.g * kG + q0) * stride;
#pragma unroll
      for (int u = 0; u < kNodes; ++u) {
        const int i = w.g * kG + q0 + u, node = min(i, a.T - 1);
        const size_t row64 = ((size_t)w.b * a.T + node) * 64;
        if constexpr (kFp8) {
          __syncwarp();
          *reinterpret_cast<float2*>(wbuf + 2 * lane) = __ldg(reinterpret_cast<const float2*>(a.w8 + row64) + lane);
          __syncwarp();
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(a.iw + row64);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 r = __ldg(src + j);
            wt[u][4 * j] = r.x;
            wt[u][4 * j + 1] = r.y;
            wt[u][4 * j + 2] = r.z;
            wt[u][4 * j + 3] = r.w;
          }
        }
        bool bad = false;
        const uint64_t m = tree_path_warp(a.parent + (size_t)w.b * a.T, a.T, node, bad);
        live[u] = i < a.T && m != 0;
        closers[u] = tree_closers(m, a.pos[w.b], a.ratio);
        if (bad && lane == 0) atomicOr(a.err, CSA_DEV_STATE);
      }
#pragma unroll 1
      for (int t = w.t; t < w.t + w.cnt; ++t) {
        // (after a wait that ran out, the run is walked without waiting)
        if (!failed) failed = __any_sync(0xffffffffu, !tc::mbar_wait(&acc_full[acc], acc_ph));
        tc::fence_after_sync();
        const bool tree = t == w.tiles - 1;
        const int col = tree ? n + row : t * kRows + row;
        const bool in = tree ? row < a.T : col < n;
        float scale = a.wscale;
        // (the tile has landed: its products have retired; this wait makes its bytes visible here)
        if constexpr (kFp8) {
          if (!failed) failed = __any_sync(0xffffffffu, !tc::mbar_wait(&full[stage], phase));
          scale *= *reinterpret_cast<const float*>(smem + C::kOffScale + (stage * kRows + row) * 16);
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        uint32_t ta = t0 + acc * kN;
#pragma unroll
        for (int u = 0; u < kNodes; ++u) {
          // four partial sums (heads 0, 1, 2, 3 mod 4), as two packed pairs
          float2 s01 = make_float2(0.f, 0.f), s23 = make_float2(0.f, 0.f);
#pragma unroll
          for (int h0 = 0; h0 < 64; h0 += C::kChunk) {
            uint32_t v[C::kChunk];
#pragma unroll
            for (int k = 0; k < C::kChunk; k += 32) tc::tmem_ld32(ta + h0 + k, v + k);
            tc::tmem_wait_ld();
            if (u == kNodes - 1 && h0 + C::kChunk == 64) {  // the accumulator has been read
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&acc_empty[acc]);
            }
#pragma unroll
            for (int k = 0; k < C::kChunk; k += 4) {
              float2 w01, w23;
              if constexpr (kFp8) {
                const float4 ww = *reinterpret_cast<const float4*>(wbuf + h0 + k);
                w01 = make_float2(ww.x, ww.y);
                w23 = make_float2(ww.z, ww.w);
              } else {
                // (the packed weights change as far as the compiler knows: unpacked ahead of the loop they would not
                // fit)
                uint32_t &w0 = wt[u][(h0 + k) / 2], &w1 = wt[u][(h0 + k) / 2 + 1];
                asm volatile("" : "+r"(w0), "+r"(w1));
                w01 = make_float2(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u));
                w23 = make_float2(__uint_as_float(w1 << 16), __uint_as_float(w1 & 0xffff0000u));
              }
              auto relu = [&](int i) { return fmaxf(__uint_as_float(v[k + i]), 0.f); };
              s01 = __ffma2_rn(w01, make_float2(relu(0), relu(1)), s01);
              s23 = __ffma2_rn(w23, make_float2(relu(2), relu(3)), s23);
            }
          }
          float s = ((s01.x + s01.y) + (s23.x + s23.y)) * scale;
          if (tree && !((closers[u] >> (row & 63)) & 1)) s = -INFINITY;
          if (in && live[u]) out[(size_t)u * stride + col] = s;
          ta += 64;
        }
        if (++acc == kAcc) { acc = 0; acc_ph ^= 1; }
      }
    }
  }
  if (failed) atomicOr(a.err, tc::kErrTimeout);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, kAcc * kN);
}

// fp8 index queries of the nodes: head row r of iq (64 a node) as codes and, folded with the query's scale and the 1/128
// of the unnormalised rotation, its weight.  A warp a row.
__global__ void __launch_bounds__(256) k_tree_quant_iq(const __nv_bfloat16* __restrict__ iq,
                                                       const __nv_bfloat16* __restrict__ iw, int n,
                                                       uint8_t* __restrict__ q8, float* __restrict__ w8) {
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= n) return;
  const uint2 raw = *reinterpret_cast<const uint2*>(iq + (size_t)r * 128 + 4 * lane);
  const float2 x0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
  const float2 x1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
  float u[4] = {x0.x, x0.y, x1.x, x1.y}, scale;
  const uint32_t packed = fp8_rotate_quantize(u, lane, &scale);
  *reinterpret_cast<uint32_t*>(q8 + (size_t)r * 128 + 4 * lane) = packed;
  if (lane == 0) w8[r] = __bfloat162float(iw[r]) * (scale * 0.0078125f);
}

}  // namespace

// (a tile's row in the key map is a 32-bit coordinate)
bool tc_tree_scores_supported(const Dims& L, int B, int cap) {
  return L.dtype == CSA_BF16 && L.Hi == 64 && L.Di == 128 && (long long)B * cap < INT32_MAX - kRows;
}

size_t tree_scores_ws(const Dims& L, int B, int T) {
  return L.ikey_fp8 ? (size_t)B * T * 64 * (128 + sizeof(float)) : 0;  // the queries' codes, the folded weights
}

cudaError_t launch_tc_tree_scores(const Dims& L, const void* iq, const void* iw, int B, int T, const int32_t* parent,
                                  const void* ikeys, int cap, const void* rows, const int32_t* n_rows,
                                  const int32_t* pos, float* scores, void* ws, int32_t* err, cudaStream_t s) {
  int sms = 0, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  TsArgs a{};
  a.iw = static_cast<const __nv_bfloat16*>(iw);
  a.parent = parent; a.pos = pos; a.n_rows = n_rows;
  a.wscale = (float)(1.0 / sqrt((double)L.Di * (double)L.Hi));
  a.B = B; a.T = T; a.cap = cap; a.ratio = L.ratio; a.groups = (T + kG - 1) / kG;
  a.scores = scores; a.err = err;
  const long long most = (long long)B * a.groups * ((cap + kRows - 1) / kRows + 1);
  const dim3 grid((unsigned)(most < sms ? most : sms));
  const uint64_t heads = (uint64_t)B * T * 64;
  CUtensorMap tk, tr, tq;
  if (L.ikey_fp8) {
    auto* q8 = static_cast<uint8_t*>(ws);
    auto* w8 = reinterpret_cast<float*>(q8 + heads * 128);
    a.w8 = w8;
    CUtensorMap tks, trs;
    constexpr int row = kFp8RowBytes;
    if (!make_tmap_2d_u8(&tk, ikeys, (uint64_t)B * cap, row, row, 128, kRows, true) ||
        !make_tmap_2d_u8(&tks, ikeys, (uint64_t)B * cap, row, row, 16, kRows, false) ||
        !make_tmap_2d_u8(&tr, rows, (uint64_t)B * T, row, row, 128, kRows, true) ||
        !make_tmap_2d_u8(&trs, rows, (uint64_t)B * T, row, row, 16, kRows, false) ||
        !make_tmap_2d_u8(&tq, q8, heads, 128, 128, 128, kN, true))
      return cudaErrorInvalidValue;
    CSA_LAUNCH(k_tree_quant_iq, dim3((unsigned)((heads + 7) / 8)), dim3(256), 0, s,
               static_cast<const __nv_bfloat16*>(iq), a.iw, (int)heads, q8, w8);
    allow_smem<TsCfg<true>::kSmem>(k_tc_tree_scores<true>);
    CSA_LAUNCH(k_tc_tree_scores<true>, grid, dim3(TsCfg<true>::kThreads), TsCfg<true>::kSmem, s, tk, tr, tq, tks, trs,
               a);
    return cudaGetLastError();
  }
  if (!make_tmap_2d_bf16(&tk, ikeys, (uint64_t)B * cap, 128, 256, kRows) ||
      !make_tmap_2d_bf16(&tr, rows, (uint64_t)B * T, 128, 256, kRows) ||
      !make_tmap_2d_bf16(&tq, iq, heads, 128, 256, kN))
    return cudaErrorInvalidValue;
  allow_smem<TsCfg<false>::kSmem>(k_tc_tree_scores<false>);
  CSA_LAUNCH(k_tc_tree_scores<false>, grid, dim3(TsCfg<false>::kThreads), TsCfg<false>::kSmem, s, tk, tr, tq, tk, tr,
             a);
  return cudaGetLastError();
}

}  // namespace csa
