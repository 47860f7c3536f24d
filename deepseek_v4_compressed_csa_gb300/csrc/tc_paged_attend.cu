// Attention over a cache in pages and 8 bits on the 5th-generation tensor cores, for the Flash shapes (64 heads over one
// 512-dim latent, bf16 queries and outputs).
//
//   S = Q K^T, P = softmax, O = P V, K = V = the codes (a row's scale enters with its column of S and of P).
//
// What bounds it: a key is 512 bytes and 4 x 64 x 512 operations, 256 a byte, so the memory's rate asks for nearly the
// whole bf16 rate of the tensor cores, and turning codes into bf16 on the way for more than the rest of the SM has.  So
// the codes go to the tensor cores as they are (kind::f8f6f4, twice the bf16 rate), and what meets them is split in two
// 8-bit parts:
//   q = 2^e (hi + lo / 16), E4M3 both: the 8 bits of a bf16 value, exact but for values 2^-13 below the head's largest.
//     The parts are two rows of one operand, M = 128 = 64 heads x 2, kept in tensor memory (its 128 columns are an A
//     operand that no product reads from shared memory);
//   P = hi + lo, E5M2 and E4M3, both added to the same accumulator: a weight p ks is off by at most 2^-8 of itself, or where
//     that is more by 2^-15 of the largest, up to 1/8 of itself (from 2^-13 of the largest on E5M2's 3 bits are all there are;
//     below 2^-20 its smallest step).  (Two E4M3 parts keep 8 bits but drop everything below 2^-16 of the largest.)  Thousands
//     of small weights that are alike (rows that repeat) would all be rounded to one side: 16K of 1.125 x 2^-14 of one dominant
//     key's weight counted for 11 % more or less than they weigh.  So a thread keeps account of what its keys have lost or
//     gained; where that passes 2^-9 of their weights and of the largest, it rounds by thresholds spread evenly over its 32
//     keys instead of to the nearest: one weight may then be off by a quarter, alike ones together by 2^-8.
// A tile is 64 keys, one 32 KB stage of six, read once from memory, used K-major for S and MN-major (as V^T) for O:
//   S [128 x 64] = [Q_hi | Q_lo] K^T, 16 products of K = 32 (two buffers);
//   O^T [128 dims x 64 heads] x 4 += V^T P^T, 16 products (2 parts x 2 steps x 4): O^T takes 256 columns where O, with its
//     64 rows, would take all 512 and half the rate.
// Row order of S: 32-lane quarter w holds heads 16 w .. 16 w + 15, hi parts in its lanes 0-15, lo parts in 16-31, so that a
// head's parts meet by one shuffle; after it the lane pair shares the head's 64 keys, 32 each.
//
// Softmax with the scales: t = scale2 S ks, m a running maximum, l = sum 2^{t - m}.  What enters the product is
// 2^t ks 2^{7.9 - R}, R a reference that follows the maximum of log2(2^t |ks|) in steps: below 2^12, where lo, up to 2^8,
// still fits E4M3.  It starts 4 times above the first tile's maximum, and O^T is rescaled only when some head's maximum
// has passed its R by 4 (powers of two); every head's R then follows.  A tile takes its four warps some 2600 clocks, most
// of them latency, and the products' pipe 1300: two groups of four take tiles in turn, each with an m and l of its own; R
// is one, so each tile's decision about it waits for the tile's before.
//
// Measured: 8 queries of 65.7K rows (272 MB) 58 us before the merge, 4.7 TB/s, 1700 clocks a tile, where shared memory moves
// 176 KB of it at 128 bytes a clock (the keys once in and three times out, P, the scores' scales).  Feeding the products
// faster changes nothing.  Short calls are the chain plan - queries - tile - output: one window of three tiles 11.8 us.  The
// account of what rounding loses costs 1 to 3 % of a call, a decision by the account of the tile before just as much.
#include "paged.cuh"
#include "tc.cuh"

namespace csa {

namespace {

constexpr int kD = 512, kH = 64, kR = 64;
constexpr int kTile = 64;                     // keys a tile
constexpr int kStages = 6;
constexpr int kBox = kTile * 128;             // 128 dims x 64 keys (8 KB)
constexpr int kStage = 4 * kBox;
constexpr int kPBuf = kH * 128;               // a head's row: 64 hi codes, 64 lo codes (8 KB)
constexpr int kLoaders = 3;                   // (twelve warps in all: 168 registers a thread)
constexpr int kMmaWarp = kLoaders;
constexpr int kGroup = 128;                   // softmax threads of a tile (four warps, one a TMEM lane quarter)
constexpr int kSoft = 2 * kGroup;
constexpr int kThreads = 32 * (kLoaders + 1) + kSoft;
constexpr int kColO = 0, kColS = 256, kColQ = 384, kCols = 512;
constexpr float kGain = 7.9f;                 // R stands for 2^7.9 in the product
constexpr float kLost = 1.f / 512;            // what the weights may lose to rounding
constexpr float kTop = 14.f;                  // a fourth (two groups, two lanes a head) of the least that the largest one is, 2^5.9
constexpr float kStep = 4.f;                  // how far a maximum may pass R
constexpr float kHead = 2.f;                  // how far R is set above the first tile's maximum: most grow a little

constexpr int kOffP = kStages * kStage;
constexpr int kOffScale = kOffP + 2 * kPBuf;              // [kStages][64]
constexpr int kOffMask = kOffScale + kStages * kTile * 4; // [kStages] u64
constexpr int kOffFac = kOffMask + kStages * 8 + 16;      // [2][64] factors of a group's rescale
constexpr int kOffRef = kOffFac + 2 * kH * 4;             // [64] R
constexpr int kOffStat = kOffRef + kH * 4;                // [2][64] float2 (m, l) of the groups
constexpr int kOffTop = kOffStat + 2 * kH * 8;            // [2][64] the first two tiles' maxima
constexpr int kOffOut = kOffTop + 2 * kH * 4;             // [64] factors of the output
constexpr int kOffMax = kOffOut + kH * 4;                 // [2][64] largest magnitudes of the query rows' halves
constexpr int kOffRope = kOffMax + 2 * kH * 4;            // cos[32], sin[32]
constexpr int kOffBars = kOffRope + 64 * 4;
constexpr int kOffTmem = kOffBars + 32 * 8;
constexpr int kOffPlan = kOffTmem + 32;                   // PagedRun, scratch of the plan
constexpr int kSmem = kOffPlan + (int)sizeof(PagedRun) + 4 * kPlanInts + 1024;
static_assert(kOffBars % 8 == 0 && kOffFac % 16 == 0 && kOffOut % 16 == 0 && kOffPlan % 16 == 0 && sizeof(PagedRun) % 16 == 0 && kSmem <= 232448, "shared memory");

// 2^x by the hardware approximation (relative error ~2^-22; results below 2^-126 flush to zero)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Key e of a softmax thread's 32 rounds up what is at least (4 + 8 i) / 256 of a step above a code, i = 0 .. 31 once each,
// neighbours far apart (the bits of e reversed): what is added before the lower 8 bits go.
__host__ __device__ constexpr int spread(int e) {
  return 4 + 8 * ((e & 1) << 4 | (e & 2) << 2 | (e & 4) | (e & 8) >> 2 | (e & 16) >> 4);
}
// The same as a shift of lo by (spread - 127.5) / 256 of its smallest step, 2^-9: (2 spread - 255) 2^-18, the bits of an fp16
__host__ __device__ constexpr uint32_t spread_lo(int e) {
  const int n = 64 * (2 * spread(e) - 255), mag = n < 0 ? -n : n;  // in 2^-24
  int s = 0;
  while (mag >> s >= 2048) ++s;
  return (n < 0 ? 0x8000u : 0u) + (mag < 1024 ? (uint32_t)mag : (uint32_t)(((s + 1) << 10) + (mag >> s) - 1024));
}
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t bits_of(const __half2& h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Four weights, of keys e .. e + 3 of the thread, below 2^12, as E5M2 and E4M3 codes (the first key in the low byte).  In pairs
// of fp16 (11 bits of a weight): hi is its upper byte, lo what the rest rounds to.  To the nearest, or (kSpread) by the spread
// thresholds: lo takes them from 2^-7 on; smaller weights leave lo nothing, and hi takes them.  lost: what the codes are short
// of; mass: the weights / 64 (a sum of 16 fits fp16).  (A NaN is no code of hi's any more, but stays one in lo.)
template <bool kSpread>
__device__ __forceinline__ void split_weights(float v0, float v1, float v2, float v3, int e, uint32_t* hi, uint32_t* lo,
                                              __half2* lost, __half2* mass) {
  uint32_t up[2], rest[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h = i ? __floats2half2_rn(v2, v3) : __floats2half2_rn(v0, v1);
    uint32_t add = 0x00800080u, shift = 0u;
    if (kSpread) {
      const uint32_t small = __hlt2_mask(__habs2(h), as_half2(0x20002000u));  // 2^-7
      add = (small & (uint32_t)(spread(e + 2 * i) | spread(e + 2 * i + 1) << 16)) | (~small & add);
      shift = ~small & (spread_lo(e + 2 * i) | spread_lo(e + 2 * i + 1) << 16);
    }
    up[i] = bits_of(h) + add;
    const __half2 rem = __hsub2(h, as_half2(up[i] & 0xff00ff00u));  // (exact)
    rest[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(kSpread ? __hadd2(rem, as_half2(shift)) : rem), __NV_SATFINITE, __NV_E4M3);
    const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)rest[i], __NV_E4M3);
    *lost = __hadd2(*lost, __hsub2(rem, __half2(back)));
    *mass = __hfma2(__habs2(h), as_half2(0x24002400u), *mass);  // 2^-6
  }
  *hi = __byte_perm(up[0], up[1], 0x7531);
  *lo = rest[0] | rest[1] << 16;
}
// The 32 weights s * gain of a thread into its row of P: (lost, mass)
template <bool kSpread>
__device__ __forceinline__ float2 store_weights(const float* s, float gain, uint8_t* row, int plane, int h) {
  __half2 lost = as_half2(0u), mass = as_half2(0u);
#pragma unroll
  for (int c2 = 0; c2 < 2; ++c2) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float* v = s + 16 * c2 + 4 * e;
      split_weights<kSpread>(v[0] * gain, v[1] * gain, v[2] * gain, v[3] * gain, 16 * c2 + 4 * e, hi + e, lo + e, &lost, &mass);
    }
    *reinterpret_cast<uint4*>(row + (((2 * plane + c2) ^ (h & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(row + (((4 + 2 * plane + c2) ^ (h & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  const float2 a = __half22float2(lost), b = __half22float2(mass);
  return make_float2(a.x + a.y, 64.f * (b.x + b.y));
}

// Run x of a query: its first logical row, the rows [lo, hi) of its section that count, and the table.
struct Run {
  int start, lo, hi;
  bool rows;  // of compressed rows
};
__device__ __forceinline__ Run run_of(const PagedQuery& k, const TileCut& c, int x, int shift) {
  Run r;
  r.rows = x < c.runs0;
  if (x < c.runs0) {
    r.start = x << shift; r.lo = 0; r.hi = k.n0;
  } else if (x < c.runs0 + c.runs1) {
    r.start = (x - c.runs0) << shift; r.lo = 0; r.hi = k.f;
  } else if (x < c.runs0 + c.runs1 + c.runs2) {
    r.start = (c.w_run + x - c.runs0 - c.runs1) << shift; r.lo = k.w0; r.hi = k.w0 + k.nw;
  } else {
    r.start = r.lo = r.hi = 0;  // behind the last run
  }
  return r;
}

struct Smem {
  uint8_t* base;
  uint64_t *full, *empty, *s_full, *s_free, *p_full, *pv_done, *decided, *q_ready, *drain;
  volatile int* dead;
};

// A bounded wait; a block in which one has run out (dead) waits no more.
__device__ __forceinline__ bool wait(const Smem& sm, uint64_t* bar, uint32_t parity) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  if (*sm.dead) return false;
  if (tc::mbar_wait(bar, parity)) return true;
  *sm.dead = 1;
  return false;
}
// The same with one answer for the warp
__device__ __forceinline__ bool warp_wait(const Smem& sm, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(sm, bar, parity));
}

__global__ void __launch_bounds__(kThreads, 1)
    k_tc_attend_pages(const __grid_constant__ CUtensorMap tm_runs, const __grid_constant__ PagedArgs a) {
  if (a.merge) pdl_trigger();  // (what follows otherwise finds the outputs written)
  extern __shared__ uint8_t smem_raw[];
  Smem sm;
  sm.base = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);  // (by an offset: the accesses stay shared-memory ones)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm.base + kOffBars);
  sm.full = bars;
  sm.empty = bars + kStages;
  sm.s_full = bars + 2 * kStages;
  sm.s_free = sm.s_full + 2;
  sm.p_full = sm.s_free + 2;
  sm.pv_done = sm.p_full + 2;
  sm.decided = sm.pv_done + 2;
  sm.q_ready = sm.decided + 2;
  sm.drain = sm.q_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm.base + kOffTmem);
  sm.dead = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = sm.dead + 1;  // a loader's last tile whose copies it has issued, + 1
  float* scales = reinterpret_cast<float*>(sm.base + kOffScale);
  volatile uint64_t* masks = reinterpret_cast<volatile uint64_t*>(sm.base + kOffMask);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tc::tma_prefetch(&tm_runs);
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(sm.full + i, 1 + 32);  // the copies, and the loader's lanes for the scales (or all they copy)
      tc::mbar_init(sm.empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(sm.s_full + i, 1);
      tc::mbar_init(sm.s_free + i, kGroup);
      tc::mbar_init(sm.p_full + i, kGroup);
      tc::mbar_init(sm.pv_done + i, 1);
      tc::mbar_init(sm.decided + i, kGroup);
    }
    tc::mbar_init(sm.q_ready, kSoft);
    tc::mbar_init(sm.drain, 1);
    *sm.dead = 0;
    for (int i = 0; i < kLoaders; ++i) issued[i] = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();  // predecessors complete: what they wrote is visible and their tensor memory is free
  // (small inputs that the softmax warps need later, before the keys that every SM fetches stand in their way)
  const bool soft = warp > kMmaWarp;
  const float freq = soft && a.inv_freq ? __ldg(a.inv_freq + lane) : 0.f;
  const float z2 = soft && a.sink ? __ldg(a.sink + 16 * (warp & 3) + (lane & 15)) * 1.4426950408889634f : -INFINITY;
  if (warp == kMmaWarp) {  // (while the plan is made, whose barrier stands behind this)
    tc::tmem_alloc(tmem_slot, kCols);
    tc::tmem_relinquish();
  }
  PagedRun* plan = reinterpret_cast<PagedRun*>(sm.base + kOffPlan);
  tc::fence_before_sync();
  paged_plan<kThreads / 32>(a, plan, reinterpret_cast<int*>(plan + 1));
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int t0 = plan->t0, t1 = plan->t1;
  if (t0 >= t1) {  // (all of the block)
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kCols);
    return;
  }
  const int pre0 = plan->pre;
  const PagedQuery k0 = plan->k;

  if (warp < kLoaders) {
    // ------------------------------------------------------------ loaders: warp w takes the tiles j with j % 3 == w
    // Dense runs come by one copy each 128 dims; selected rows by a warp's 512-byte cp.async each (tile::gather4 takes a
    // warp some 75 clocks per 512 bytes: 4.8K a tile, against 1K), which are waited for before the warp's next tile.
    int pre = pre0, j = 0;  // j: tiles of this block before the query
    const int shift = a.shift, per = kTile >> shift, copies = 4 * per;
    PagedQuery k = k0;
    bool ok = true;
    int pending = -1;  // stage of selected rows on their way
    auto landed = [&] {
      if (pending < 0) return;
      tc::cp_async_wait_all();
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(sm.full + pending);
      if (lane == 0) tc::mbar_arrive(sm.full + pending);  // (in place of the copies' own arrival)
      pending = -1;
    };
#pragma unroll 1
    while (true) {
      const TileCut cut = cut_tiles(a.sel != nullptr, k, kTile, shift);
      const int begin = max(t0 - pre, 0), end = min(t1 - pre, k.tiles);
      const int32_t* sel = a.sel + (size_t)k.q * a.topk;
      const int32_t* rows_b = a.row_table + (size_t)k.b * a.row_pages;
      const int32_t* tokens_b = a.token_table + (size_t)k.b * a.token_pages;
      // The lookups run ahead: a tile's selected rows two of the warp's tiles before its copies are issued, its pages one
      // before.  Each is loaded into the registers of the tile's before, dead by then: a move would wait for the load.
      auto selected = [&](int t, int e) -> int {  // key lane + 32 e of tile t: its row, -1 behind the last
        const int x = t * kTile + lane + 32 * e;
        return t < end && t < cut.sel_tiles && x < k.n0 ? (int)tc::ld_nc_u32_now(sel + x) : -1;
      };
      // a tile's pages as the table has them: selected, of both keys; dense, of the lane's run
      auto pages_of = [&](int t, int j0, int j1, int& p0, int& p1) {
        p0 = p1 = -1;
        if (t >= end) return;
        if (t < cut.sel_tiles) {
          if ((unsigned)j0 < (unsigned)k.n_rows) p0 = (int)tc::ld_nc_u32_now(rows_b + page_of(a, j0));
          if ((unsigned)j1 < (unsigned)k.n_rows) p1 = (int)tc::ld_nc_u32_now(rows_b + page_of(a, j1));
        } else if (lane < per) {
          const Run r = run_of(k, cut, (t - cut.sel_tiles) * per + lane, shift);
          if (r.hi > r.lo) p0 = (int)tc::ld_nc_u32_now((r.rows ? rows_b : tokens_b) + page_of(a, r.start));
        }
      };
      int t = begin + (warp + kLoaders - j % kLoaders) % kLoaders;
      int j0 = selected(t, 0), j1 = selected(t, 1), n0 = selected(t + kLoaders, 0), n1 = selected(t + kLoaders, 1), p0, p1;
      pages_of(t, j0, j1, p0, p1);
#pragma unroll 1
      for (; t < end; t += kLoaders) {
        const int jt = j + t - begin, st = jt % kStages;
        const bool is_sel = t < cut.sel_tiles;
        int r0, r1;        // physical rows of keys lane and lane + 32, -1 for none
        int run_row = -1;  // dense: the first physical row of the lane's run, -1 for none
        if (is_sel) {
          const int x = t * kTile + lane;
          r0 = (unsigned)p0 < (unsigned)a.n_pages ? p0 * a.P + (j0 - page_of(a, j0) * a.P) : -1;
          r1 = (unsigned)p1 < (unsigned)a.n_pages ? p1 * a.P + (j1 - page_of(a, j1) * a.P) : -1;
          if ((x < k.n0 && r0 < 0) || (x + 32 < k.n0 && r1 < 0)) atomicOr(a.err, CSA_DEV_RANGE);
        } else {
          int span = 0;  // the run's rows [lo, hi) that count, 8 bits each
          if (lane < per) {
            const Run r = run_of(k, cut, (t - cut.sel_tiles) * per + lane, shift);
            if (r.hi > r.lo) {
              if ((unsigned)p0 < (unsigned)a.n_pages) {
                run_row = p0 * a.P + (r.start - page_of(a, r.start) * a.P);
                span = max(r.lo - r.start, 0) | min(r.hi - r.start, kTile) << 8;
              } else {
                atomicOr(a.err, CSA_DEV_RANGE);
              }
            }
          }
          int rr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = lane + 32 * e, from = key >> shift, off = key & ((1 << shift) - 1);
            const int row = __shfl_sync(0xffffffffu, run_row, from), sp = __shfl_sync(0xffffffffu, span, from);
            rr[e] = off >= (sp & 255) && off < sp >> 8 ? row + off : -1;
          }
          r0 = rr[0];
          r1 = rr[1];
        }
        j0 = n0;
        j1 = n1;
        pages_of(t + kLoaders, j0, j1, p0, p1);
        n0 = selected(t + 2 * kLoaders, 0);
        n1 = selected(t + 2 * kLoaders, 1);
        landed();
        ok = warp_wait(sm, sm.empty + st, ((jt / kStages) & 1) ^ 1);
        if (!ok) break;
        const uint32_t on0 = __ballot_sync(0xffffffffu, r0 >= 0), on1 = __ballot_sync(0xffffffffu, r1 >= 0);
        const uint32_t sdst = tc::smem_u32(scales + st * kTile + lane);
        if (lane == 0) {
          masks[st] = (uint64_t)on1 << 32 | on0;
          issued[warp] = jt + 1;
        }
        __syncwarp();
        if (!is_sel) {
          // copy x: run x / 4, dims 128 (x % 4) ..; a run in no page: rows behind the pool's end, which come as zeros
          if (lane == 0) tc::mbar_arrive_expect_tx(sm.full + st, kStage);
          __syncwarp();
          const int part = min(lane >> 2, per - 1), row = __shfl_sync(0xffffffffu, run_row, part);
          if (lane < copies)
            tc::tma_load_2d(sm.base + st * kStage + (lane & 3) * kBox + (part << shift) * 128, &tm_runs, sm.full + st,
                            (lane & 3) * 128, row >= 0 ? row : a.n_pages * a.P);
        }
        tc::cp_async4(sdst, a.scales + max(r0, 0), r0 >= 0 ? 4u : 0u);
        tc::cp_async4(sdst + 128, a.scales + max(r1, 0), r1 >= 0 ? 4u : 0u);
        if (!is_sel) {
          tc::cp_async_arrive(sm.full + st);
        } else {
          const uint32_t dst = tc::smem_u32(sm.base + st * kStage) + (lane >> 3) * kBox;
          const uint8_t* src = a.codes + lane * 16;
#pragma unroll 8
          for (int r = 0; r < kTile; ++r) {
            const int row = __shfl_sync(0xffffffffu, r < 32 ? r0 : r1, r & 31);
            tc::cp_async16(dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4), src + (size_t)max(row, 0) * kD, row >= 0 ? 16u : 0u);
          }
          pending = st;
        }
      }
      j += end - begin;
      pre += k.tiles;
      if (!ok || pre >= t1) break;
      k = next_query(a, k.q);
      // (the softmax warps want its 64 KB when they are done with the query before: 512 windows 49.5 -> 45.6 us)
      if (warp == 0 && lane == 0)
        tc::prefetch_l2(static_cast<const __nv_bfloat16*>(a.q) + (size_t)k.q * kH * kD, kH * kD * 2);
    }
    landed();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    // (one elected thread for all of it, stages and phases counted up, descriptors a base plus constants: what this thread
    // does between two products is time that the tensor pipe may stand still; issued by elections product by product, with
    // descriptors from the tile's number, they cost 70 clocks each, where the pipe takes 32 and 48)
    if (tc::elect_one()) {
      constexpr uint32_t id_qk = tc::idesc_e4m3(128, kTile);
      constexpr uint32_t id_hi = tc::idesc_e4m3(128, kH, true, true), id_lo = tc::idesc_e4m3(128, kH, true);
      const uint64_t kd = tc::sdesc_kmajor_sw128(tc::smem_u32(sm.base));
      const uint64_t vd = tc::sdesc_mnmajor_sw128(tc::smem_u32(sm.base), kBox, 1024);
      const uint64_t pd = tc::sdesc_kmajor_sw128(tc::smem_u32(sm.base + kOffP));
      int sq = 0, sp = 0, bq = 0, bp = 0;       // stages and buffers of the next scores and the next output
      uint32_t fq = 0, hq = 1, hp = 0, seg = 0; // phases: of full[sq], of s_free[bq], of p_full[bp]; of q_ready
      // S of the next tile, whose buffer's last scores the softmax warps have read
      auto qk = [&] {
        if (!wait(sm, sm.full + sq, fq) || !wait(sm, sm.s_free + bq, hq)) return false;
        tc::fence_after_sync();
        const uint64_t kb = kd + sq * (kStage >> 4);
        const uint32_t d = tmem + kColS + 64 * bq;
#pragma unroll
        for (int s = 0; s < 16; ++s)
          tc::mma_f8_ta(d, tmem + kColQ + 8 * s, kb + (((s >> 2) * kBox + (s & 3) * 32) >> 4), id_qk, s > 0);
        tc::mma_commit(sm.s_full + bq);
        if (++sq == kStages) { sq = 0; fq ^= 1; }
        if ((bq ^= 1) == 0) hq ^= 1;
        return true;
      };
      // O^T += of the next tile, whose probabilities they have written
      auto pv = [&](uint32_t add) {
        if (!wait(sm, sm.p_full + bp, hp)) return false;
        tc::fence_after_sync();
        const uint64_t va = vd + sp * (kStage >> 4), pa = pd + bp * (kPBuf >> 4);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int s = 0; s < 4; ++s)  // hi keys 0-31, 32-63, lo keys 0-31, 32-63
            tc::mma_f8(tmem + kColO + 64 * m, va + ((m * kBox + (s & 1) * 4096) >> 4), pa + (s * 32 >> 4),
                       s < 2 ? id_hi : id_lo, s > 0 ? 1u : add);
        tc::mma_commit(sm.empty + sp);
        tc::mma_commit(sm.pv_done + bp);
        if (++sp == kStages) sp = 0;
        if ((bp ^= 1) == 0) hp ^= 1;
        return true;
      };
      int pre = pre0;
      PagedQuery k = k0;
      bool ok = true;
#pragma unroll 1
      while (true) {
        const int n = min(t1 - pre, k.tiles) - max(t0 - pre, 0);
        ok = wait(sm, sm.q_ready, seg & 1);
        ++seg;
        // scores two tiles ahead of the outputs: they wait for keys and for a buffer that is free once its scores have been
        // read, so the softmax groups always find the next ones
        ok = ok && qk() && (n < 2 || qk());
#pragma unroll 1
        for (int i = 0; ok && i < n; ++i) {
          if (i + 2 < n) ok = qk();
          ok = ok && pv(i > 0);
        }
        pre += k.tiles;
        if (!ok || pre >= t1) break;
        k = next_query(a, k.q);
      }
      tc::mma_commit(sm.drain);  // every product retires before tensor memory is released
      if (!tc::mbar_wait(sm.drain, 0)) *sm.dead = 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax: group g takes the tiles j with j % 2 == g
    const int quad = warp & 3, plane = lane >> 4, h = 16 * quad + (lane & 15);
    const int g = warp >= kMmaWarp + 5, gt = tid - 32 * (kLoaders + 1) - g * kGroup;  // thread of the group
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    float* fac = reinterpret_cast<float*>(sm.base + kOffFac) + g * kH;
    float* refs = reinterpret_cast<float*>(sm.base + kOffRef);
    float2* stat = reinterpret_cast<float2*>(sm.base + kOffStat);
    float* top = reinterpret_cast<float*>(sm.base + kOffTop);
    float* fout = reinterpret_cast<float*>(sm.base + kOffOut);
    float* rcos = reinterpret_cast<float*>(sm.base + kOffRope);
    float* rsin = rcos + 32;
    uint8_t* pbuf = sm.base + kOffP + g * kPBuf;
    const uint32_t t_s = tmem + kColS + 64 * g + lanes;
    int pre = pre0, j = 0;
    PagedQuery k = k0;
#pragma unroll 1
    while (true) {
      const int begin = max(t0 - pre, 0), end = min(t1 - pre, k.tiles), n = end - begin;
      // ---- the query as two parts of 2^-e q into tensor memory, a group half of the dims: a thread has, of rows lane / 4
      // and lane / 4 + 8 of its quarter's 16 heads, every fourth eight values (every product that read the last query's
      // parts has retired)
      {
        const int r = lane >> 2;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)k.q * kH + 16 * quad + r) * kD + 256 * g + 8 * (lane & 3);
        uint4 v[2][8];  // (a line of memory a row and load: what the loads take is counted in lines, a clock each)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[0][e] = tc::ld_nc_v4_now(src + 32 * e);
          v[1][e] = tc::ld_nc_v4_now(src + 8 * kD + 32 * e);
        }
        uint32_t* amax = reinterpret_cast<uint32_t*>(sm.base + kOffMax);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          __nv_bfloat162 m4[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t w[4] = {v[x][e].x, v[x][e].y, v[x][e].z, v[x][e].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 u = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
              m4[i] = e == 0 ? u : __hmax2_nan(m4[i], u);
            }
          }
          const __nv_bfloat162 m2 = __hmax2_nan(__hmax2_nan(m4[0], m4[1]), __hmax2_nan(m4[2], m4[3]));
          uint32_t mx = *reinterpret_cast<const uint32_t*>(&m2) & 0x7fff7fffu;
          mx = max(mx & 0xffffu, mx >> 16);  // (the bits of magnitudes are ordered as they are, a NaN's above all)
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          if ((lane & 3) == 0) amax[g * kH + 16 * quad + r + 8 * x] = mx;
        }
        tc::named_bar(4, kSoft);
        // 2^-e with e = exponent - 7: values below 2^8, exact products; a row of denormals, or zeros, stays small; a row that
        // holds an infinity or a NaN becomes NaN (by its product with 0, and its scores by their factor)
        auto expo = [&](int hh) { return max((int)(max(amax[hh], amax[kH + hh]) >> 7), 12); };
        __nv_bfloat162 inv[2], inv16[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int be = expo(16 * quad + r + 8 * x);
          inv[x] = __float2bfloat162_rn(be == 255 ? 0.f : __uint_as_float((uint32_t)(261 - be) << 23));
          inv16[x] = __float2bfloat162_rn(be == 255 ? 0.f : __uint_as_float((uint32_t)(265 - be) << 23));
        }
        // hi: the value cut to the four digits that E4M3 has, lo: the four behind them, both exact, as are the products with
        // powers of two, so bf16 pairs do.  (hi below E4M3's normal numbers, 2^-13 of the head's largest, is rounded, by at
        // most 2^-17 of that.  With lo from what hi became, converted back, it would be 2^-21, and 3K clocks instead of 2K.)
        auto parts = [&](int x, uint32_t u0, uint32_t u1, uint32_t* hi, uint32_t* lo) {
          float h[4], l[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = i ? u1 : u0, m = w & 0xfff0fff0u;
            const __nv_bfloat162 wv = *reinterpret_cast<const __nv_bfloat162*>(&w), mv = *reinterpret_cast<const __nv_bfloat162*>(&m);
            const __nv_bfloat162 a2 = __hmul2(mv, inv[x]), b2 = __hmul2(__hsub2(wv, mv), inv16[x]);
            const uint32_t aw = *reinterpret_cast<const uint32_t*>(&a2), bw = *reinterpret_cast<const uint32_t*>(&b2);
            h[2 * i] = __uint_as_float(aw << 16); h[2 * i + 1] = __uint_as_float(aw & 0xffff0000u);
            l[2 * i] = __uint_as_float(bw << 16); l[2 * i + 1] = __uint_as_float(bw);  // (what is behind its four digits rounds away)
          }
          *hi = e4m3x4(h[0], h[1], h[2], h[3]);
          *lo = e4m3x4(l[0], l[1], l[2], l[3]);
        };
        // (four rounds of the same code, the values moved up in between: unrolled, its 15 KB of instructions arrive behind
        // the keys that every SM is fetching: 9.5K clocks in the largest batch, 3K by itself)
#pragma unroll 1
        for (int round = 0; round < 4; ++round) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              parts(x, v[x][e].x, v[x][e].y, hi + 4 * e + 2 * x, lo + 4 * e + 2 * x);
              parts(x, v[x][e].z, v[x][e].w, hi + 4 * e + 2 * x + 1, lo + 4 * e + 2 * x + 1);
            }
#pragma unroll
            for (int e = 0; e < 6; ++e) v[x][e] = v[x][e + 2];
          }
          const uint32_t col = tmem + kColQ + 64 * g + 16 * round + lanes;
          tc::tmem_st_16x16(col, hi);
          tc::tmem_st_16x16(col + (16u << 16), lo);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(sm.q_ready);
        // what a product of the parts stands for: 2^e, and the softmax scale with it
        const int be_h = expo(h);
        const float c = be_h == 255 ? NAN : __uint_as_float((uint32_t)(be_h - 7) << 23) * a.scale2;
        const float c_own = plane ? c * 0.0625f : c, c_other = plane ? c : c * 0.0625f;
        float m = -INFINITY, l = 0.f;
        float lost = 0.f, mass = 0.f;  // what this thread's keys have lost to rounding, and their weights, relative to 2^m
        const int first = (j & 1) == g ? 0 : 1;  // this group's first tile of the query
#pragma unroll 1
        for (int i = first; i < n; i += 2) {
          const int jt = j + i, st = jt % kStages;
          wait(sm, sm.full + st, (jt / kStages) & 1);
          wait(sm, sm.s_full + g, (jt >> 1) & 1);
          tc::fence_after_sync();
          float s[32];
          {
            uint32_t x[64];
            tc::tmem_ld32(t_s, x);
            tc::tmem_ld32(t_s + 32, x + 32);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            tc::mbar_arrive(sm.s_free + g);
            // hi part lanes keep keys 0-31 and send 32-63, lo part lanes the other way round
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t send = plane ? x[e] : x[e + 32], keep = plane ? x[e + 32] : x[e];
              const float got = __uint_as_float(__shfl_xor_sync(0xffffffffu, send, 16));
              s[e] = fmaf(got, c_other, __uint_as_float(keep) * c_own);
            }
          }
          const uint64_t mask64 = masks[st];
          const float* ks = scales + st * kTile + 32 * plane;
          float mt = -INFINITY;
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 k4 = reinterpret_cast<const float4*>(ks)[e4];
            s[4 * e4] *= k4.x; s[4 * e4 + 1] *= k4.y; s[4 * e4 + 2] *= k4.z; s[4 * e4 + 3] *= k4.w;
          }
          if (mask64 != ~0ull) {
            const uint32_t on = (uint32_t)(mask64 >> (32 * plane));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(on >> e & 1u)) s[e] = -INFINITY;
            // rows that are no keys hold whatever their page does: zeros, before the product would meet a NaN among them
            uint8_t* z = sm.base + st * kStage + ((gt & 31) >> 3) * kBox + (gt & 7) * 16;  // a warp a row
#pragma unroll 4
            for (int r = gt >> 5; r < kTile; r += 4)
              if (!((uint32_t)(mask64 >> (r & 32)) >> (r & 31) & 1u)) *reinterpret_cast<uint4*>(z + r * 128) = make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) mt = fmaxf(mt, s[e]);
          mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
          const float mn = fmaxf(m, mt), mr = mn == -INFINITY ? 0.f : mn;
          const float keep = ex2(m - mr);
          l *= keep;
          lost *= keep;
          mass *= keep;
          m = mn;
          float vt = 0.f, l2 = 0.f;
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 k4 = reinterpret_cast<const float4*>(ks)[e4];
            const float p0 = ex2(s[4 * e4] - mr), p1 = ex2(s[4 * e4 + 1] - mr), p2 = ex2(s[4 * e4 + 2] - mr),
                        p3 = ex2(s[4 * e4 + 3] - mr);
            l += p0 + p1;
            l2 += p2 + p3;
            // (a key that does not count has scale 0)
            s[4 * e4] = p0 * k4.x; s[4 * e4 + 1] = p1 * k4.y; s[4 * e4 + 2] = p2 * k4.z; s[4 * e4 + 3] = p3 * k4.w;
            vt = fmaxf(fmaxf(vt, fmaxf(fabsf(s[4 * e4]), fabsf(s[4 * e4 + 1]))), fmaxf(fabsf(s[4 * e4 + 2]), fabsf(s[4 * e4 + 3])));
          }
          l += l2;
          vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 16));
          // ---- the reference follows log2 of the largest 2^t ks: the first two tiles find it together, later ones after
          // the tile before has decided
          // (at least 2^-115 of the probabilities: the gain stays finite, and smaller scales lose digits)
          const float lv = vt > 0.f ? mr + fmaxf(lg2(vt), -115.f) : -INFINITY;
          float ref;
          if (i < 2 && n > 1) {
            if (plane == 0) top[i * kH + h] = lv;
            tc::named_bar(4, kSoft);
            ref = fmaxf(top[h], top[kH + h]) + kHead;
          } else if (i == 0) {
            ref = lv + kHead;
          } else {
            wait(sm, sm.decided + (g ^ 1), ((jt - 1) >> 1) & 1);
            ref = refs[h];
          }
          if (i < 2) {
            if (i == 0 && plane == 0) refs[h] = ref;
          } else if (tc::named_bar_any(2 + g, kGroup, lv > ref + kStep)) {
            const float up = fmaxf(ref, lv);
            // (a head of which nothing but zeros has entered the product needs no factor)
            if (plane == 0) fac[h] = ref == -INFINITY ? 1.f : ex2(ref - up);
            ref = up;
            wait(sm, sm.pv_done + (g ^ 1), ((jt - 1) >> 1) & 1);
            tc::fence_after_sync();
            tc::named_bar(2 + g, kGroup);  // (every thread has read its R)
            if (plane == 0) refs[h] = up;
#pragma unroll 1
            for (int c8 = 0; c8 < 8; ++c8) {
              uint32_t x[32];
              tc::tmem_ld32(tmem + kColO + 32 * c8 + lanes, x);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e4 = 0; e4 < 8; ++e4) {
                const float4 f4 = reinterpret_cast<const float4*>(fac + 32 * (c8 & 1))[e4];
                x[4 * e4] = __float_as_uint(__uint_as_float(x[4 * e4]) * f4.x);
                x[4 * e4 + 1] = __float_as_uint(__uint_as_float(x[4 * e4 + 1]) * f4.y);
                x[4 * e4 + 2] = __float_as_uint(__uint_as_float(x[4 * e4 + 2]) * f4.z);
                x[4 * e4 + 3] = __float_as_uint(__uint_as_float(x[4 * e4 + 3]) * f4.w);
              }
              tc::tmem_st32(tmem + kColO + 32 * c8 + lanes, x);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
          }
          tc::mbar_arrive(sm.decided + g);
          // (nothing in this tile weighs anything: lv does not bound mr - ref then, and a gain out of range would make the
          // zeros NaN; a NaN stays one beside a gain of 0)
          const float gain = lv == -INFINITY ? 0.f : ex2(kGain + mr - ref);
          // ---- the probabilities' two parts, once the buffer's last product has retired
          if (jt >= 2) wait(sm, sm.pv_done + g, ((jt >> 1) & 1) ^ 1);
          uint8_t* row = pbuf + h * 128;
          const float unit = ex2(fminf(ref - kGain - mr, 120.f));  // 1 / gain
          float2 w = store_weights<false>(s, gain, row, plane, h);
          mass = fmaf(w.y, unit, mass);
          if (fabsf(fmaf(w.x, unit, lost)) > fmaf(mass, kLost, kTop * kLost * unit)) w = store_weights<true>(s, gain, row, plane, h);
          lost = fmaf(w.x, unit, lost);
          tc::fence_proxy_async_smem();
          tc::fence_before_sync();
          tc::mbar_arrive(sm.p_full + g);
        }
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (plane == 0) stat[g * kH + h] = make_float2(m, l);
      }
      j += n;
      // (the group that has not the last tile: it waits for the other one; earlier, its instructions arrive behind the keys)
      if ((j & 1) == g && gt < 32 && a.inv_freq) turn_cs(k.p, freq, rcos + gt, rsin + gt);
      // ---- the run's part of this query, or its output
      const bool whole = begin == 0 && end == k.tiles;
      const size_t slot = 2 * blockIdx.x + (begin == 0 ? 1 : 0);
      tc::named_bar(4, kSoft);  // (both groups' statistics, the last R, the angles)
      if (begin == 0 && !whole && g == 1 && gt < kR / 2 && a.inv_freq)
        a.turns[blockIdx.x * (kR / 2) + gt] = make_float2(rcos[gt], rsin[gt]);
      if (g == 0 && plane == 0) {
        const float2 s0 = stat[h], s1 = stat[kH + h];
        const float m = fmaxf(s0.x, s1.x), mr = m == -INFINITY ? 0.f : m, ref = refs[h];
        const float l = fmaf(s0.y, ex2(s0.x - mr), s1.y * ex2(s1.x - mr));
        // O^T * f = sum 2^{t - m} key.  (f as a square: where the largest weight is below 2^-117 of 2^m, a row of scale 0, f is
        // below the normal numbers, which ex2 flushes and a product does not.)
        const float root = ref == -INFINITY ? 0.f : ex2(0.5f * (ref - kGain - mr));
        float f = root * root;
        if (whole) {
          const float M = fmaxf(m, z2), gm = m == -INFINITY ? 0.f : ex2(m - M);
          const float Z = l * gm + (z2 == -INFINITY ? 0.f : ex2(z2 - M));
          f = Z == 0.f ? 0.f : f * (gm / Z);
        } else {
          a.ml[slot * kH + h] = make_float2(l == l ? m : l, l);  // (a NaN is one for the merge, too)
        }
        fout[h] = f;
      }
      wait(sm, sm.pv_done + ((j - 1) & 1), ((j - 1) >> 1) & 1);
      if (j >= 2) wait(sm, sm.pv_done + (j & 1), ((j - 2) >> 1) & 1);  // (the other buffer's, retired before)
      tc::fence_after_sync();
      tc::named_bar(4, kSoft);
      // 32 heads of the warp's 32 dims a step, a lane a dim, from tensor memory to where they go: a part's 128 bytes a head in
      // one store, of an output's two heads 64 bytes each, their pairs of dims put together by one shuffle.  (Through shared
      // memory, turned by stmatrix, and from there by copies of boxes, it took 5.4K clocks; so it takes 2K.)
      const bool odd = lane & 1;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        const int blk = 2 * g + (c >> 1), h0 = 32 * (c & 1);
        uint32_t x[32];
        tc::tmem_ld32(tmem + kColO + 64 * blk + h0 + lanes, x);
        tc::tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int e4 = 0; e4 < 8; ++e4) {
          const float4 f4 = *reinterpret_cast<const float4*>(fout + h0 + 4 * e4);
          v[4 * e4] = __uint_as_float(x[4 * e4]) * f4.x;
          v[4 * e4 + 1] = __uint_as_float(x[4 * e4 + 1]) * f4.y;
          v[4 * e4 + 2] = __uint_as_float(x[4 * e4 + 2]) * f4.z;
          v[4 * e4 + 3] = __uint_as_float(x[4 * e4 + 3]) * f4.w;
        }
        if (!whole) {
          float* part = a.part + slot * kH * kD + (size_t)((blk * 4 + quad) * kH + h0) * 32 + lane;
#pragma unroll
          for (int e = 0; e < 32; ++e) part[32 * e] = v[e];
          continue;
        }
        if (blk == 3 && quad >= 2 && a.inv_freq) {  // the last 64 dims: the pair's other one is the next lane's
          const int ri = (32 * (quad - 2) + lane) >> 1;
          const float cs = rcos[ri], sn = odd ? -rsin[ri] : rsin[ri];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = fmaf(v[e], cs, __shfl_xor_sync(0xffffffffu, v[e], 1) * sn);
        }
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + ((size_t)k.q * kH + h0 + odd) * kD + 128 * blk + 32 * quad + (lane & ~1);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {  // even lanes take the first head of two, odd lanes the second
          const float got = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[e + 1], 1), keep = odd ? v[e + 1] : v[e];
          *reinterpret_cast<__nv_bfloat162*>(o + e * kD) = __floats2bfloat162_rn(odd ? got : keep, odd ? keep : got);
        }
      }
      tc::fence_before_sync();
      tc::named_bar(4, kSoft);  // (O^T and the statistics have been read)
      pre += k.tiles;
      if (pre >= t1) break;
      k = next_query(a, k.q);
    }
  }
  // ---- everything in flight has landed and retired before shared and tensor memory go
  tc::fence_before_sync();
  __syncthreads();
  if (*sm.dead) {
    if (tid == 0) {
      atomicOr(a.err, tc::kErrTimeout);
      for (int w = 0; w < kLoaders; ++w)
        for (int i = issued[w] - 1; i >= 0 && i > issued[w] - 1 - kStages; i -= kLoaders)
          tc::mbar_wait(sm.full + i % kStages, (i / kStages) & 1);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kCols);
}

}  // namespace

bool tc_paged_supported(const Dims& L, int P) {
  return L.dtype == CSA_BF16 && L.H == kH && L.D == kD && L.R == kR && P % 8 == 0;
}

cudaError_t launch_tc_paged(const PagedArgs& a, cudaStream_t s) {
  const uint64_t rows = (uint64_t)a.n_pages * a.P;
  CUtensorMap tm_runs;
  if (!make_tmap_2d_u8(&tm_runs, a.codes, rows, kD, kD, 128, 1u << a.shift, true)) return cudaErrorInvalidValue;
  allow_smem<kSmem>(k_tc_attend_pages);
  CSA_LAUNCH(k_tc_attend_pages, dim3(kPagedBlocks), dim3(kThreads), kSmem, s, tm_runs, a);
  return cudaGetLastError();
}

}  // namespace csa
