// Attention over a cache in pages and 8 bits on the 5th-generation tensor cores, for the Flash shapes (64 heads over one
// 512-dim latent, bf16 queries and outputs).
//
//   S = Q K^T, P = softmax, O = P V, K = V = the codes (a row's scale enters with its column of S and of P).
//
// What bounds it: a key is 512 bytes and 4 x 64 x 512 operations, 256 a byte, so the memory's rate asks for nearly the
// whole bf16 rate of the tensor cores, and turning codes into bf16 on the way for more than the rest of the SM has.  So
// the codes go to the tensor cores as they are (kind::f8f6f4, twice the bf16 rate), and what meets them is split in two
// E4M3 parts, which carry the 8 bits of a bf16 value:
//   q = 2^e (hi + lo / 16), exact but for values 2^-14 below the head's largest: the parts are two rows of one operand, M = 128 =
//     64 heads x 2, kept in tensor memory (its 128 columns are an A operand that no product reads from shared memory);
//   P = hi + lo, both added to the same accumulator.
// A tile is 64 keys, one 32 KB stage of six, read once from memory, used K-major for S and MN-major (as V^T) for O:
//   S [128 x 64] = [Q_hi | Q_lo] K^T, 16 products of K = 32 (two buffers);
//   O^T [128 dims x 64 heads] x 4 += V^T P^T, 16 products (2 parts x 2 steps x 4): O^T takes 256 columns where O, with its
//     64 rows, would take all 512 and half the rate.
// Row order of S: 32-lane quarter w holds heads 16 w .. 16 w + 15, hi parts in its lanes 0-15, lo parts in 16-31, so that a
// head's parts meet by one shuffle; after it the lane pair shares the head's 64 keys, 32 each.
//
// Softmax with the scales: t = scale2 S ks, m its running maximum, l = sum 2^{t - m}.  What enters the product is
// 2^t ks 2^{6 - R}, R a running reference of log2(2^t ks) that follows its maximum in steps: at most 2^8 (E4M3 holds
// 448), parts down to 2^-10 of that scale.  O^T is rescaled only when a head's maximum has passed R by 2 (powers of two).
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
constexpr int kLoaders = 4;                   // a warp per 128 dims
constexpr int kMmaWarp = kLoaders;
constexpr int kSoft = 128;                    // softmax threads (four warps, one a TMEM lane quarter)
constexpr int kThreads = 32 * (kLoaders + 1) + kSoft;
constexpr int kColO = 0, kColS = 256, kColQ = 384, kCols = 512;
constexpr float kGain = 6.f;                  // R stands for 2^6 in the product
constexpr float kStep = 2.f;                  // how far a maximum may pass R

constexpr int kOffP = kStages * kStage;
constexpr int kOffScale = kOffP + 2 * kPBuf;              // [kStages][64]
constexpr int kOffMask = kOffScale + kStages * kTile * 4; // [kStages] u64
constexpr int kOffHead = kOffMask + kStages * 8 + 16;     // [64] factors of a rescale, or of the output
constexpr int kOffQs = kOffHead + kH * 4;                 // [64] 2^-e of the query rows
constexpr int kOffRope = kOffQs + kH * 4;                 // cos[32], sin[32]
constexpr int kOffBars = kOffRope + 64 * 4;
constexpr int kOffPlan = kOffBars + 32 * 8;
constexpr int kOffTmem = kOffPlan + 40 * 4;
constexpr int kSmem = kOffTmem + 32 + 1024;
static_assert(kOffBars % 8 == 0 && kOffHead % 16 == 0 && kSmem <= 232448, "shared memory");

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

// Tiles of a query: a selection's 64 rows each; then runs of u rows (u the largest common part of a page and a tile, so a
// run lies in one page) of the dense sections, 64 / u to a tile.
struct TileCut {
  int sel_tiles, runs0, runs1, runs2;  // runs of rows, of first tokens, of window tokens
  int w_run;                           // first run of the window
  int tiles;
};
__device__ __forceinline__ TileCut cut_tiles(const PagedArgs& a, const PagedQuery& k, int u) {
  TileCut c;
  c.sel_tiles = a.sel ? (k.n0 + kTile - 1) / kTile : 0;
  c.runs0 = a.sel ? 0 : (k.n0 + u - 1) / u;  // (tables hold at most 2^30 rows)
  c.runs1 = (k.f + u - 1) / u;
  c.w_run = k.w0 / u;
  c.runs2 = k.nw > 0 ? (k.w0 + k.nw - 1) / u - c.w_run + 1 : 0;
  const int per = kTile / u;
  c.tiles = k.live ? max(1, c.sel_tiles + (int)(((long long)c.runs0 + c.runs1 + c.runs2 + per - 1) / per)) : 0;
  return c;
}

// Run x of a query: its first logical row, the rows [lo, hi) of its section that count, and the table.
struct Run {
  int start, lo, hi;
  const int32_t* table;
  int pages;
};
__device__ __forceinline__ Run run_of(const PagedArgs& a, const PagedQuery& k, const TileCut& c, int x, int u) {
  Run r;
  r.table = a.token_table;
  r.pages = a.token_pages;
  if (x < c.runs0) {
    r.start = x * u; r.lo = 0; r.hi = k.n0;
    r.table = a.row_table;
    r.pages = a.row_pages;
  } else if (x < c.runs0 + c.runs1) {
    r.start = (x - c.runs0) * u; r.lo = 0; r.hi = k.f;
  } else if (x < c.runs0 + c.runs1 + c.runs2) {
    r.start = (c.w_run + x - c.runs0 - c.runs1) * u; r.lo = k.w0; r.hi = k.w0 + k.nw;
  } else {
    r.start = r.lo = r.hi = 0;  // behind the last run
  }
  return r;
}

struct Smem {
  uint8_t* base;
  uint64_t *full, *empty, *s_full, *p_full, *pv_done, *q_ready, *drain;
  volatile int* dead;
};

// A bounded wait; a block in which one has run out (dead) waits no more.
__device__ __forceinline__ bool wait(const Smem& sm, uint64_t* bar, uint32_t parity) {
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
    k_tc_attend_pages(const __grid_constant__ CUtensorMap tm_runs, const __grid_constant__ CUtensorMap tm_rows,
                      const __grid_constant__ PagedArgs a, int u) {
  tc::tma_prefetch(&tm_runs);
  pdl_trigger();  // (the merge alone follows, and waits)
  extern __shared__ uint8_t smem_raw[];
  Smem sm;
  sm.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm.base + kOffBars);
  sm.full = bars;
  sm.empty = bars + kStages;
  sm.s_full = bars + 2 * kStages;
  sm.p_full = sm.s_full + 2;
  sm.pv_done = sm.p_full + 2;
  sm.q_ready = sm.pv_done + 2;
  sm.drain = sm.q_ready + 1;
  int* plan = reinterpret_cast<int*>(sm.base + kOffPlan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm.base + kOffTmem);
  sm.dead = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = sm.dead + 1;  // tiles whose copies were issued (of the loader warp 0, when a wait ran out)
  float* scales = reinterpret_cast<float*>(sm.base + kOffScale);
  volatile uint64_t* masks = reinterpret_cast<volatile uint64_t*>(sm.base + kOffMask);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(sm.full + i, kLoaders + 32);  // every loader's copy, and loader 0's lanes for the scales
      tc::mbar_init(sm.empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(sm.s_full + i, 1);
      tc::mbar_init(sm.p_full + i, kSoft);
      tc::mbar_init(sm.pv_done + i, 1);
    }
    tc::mbar_init(sm.q_ready, kSoft);
    tc::mbar_init(sm.drain, 1);
    *sm.dead = 0;
    *issued = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();  // predecessors complete: what they wrote is visible and their tensor memory is free
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  const PagedRun run = paged_run(a, plan, [&](int q) { return cut_tiles(a, paged_query(a, q, false), u).tiles; });
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp < kLoaders) {
    // ------------------------------------------------------------ loaders: 128 dims each of every tile
    int pre = run.pre, j = 0;  // j: tiles of this block so far
    const int c = warp, per = kTile / u, shift = __ffs(u) - 1;
    bool ok = true;
#pragma unroll 1
    for (int q = run.q; ok && pre < run.t1; ++q) {
      const PagedQuery k = paged_query(a, q, false);
      const TileCut cut = cut_tiles(a, k, u);
      if (cut.tiles == 0) continue;
      const int begin = max(run.t0 - pre, 0), end = min(run.t1 - pre, cut.tiles);
      const int n_rows = a.sel ? a.n_rows[k.b] : 0;
#pragma unroll 1
      for (int t = begin; t < end; ++t, ++j) {
        const int st = j % kStages;
        int r0, r1;       // physical rows of keys lane and lane + 32, -1 for none
        int run_row = 0;  // dense: lane's run's first physical row, -1 for none
        const bool selected = t < cut.sel_tiles;
        if (selected) {
          const int x = t * kTile + lane;
          const int32_t* sel = a.sel + (size_t)q * a.topk;
          const int j0 = x < k.n0 ? __ldg(sel + x) : -1, j1 = x + 32 < k.n0 ? __ldg(sel + x + 32) : -1;
          r0 = x < k.n0 ? paged_selected(a, k, j0, n_rows) : -1;
          r1 = x + 32 < k.n0 ? paged_selected(a, k, j1, n_rows) : -1;
        } else {
          const int x = (t - cut.sel_tiles) * per + lane;
          Run run_l = run_of(a, k, cut, lane < per ? x : INT32_MAX, u);
          run_row = -1;
          if (run_l.hi > run_l.lo) {
            run_row = paged_row(run_l.table, run_l.pages, k.b, run_l.start, a.P, a.n_pages);
            if (run_row < 0) atomicOr(a.err, CSA_DEV_RANGE);
          }
          int rr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = lane + 32 * e, from = key >> shift, off = key & (u - 1);
            const int row = __shfl_sync(0xffffffffu, run_row, from), start = __shfl_sync(0xffffffffu, run_l.start, from);
            const int lo = __shfl_sync(0xffffffffu, run_l.lo, from), hi = __shfl_sync(0xffffffffu, run_l.hi, from);
            rr[e] = row >= 0 && start + off >= lo && start + off < hi ? row + off : -1;
          }
          r0 = rr[0];
          r1 = rr[1];
        }
        ok = warp_wait(sm, sm.empty + st, ((j / kStages) & 1) ^ 1);
        if (!ok) break;
        if (warp == 0) {
          const uint32_t on0 = __ballot_sync(0xffffffffu, r0 >= 0), on1 = __ballot_sync(0xffffffffu, r1 >= 0);
          const uint32_t dst = tc::smem_u32(scales + st * kTile + lane);
          tc::cp_async4(dst, a.scales + max(r0, 0), r0 >= 0 ? 4u : 0u);
          tc::cp_async4(dst + 128, a.scales + max(r1, 0), r1 >= 0 ? 4u : 0u);
          if (lane == 0) {
            masks[st] = (uint64_t)on1 << 32 | on0;
            *issued = j + 1;
          }
          __syncwarp();
          tc::cp_async_arrive(sm.full + st);
        }
        if (lane == 0) tc::mbar_arrive_expect_tx(sm.full + st, kBox);
        __syncwarp();
        uint8_t* dst = sm.base + st * kStage + c * kBox;
        if (selected) {
          // four rows a request; an empty row is row 0 of the pool, cleared before the product that its values would enter
          const int l4 = 4 * (lane & 15);
          int g[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x0 = __shfl_sync(0xffffffffu, r0, (l4 + e) & 31), x1 = __shfl_sync(0xffffffffu, r1, (l4 + e) & 31);
            g[e] = max(l4 + e < 32 ? x0 : x1, 0);
          }
          if (lane < 16) tc::tma_gather4(dst + l4 * 128, &tm_rows, sm.full + st, c * 128, g[0], g[1], g[2], g[3]);
        } else if (lane < per) {
          // (a run in no page: rows behind the pool's end, which the copy fills with zeros)
          tc::tma_load_2d(dst + lane * u * 128, &tm_runs, sm.full + st, c * 128, run_row >= 0 ? run_row : a.n_pages * a.P);
        }
      }
      pre += cut.tiles;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    constexpr uint32_t id_qk = tc::idesc_e4m3(128, kTile);
    constexpr uint32_t id_pv = tc::idesc_e4m3(128, kH, true);
    const uint64_t kd = tc::sdesc_kmajor_sw128(tc::smem_u32(sm.base));
    const uint64_t vd = tc::sdesc_mnmajor_sw128(tc::smem_u32(sm.base), kBox, 1024);
    const uint64_t pd = tc::sdesc_kmajor_sw128(tc::smem_u32(sm.base + kOffP));
    int pre = run.pre, j = 0, seg = 0;
    // the product O^T of tile jp, whose probabilities the softmax warps have written
    auto pv = [&](int jp, bool first) {
      if (!warp_wait(sm, sm.p_full + (jp & 1), (jp >> 1) & 1)) return false;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        const uint64_t va = vd + (uint64_t)((jp % kStages) * kStage >> 4), pa = pd + (uint64_t)((jp & 1) * kPBuf >> 4);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int s = 0; s < 4; ++s)  // hi keys 0-31, 32-63, lo keys 0-31, 32-63
            tc::mma_f8(tmem + kColO + 64 * m, va + ((m * kBox + (s & 1) * 4096) >> 4), pa + (s * 32 >> 4), id_pv,
                       !first || s > 0);
        tc::mma_commit(sm.empty + jp % kStages);
        tc::mma_commit(sm.pv_done + (jp & 1));
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
#pragma unroll 1
    for (int q = run.q; ok && pre < run.t1; ++q) {
      const int n = cut_tiles(a, paged_query(a, q, false), u).tiles;
      if (n == 0) continue;
      const int begin = max(run.t0 - pre, 0), end = min(run.t1 - pre, n);
      ok = warp_wait(sm, sm.q_ready, seg & 1);
      ++seg;
      tc::fence_after_sync();
#pragma unroll 1
      for (int t = begin; ok && t < end; ++t, ++j) {
        ok = warp_wait(sm, sm.full + j % kStages, (j / kStages) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint64_t kb = kd + (uint64_t)((j % kStages) * kStage >> 4);
#pragma unroll
          for (int s = 0; s < 16; ++s)
            tc::mma_f8_ta(tmem + kColS + 64 * (j & 1), tmem + kColQ + 8 * s, kb + (((s >> 2) * kBox + (s & 3) * 32) >> 4),
                          id_qk, s > 0);
          tc::mma_commit(sm.s_full + (j & 1));
        }
        __syncwarp();
        if (t > begin) ok = pv(j - 1, t - 1 == begin);
      }
      if (ok) ok = pv(j - 1, end - 1 == begin);
      pre += n;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, plane = lane >> 4, h = 16 * quad + (lane & 15), st_id = tid - 32 * (kLoaders + 1);
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    float* fac = reinterpret_cast<float*>(sm.base + kOffHead);
    float* qs = reinterpret_cast<float*>(sm.base + kOffQs);
    float* rcos = reinterpret_cast<float*>(sm.base + kOffRope);
    float* rsin = rcos + 32;
    int pre = run.pre, j = 0;
#pragma unroll 1
    for (int q = run.q; pre < run.t1; ++q) {
      const PagedQuery k = paged_query(a, q, false);
      const int n = cut_tiles(a, k, u).tiles;
      if (n == 0) continue;
      const int begin = max(run.t0 - pre, 0), end = min(run.t1 - pre, n);
      // ---- the query's 64 rows as two E4M3 parts of 2^-e q, into tensor memory (every product that read the last
      // query has retired; the probabilities' buffers are free: 4 KB a warp to turn rows into lanes)
      {
        const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)q * kH + 16 * quad) * kD;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const uint4* src = reinterpret_cast<const uint4*>(qp + i * kD);
          const uint4 v0 = __ldg(src + lane), v1 = __ldg(src + 32 + lane);
          // the largest magnitude by its bits: bf16 pairs compared as unsigned 16-bit halves
          uint32_t mx = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t w = e < 4 ? (&v0.x)[e & 3] : (&v1.x)[e & 3];
            mx = __vmaxu2(mx, w & 0x7fff7fffu);
          }
          mx = max(mx & 0xffffu, mx >> 16);
          mx = __reduce_max_sync(0xffffffffu, mx);
          // 2^-e with e = exponent - 7: values below 2^8; a row of denormals, or zeros, is left small; a row that holds
          // an infinity or a NaN becomes NaN by its product with 0
          const int be = max((int)(mx >> 7), 8);
          if (lane == 0) qs[16 * quad + i] = be == 255 ? 0.f : __uint_as_float((uint32_t)max(261 - be, 1) << 23);
        }
        __syncwarp();
        uint8_t* stage = sm.base + kOffP + quad * 4096;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int hh = 2 * i + plane, c8 = lane & 15;
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(qp + hh * kD + c * 128) + c8);
            const float inv = qs[16 * quad + hh];
            uint2 hi, lo;
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = (&v.x)[e];
              x[2 * e] = __uint_as_float(w << 16) * inv;
              x[2 * e + 1] = __uint_as_float(w & 0xffff0000u) * inv;
            }
            hi.x = e4m3x4(x[0], x[1], x[2], x[3]);
            hi.y = e4m3x4(x[4], x[5], x[6], x[7]);
            const float2 b0 = e4m3x2_f(hi.x), b1 = e4m3x2_f(hi.x >> 16), b2 = e4m3x2_f(hi.y), b3 = e4m3x2_f(hi.y >> 16);
            lo.x = e4m3x4((x[0] - b0.x) * 16.f, (x[1] - b0.y) * 16.f, (x[2] - b1.x) * 16.f, (x[3] - b1.y) * 16.f);
            lo.y = e4m3x4((x[4] - b2.x) * 16.f, (x[5] - b2.y) * 16.f, (x[6] - b3.x) * 16.f, (x[7] - b3.y) * 16.f);
            const int at = (((c8 >> 1) ^ (hh & 7)) << 4) + (c8 & 1) * 8;
            *reinterpret_cast<uint2*>(stage + hh * 128 + at) = hi;
            *reinterpret_cast<uint2*>(stage + (16 + hh) * 128 + at) = lo;
          }
          __syncwarp();
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(w + 4 * e) = *reinterpret_cast<const uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4));
          tc::tmem_st32(tmem + kColQ + 32 * c + lanes, w);
          __syncwarp();
        }
        tc::tmem_wait_st();
        if (st_id < 32 && a.inv_freq) rope_cs(k.p, a.inv_freq, st_id, rcos + st_id, rsin + st_id);
        tc::named_bar(2, kSoft);  // (every warp's rows have left the buffers, and the angles are there)
        tc::fence_before_sync();
        tc::mbar_arrive(sm.q_ready);
      }
      const float inv_q = qs[h], c_h = inv_q == 0.f ? NAN : a.scale2 / inv_q;
      const float c_own = plane ? c_h * 0.0625f : c_h, c_other = plane ? c_h : c_h * 0.0625f;
      float m = -INFINITY, l = 0.f, ref = -INFINITY;
#pragma unroll 1
      for (int t = begin; t < end; ++t, ++j) {
        const int st = j % kStages, pb = j & 1;
        wait(sm, sm.full + st, (j / kStages) & 1);
        wait(sm, sm.s_full + pb, (j >> 1) & 1);
        tc::fence_after_sync();
        float s[32];
        {
          uint32_t x[64];
          tc::tmem_ld32(tmem + kColS + 64 * pb + lanes, x);
          tc::tmem_ld32(tmem + kColS + 64 * pb + 32 + lanes, x + 32);
          tc::tmem_wait_ld();
          // hi part lanes keep keys 0-31 and send 32-63, lo part lanes the other way round
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t send = plane ? x[e] : x[e + 32], keep = plane ? x[e + 32] : x[e];
            const float got = __uint_as_float(__shfl_xor_sync(0xffffffffu, send, 16));
            s[e] = fmaf(got, c_other, __uint_as_float(keep) * c_own);
          }
        }
        const uint64_t mask64 = masks[st];
        const uint32_t on = (uint32_t)(mask64 >> (32 * plane));
        const float* ks = scales + st * kTile + 32 * plane;
        float mt = -INFINITY;
#pragma unroll
        for (int e4 = 0; e4 < 8; ++e4) {
          const float4 k4 = reinterpret_cast<const float4*>(ks)[e4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * e4 + i;
            s[e] = (on >> e & 1u) ? s[e] * (&k4.x)[i] : -INFINITY;
            mt = fmaxf(mt, s[e]);
          }
        }
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
        const float mn = fmaxf(m, mt), mr = mn == -INFINITY ? 0.f : mn;
        l *= ex2(m - mr);
        m = mn;
        float vt = 0.f;
#pragma unroll
        for (int e4 = 0; e4 < 8; ++e4) {
          const float4 k4 = reinterpret_cast<const float4*>(ks)[e4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * e4 + i;
            const float p = ex2(s[e] - mr);
            l += p;
            s[e] = p * (&k4.x)[i];  // (a masked key's scale is 0)
            vt = fmaxf(vt, s[e]);
          }
        }
        vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 16));
        // the reference follows log2 of the largest 2^t ks
        const float lv = vt > 0.f ? mr + lg2(vt) : -INFINITY;
        bool moved = false;
        if (t == begin) {
          ref = lv;
        } else if (lv > ref + kStep) {
          if (plane == 0) fac[h] = ref == -INFINITY ? 1.f : ex2(ref - lv);  // (nothing has entered the product so far: zeros)
          ref = lv;
          moved = true;
        } else if (plane == 0) {
          fac[h] = 1.f;
        }
        const float gain = ref == -INFINITY ? 0.f : ex2(kGain + mr - ref);
        // the buffer's last reader, and before a rescale the last product's accumulators
        if (j >= 2) wait(sm, sm.pv_done + pb, ((j >> 1) & 1) ^ 1);
        if (tc::named_bar_any(3, kSoft, moved)) {
          wait(sm, sm.pv_done + (pb ^ 1), ((j - 1) >> 1) & 1);
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t x[32];
            tc::tmem_ld32(tmem + kColO + 32 * c + lanes, x);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
              const float4 f4 = reinterpret_cast<const float4*>(fac + 32 * (c & 1))[e4];
#pragma unroll
              for (int i = 0; i < 4; ++i) x[4 * e4 + i] = __float_as_uint(__uint_as_float(x[4 * e4 + i]) * (&f4.x)[i]);
            }
            tc::tmem_st32(tmem + kColO + 32 * c + lanes, x);
          }
          tc::tmem_wait_st();
          tc::named_bar(2, kSoft);  // (the factors have been read)
        }
        // ---- the probabilities' two parts
        uint8_t* row = sm.base + kOffP + pb * kPBuf + h * 128;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 hi, lo;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = s[16 * c + 4 * i + e] * gain;
            const uint32_t w = e4m3x4(v[0], v[1], v[2], v[3]);
            const float2 b0 = e4m3x2_f(w), b1 = e4m3x2_f(w >> 16);
            (&hi.x)[i] = w;
            (&lo.x)[i] = e4m3x4(v[0] - b0.x, v[1] - b0.y, v[2] - b1.x, v[3] - b1.y);
          }
          *reinterpret_cast<uint4*>(row + (((2 * plane + c) ^ (h & 7)) << 4)) = hi;
          *reinterpret_cast<uint4*>(row + (((4 + 2 * plane + c) ^ (h & 7)) << 4)) = lo;
        }
        if (mask64 != ~0ull) {
          // rows that are no keys hold whatever their page does: zeros, before the product would meet a NaN among them
          for (int e = st_id; e < kTile * 32; e += kSoft) {
            const int r = e >> 5;
            if (!(mask64 >> r & 1ull))
              *reinterpret_cast<uint4*>(sm.base + st * kStage + ((e & 31) >> 3) * kBox + r * 128 + (e & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
        }
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        tc::mbar_arrive(sm.p_full + pb);
      }
      // ---- the run's part of this query, or its output
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const bool whole = begin == 0 && end == n;
      const size_t slot = 2 * blockIdx.x + (begin == 0 ? 1 : 0);
      if (plane == 0) {
        float f = ref == -INFINITY ? 0.f : ex2(ref - kGain - m);  // O^T * f = sum 2^{t - m} key
        if (whole) {
          const float z2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
          const float M = fmaxf(m, z2), g = m == -INFINITY ? 0.f : ex2(m - M);
          const float Z = l * g + (z2 == -INFINITY ? 0.f : ex2(z2 - M));
          f = Z == 0.f ? 0.f : f * (g / Z);
        } else {
          a.ml[slot * kH + h] = make_float2(m, l);
        }
        fac[h] = f;
      }
      wait(sm, sm.pv_done + ((j - 1) & 1), ((j - 1) >> 1) & 1);
      tc::fence_after_sync();
      if (!tc::named_bar_any(3, kSoft, *sm.dead != 0)) {
        // a thread holds dim 128 c + 32 quad + lane of every head: a warp writes 32 consecutive values a head
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          const int d = 128 * (c >> 1) + 32 * quad + lane;
          uint32_t x[32];
          tc::tmem_ld32(tmem + kColO + 32 * c + lanes, x);
          tc::tmem_wait_ld();
          const float* f = fac + 32 * (c & 1);
          if (!whole) {
            float* dst = a.part + (slot * kH + 32 * (c & 1)) * kD + d;
#pragma unroll
            for (int e = 0; e < 32; ++e) dst[e * kD] = __uint_as_float(x[e]) * f[e];
            continue;
          }
          // two heads at a time: even lanes write head e's pair of dims, odd lanes head e + 1's
          const int odd = lane & 1, dp = d - odd, i = (dp - (kD - kR)) >> 1;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + ((size_t)q * kH + 32 * (c & 1) + odd) * kD + dp;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float v0 = __uint_as_float(x[e]) * f[e], v1 = __uint_as_float(x[e + 1]) * f[e + 1];
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
            float y0 = odd ? got : v0, y1 = odd ? v1 : got;
            if (dp >= kD - kR && a.inv_freq) {
              const float cs = rcos[i], sn = rsin[i], z0 = y0;
              y0 = fmaf(z0, cs, y1 * sn);
              y1 = fmaf(-z0, sn, y1 * cs);
            }
            *reinterpret_cast<__nv_bfloat162*>(dst + (size_t)e * kD) = __floats2bfloat162_rn(y0, y1);
          }
        }
      }
      tc::fence_before_sync();
      tc::named_bar(2, kSoft);  // (the factors have been read)
      pre += n;
    }
  }
  // ---- everything in flight has landed and retired before shared and tensor memory go
  tc::fence_before_sync();
  __syncthreads();
  if (*sm.dead) {
    if (tid == 0) {
      atomicOr(a.err, tc::kErrTimeout);
      const int upto = *issued;
      for (int j = max(0, upto - kStages); j < upto; ++j) tc::mbar_wait(sm.full + j % kStages, (j / kStages) & 1);
    }
  }
  if (warp == kMmaWarp) {
    if (tc::elect_one()) {
      tc::mma_commit(sm.drain);
      if (!tc::mbar_wait(sm.drain, 0)) atomicOr(a.err, tc::kErrTimeout);
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kCols);
}

}  // namespace

bool tc_paged_supported(const Dims& L, int n_pages, int P) {
  return L.dtype == CSA_BF16 && L.H == kH && L.D == kD && L.R == kR && P % 8 == 0;
}

cudaError_t launch_tc_paged(const Dims& L, const PagedArgs& a, int blocks, cudaStream_t s) {
  const int u = min(kTile, a.P & -a.P);  // the largest power of two that divides a page, at most a tile
  const uint64_t rows = (uint64_t)a.n_pages * a.P;
  CUtensorMap tm_runs, tm_rows;
  if (!make_tmap_2d_u8(&tm_runs, a.codes, rows, kD, kD, 128, u, true) ||
      !make_tmap_2d_u8(&tm_rows, a.codes, rows, kD, kD, 128, 1, true))
    return cudaErrorInvalidValue;
  allow_smem<kSmem>(k_tc_attend_pages);
  PagedArgs b = a;
  b.min_tiles = 2;
  CSA_LAUNCH(k_tc_attend_pages, dim3(blocks), dim3(kThreads), kSmem, s, tm_runs, tm_rows, b, u);
  return cudaGetLastError();
}

}  // namespace csa
