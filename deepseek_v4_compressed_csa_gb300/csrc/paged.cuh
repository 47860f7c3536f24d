// A cache in pages and 8 bits, as its kernels see it.
//
// codes [n_pages, P, D] E4M3 and scales [n_pages, P] fp32: row (page, s) stands for scale * code.  A table per sequence
// names the page of its logical rows [k P, (k + 1) P).  What attends reads two such views of one pool of pages: tokens
// (logical row t = token t: a window and a few first ones) and compressed rows (all visible ones, or a selection).
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace csa {

// values v = x / scale as four E4M3 codes (nearest even, saturating; NaN stays NaN), the first in the low byte
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// two codes (low 16 bits) as fp32
__device__ __forceinline__ float2 e4m3x2_f(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xffffu), __NV_E4M3);
  return __half22float2(__half2(h));
}
// fmaxf that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// (mean(x^2) + eps)^-1/2 of a row whose square sum may pass fp32's range (values from about 2^57 on): then anew from the
// values times 2^-80, sum(f) being their square sum times f^2 (the same answer in every thread that shares the row): 2^14
// squares of the largest values there are sum up to 2^110.
template <typename Sum>
__device__ __forceinline__ float inv_rms(float inv_n, float eps, Sum sum) {
  const float ss = sum(1.f);
  if (!isinf(ss)) return rsqrtf(fmaf(ss, inv_n, eps));
  constexpr float f = 8.27180612553027674871e-25f;  // 2^-80
  return rsqrtf(fmaf(sum(f), inv_n, eps * f * f)) * f;
}
// cos and sin of theta = (float)p * freq (one fp32 product, as in rope_cs).  Far positions: theta = m 2^e as a fraction
// of a turn, m 2^e / 2 pi modulo 1, in 64-bit fixed point (M. H. Payne and R. N. Hanek, Radian Reduction for Trigonometric
// Functions; one word of 1 / 2 pi is enough up to theta = 2^29, off by less than 2^-35 turns), and from it the remainder to
// the nearest quarter turn: sincosf's own reduction of angles above 10^5 cost a warp of the attention 5K clocks, one in fp64
// nearly as much.
__device__ __forceinline__ void turn_cs(int p, float freq, float* c, float* s) {
  const float th = __fmul_rn((float)p, freq), mag = fabsf(th);
  float r = th, sr, cr;
  int n = 0;
  if (mag > 1e5f && mag < 536870912.f) {
    const uint32_t bits = __float_as_uint(mag);
    const int e = (int)(bits >> 23) - 150;  // -7 .. 5
    const uint64_t m = (bits & 0x7fffffu) | 0x800000u, f = 0x28be60db9391054aull;  // f: 2^64 / 2 pi
    const uint64_t lo = m * f, hi = __umul64hi(m, f);
    uint64_t u = e >= 0 ? lo << e : (lo >> -e) | (hi << (64 + e));
    if (th < 0.f) u = 0 - u;
    const uint64_t quarter = (u + (1ull << 61)) >> 62;
    n = (int)quarter & 3;
    r = (float)(int64_t)(u - (quarter << 62)) * 3.4061215800304e-19f;  // 2 pi / 2^64
  }
  sincosf(r, &sr, &cr);
  const float x = n & 1 ? sr : cr, y = n & 1 ? cr : sr;
  *c = n == 1 || n == 2 ? -x : x;
  *s = n & 2 ? -y : y;
}
// v / s rounded once, 0 where the scale is 0 (a row of zeros, or so small that amax / 448 is)
__device__ __forceinline__ float over_scale(float v, float s) { return s == 0.f ? 0.f : __fdiv_rn(v, s); }

// ---------------------------------------------------------------- the queries of a call and their keys
__device__ __forceinline__ int divided(const FastDiv& d, int n) { return (int)((__umulhi(d.m, (uint32_t)n) + (uint32_t)n) >> d.l); }
// The page of a table that logical row j lies in
__device__ __forceinline__ int page_of(const PagedArgs& a, int j) { return divided(a.by_page, j); }
// Physical row of logical row j of a sequence's table, -1 where the table names no page of the pool.
__device__ __forceinline__ int paged_row(const PagedArgs& a, const int32_t* __restrict__ table, int j) {
  const int k = page_of(a, j), page = __ldg(table + k);
  return (unsigned)page < (unsigned)a.n_pages ? page * a.P + (j - k * a.P) : -1;
}

// Query q = b T + i sits at p = pos[b] + i.  Its keys, in this order:
//   n0 compressed rows: sel[q][0 .. n0), or rows 0 .. n0 - 1 without a selection;
//   f first tokens 0 .. f - 1 (those before its window);
//   nw window tokens w0 .. p.
// tiles: what the attention kernel cuts them into (at least one for a query that is there, 0 for none); n_rows bounds the
// selected rows.
struct PagedQuery {
  int q, b, p, n0, f, w0, nw, n_rows, tiles;
};

// Tiles of a.tile keys, a power of two.  shift == 0: the keys in a row.  Else (the tensor-core kernel) a selection's rows by themselves,
// then runs of 2^shift rows, which lie in one page each, some to a tile.
struct TileCut {
  int sel_tiles, runs0, runs1, runs2;  // runs of rows, of first tokens, of window tokens
  int w_run;                           // first run of the window
};
__device__ __forceinline__ TileCut cut_tiles(bool selected, const PagedQuery& k, int tile, int shift) {
  TileCut c;  // (tables hold at most 2^30 rows: no sum overflows)
  const int u = 1 << shift;
  c.sel_tiles = selected ? (k.n0 + tile - 1) >> (31 - __clz(tile)) : 0;
  c.runs0 = selected ? 0 : (k.n0 + u - 1) >> shift;
  c.runs1 = (k.f + u - 1) >> shift;
  c.w_run = k.w0 >> shift;
  c.runs2 = k.nw > 0 ? ((k.w0 + k.nw - 1) >> shift) - c.w_run + 1 : 0;
  return c;
}

// report: raise the error bits of what is wrong with query q
__device__ __forceinline__ PagedQuery find_query(const PagedArgs& a, int q, bool report) {
  PagedQuery k;
  const int b = divided(a.by_T, q), i = q - b * a.T;
  // (all at once: one round trip)
  const int p0 = a.pos[b], n = a.n_new ? a.n_new[b] : a.T, rows = a.row_table ? a.n_rows[b] : 0, ns = a.sel ? a.n_sel[q] : 0;
  const bool ok = p0 >= 0 && p0 <= INT32_MAX - a.T && n >= 0 && n <= a.T;
  int bits = ok ? 0 : CSA_DEV_STATE;
  k.q = q;
  k.b = b;
  k.p = p0 + i;
  k.n0 = k.f = k.w0 = k.nw = k.n_rows = k.tiles = 0;
  if (ok && i < n) {
    if (a.row_table) {
      if (rows < 0) bits |= CSA_DEV_STATE;
      k.n_rows = max(rows, 0);
      const int held = a.row_pages * a.P;  // rows that the table has room for (at most 2^30)
      if (a.sel) {
        if (ns < 0 || ns > a.topk) bits |= CSA_DEV_RANGE;
        k.n0 = min(max(ns, 0), a.topk);
        k.n_rows = min(k.n_rows, held);  // (a selected row behind the table's end is out of range)
      } else {
        k.n0 = min(k.n_rows, divided(a.by_ratio, k.p + 1));
        if (k.n0 > held) {
          bits |= CSA_DEV_CAPACITY;
          k.n0 = held;
        }
      }
    }
    if (a.token_table) {
      int last = k.p;
      const int held = a.token_pages * a.P;
      if (last >= held) {
        bits |= CSA_DEV_CAPACITY;
        last = held - 1;
      }
      k.w0 = k.p >= a.W ? k.p - a.W + 1 : 0;
      k.nw = max(0, last - k.w0 + 1);
      k.f = min(min(a.first, k.w0), last + 1);
    }
    const TileCut c = cut_tiles(a.sel != nullptr && a.shift > 0, k, a.tile, a.shift);
    const int per = a.tile >> a.shift;
    const unsigned runs = (unsigned)c.runs0 + c.runs1 + c.runs2;  // (at most 2^30 each)
    k.tiles = max(1, c.sel_tiles + (int)((runs + per - 1) >> (31 - __clz(per))));
  }
  if (report && bits) atomicOr(a.err, bits);
  return k;
}
// The next query that has tiles (the caller knows that there is one)
__device__ __forceinline__ PagedQuery next_query(const PagedArgs& a, int q) {
  PagedQuery k;
  do k = find_query(a, ++q, false);
  while (k.tiles == 0);
  return k;
}

// ---------------------------------------------------------------- work over the blocks
// Each query is cut into equal pieces of at most L tiles, and a block takes one piece, or neighbouring ones: its run
// [t0, t1) of all queries' tiles, one after another.  A run that covers a query whole writes its output; otherwise it leaves
// its part: slot 2 c + 1 if the query begins in the run of block c, 2 c if it began before.  parts[q] says where a query's
// parts are.  A part costs its block some 2 us and the merge as much, so queries are not cut for the last bit of balance:
//   fewer queries than blocks: every piece has a block of its own.  Of two lengths at which there are enough, the shorter:
//     the longest query over blocks / queries pieces, and total / (blocks - queries), since ceil(n / L) <= n / L + 1 (128
//     queries of 11 tiles on 152 blocks stay whole, 24 us; in even runs of 10 tiles, when the kernel took 29, 55);
//   more: L = total / blocks, so only longer queries than that are cut, and block c takes the pieces that begin in
//     [c, c + 1) total / blocks.  No piece of a cut query is longer than that, so all its blocks have one.
// Every block finds the plan itself (a few loads a query, spread over its threads): a kernel before it would cost more than
// that for the batches that count in microseconds.
struct PagedRun {
  int t0, t1;      // the run's tiles
  int pre;         // tiles before its first query
  PagedQuery k;    // that query
};
constexpr int kPlanInts = 96;  // scratch of paged_plan
constexpr int kPlanWarp = 32;  // queries whose plan one warp makes

__device__ __forceinline__ unsigned div_up(unsigned n, unsigned d) { return (n + d - 1) / d; }

// Sums over the block's threads of v: before this one, and of all.  scratch: 32 ints, 16-byte aligned; the block's barrier
// stands between the sums' writes and their reads.
__device__ __forceinline__ int warp_scan(int v, int* scratch) {
  const int lane = threadIdx.x & 31;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) scratch[threadIdx.x >> 5] = inc;
  return inc - v;
}
template <int nw>
__device__ __forceinline__ int2 scan_warps(const int* scratch) {
  const int warp = threadIdx.x >> 5;
  int before = 0, total = 0;
#pragma unroll
  for (int w4 = 0; w4 < nw; w4 += 4) {
    const int4 v = *reinterpret_cast<const int4*>(scratch + w4);
    before += (w4 < warp ? v.x : 0) + (w4 + 1 < warp ? v.y : 0) + (w4 + 2 < warp ? v.z : 0) + (w4 + 3 < warp ? v.w : 0);
    total += v.x + v.y + v.z + v.w;
  }
  return make_int2(before, total);
}

// Equal pieces of n tiles: the first n % m of them are a tile longer
struct Pieces {
  int m, base, rem;
  __device__ __forceinline__ Pieces(int n, int count) : m(count), base(n / max(count, 1)), rem(n - base * count) {}
  __device__ __forceinline__ int start(int i) const { return i * base + min(i, rem); }
  // the first piece that starts at or behind tile x (m if none)
  __device__ __forceinline__ int from(int x) const {
    if (x <= 0) return 0;
    const int longer = rem * (base + 1);
    const unsigned i = x <= longer ? div_up(x, base + 1) : rem + div_up(x - longer, max(base, 1));
    return (int)min(i, (unsigned)m);
  }
};

// The length of pieces where every piece gets a block of its own (queries < kPagedBlocks)
__device__ __forceinline__ int piece_length(const PagedArgs& a, int total, int queries, int longest) {
  const int each = (int)((float)kPagedBlocks / (float)max(queries, 1));  // (rounded right: whole quotients are exact)
  return max(max(a.min_tiles, (int)div_up(total, kPagedBlocks)),
             min((int)div_up(longest, each), (int)div_up(total, kPagedBlocks - queries)));
}

// Up to 32 queries, by one warp (the others wait at the barrier at its end): a third of the instructions of the plan below,
// which a launch has to fetch before it runs them.
__device__ __forceinline__ void paged_plan_warp(const PagedArgs& a, PagedRun* sm) {
  const int Q = a.B * a.T, lane = threadIdx.x, c = blockIdx.x;
  if (threadIdx.x < 32) {
    PagedQuery k;
    k.tiles = 0;
    if (lane < Q) k = find_query(a, lane, c == 0);
    const int n = k.tiles;
    const int total = __reduce_add_sync(0xffffffffu, n), queries = __popc(__ballot_sync(0xffffffffu, n > 0));
    const int L = piece_length(a, total, queries, __reduce_max_sync(0xffffffffu, n));
    const Pieces p(n, (int)div_up(n, L));
    int first = p.m, pre = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, first, o), v = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) {
        first += u;
        pre += v;
      }
    }
    const int pieces = __shfl_sync(0xffffffffu, first, 31), i = c - (first - p.m);
    pre -= n;
    if (i >= 0 && i < p.m) {
      sm->t0 = pre + p.start(i);
      sm->t1 = pre + p.start(i + 1);
      sm->pre = pre;
      sm->k = k;
    }
    if (c >= pieces && lane == 0) sm->t0 = sm->t1 = 0;
    if (c == 0 && lane < Q) a.parts[lane] = make_int2(first - p.m, p.m);
  }
  __syncthreads();
}

// Whole block of 32 nw threads (nw a multiple of 4); `sm` in shared memory is the result.
template <int nw>
__device__ __noinline__ void paged_plan_block(const PagedArgs& a, PagedRun* sm, int* scratch) {
  constexpr int nt = 32 * nw;
  const int Q = a.B * a.T, tid = threadIdx.x, G = kPagedBlocks, c = blockIdx.x;
  const int each = (Q + nt - 1) / nt, q0 = min(Q, tid * each), q1 = min(Q, q0 + each);
  const bool lead = c == 0;
  int mine = 0, live = 0, longest = 0;
  PagedQuery k;
  for (int q = q0; q < q1; ++q) {
    k = find_query(a, q, lead);
    mine += k.tiles;
    live += k.tiles > 0;
    longest = max(longest, k.tiles);
  }
  int pre = warp_scan(mine, scratch);
  longest = __reduce_max_sync(0xffffffffu, longest);
  live = __reduce_add_sync(0xffffffffu, live);
  if ((tid & 31) == 0) {
    scratch[32 + (tid >> 5)] = longest;
    scratch[48 + (tid >> 5)] = live;
  }
  __syncthreads();
  // (a call has fewer than 2^31 tiles: the host refuses tables and batches that could hold more)
  const int2 warps = scan_warps<nw>(scratch);
  const int total = warps.y, queries = scan_warps<nw>(scratch + 48).y;
  pre += warps.x;
#pragma unroll
  for (int w = 0; w < nw; ++w) longest = max(longest, scratch[32 + w]);
  int t0 = total, t1 = total;  // (a block behind the last piece has nothing)
  if (queries < G) {
    const int L = piece_length(a, total, queries, longest);
    // (each is 1 but for batches of some hundred slots of which few are in use)
    int count = 0;
    for (int q = q0; q < q1; ++q) {
      if (each > 1) k = find_query(a, q, false);
      count += (int)div_up(k.tiles, L);
    }
    int first = warp_scan(tid < Q ? count : 0, scratch + 64);
    __syncthreads();
    first += scan_warps<nw>(scratch + 64).x;
    for (int q = q0; q < q1; ++q) {
      if (each > 1) k = find_query(a, q, false);
      const Pieces p(k.tiles, (int)div_up(k.tiles, L));
      const int i = c - first;
      if (i >= 0 && i < p.m) {
        sm->t0 = pre + p.start(i);
        sm->t1 = pre + p.start(i + 1);
        sm->pre = pre;
        sm->k = k;
      }
      if (lead) a.parts[q] = make_int2(first, p.m);
      first += p.m;
      pre += k.tiles;
    }
    if (tid == 0) scratch[80] = scan_warps<nw>(scratch + 64).y;
    __syncthreads();
    if (c >= scratch[80]) {  // a block without a piece
      if (tid == 0) sm->t0 = sm->t1 = 0;
      __syncthreads();
    }
    return;
  }
  const int base = total / G, rem = total - base * G, L = a.merge ? max(1, base) : max(a.min_tiles, base);
  auto begin = [&](int b) { return b * base + (b * rem + G - 1) / G; };  // ceil(b total / G)
  const int lo = begin(c), hi = begin(c + 1);
  int* run = scratch + 80;
  if (tid == 0) run[0] = run[1] = total;
  __syncthreads();
  int at = pre;
  for (int q = q0; q < q1; ++q) {
    if (each > 1) k = find_query(a, q, false);
    const Pieces p(k.tiles, (int)div_up(k.tiles, L));
    const int i0 = p.from(lo - at), i1 = p.from(hi - at);
    if (i0 < p.m) atomicMin(run, at + p.start(i0));
    if (i1 < p.m) atomicMin(run + 1, at + p.start(i1));
    if (lead) {
      auto block_of = [&](int x) {  // the block in whose share tile x lies
        int b = min(G - 1, (int)((float)x * ((float)G / (float)total)));
        while (b > 0 && begin(b) > x) --b;
        while (b < G - 1 && begin(b + 1) <= x) ++b;
        return b;
      };
      const int b0 = p.m > 0 ? block_of(at) : 0;
      a.parts[q] = make_int2(b0, p.m > 0 ? block_of(at + p.start(p.m - 1)) - b0 + 1 : 0);
    }
    at += k.tiles;
  }
  __syncthreads();
  t0 = run[0];
  t1 = run[1];
  at = pre;
  for (int q = q0; q < q1 && t0 < t1; ++q) {
    if (each > 1) k = find_query(a, q, false);
    if (k.tiles > 0 && at <= t0 && t0 < at + k.tiles) {
      sm->pre = at;
      sm->k = k;
    }
    at += k.tiles;
  }
  if (tid == 0) {
    sm->t0 = t0;
    sm->t1 = t1;
  }
  __syncthreads();
}

template <int nw>
__device__ __forceinline__ void paged_plan(const PagedArgs& a, PagedRun* sm, int* scratch) {
  if (a.B * a.T <= kPlanWarp) paged_plan_warp(a, sm);
  else paged_plan_block<nw>(a, sm, scratch);
}

}  // namespace csa
