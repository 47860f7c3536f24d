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
// (mean(x^2) + eps)^-1/2 of a row whose square sum may pass fp32's range (values from about 2^60 on): then anew from the
// values times 2^-64, sum(f) being their square sum times f^2 (the same answer in every thread that shares the row).
template <typename Sum>
__device__ __forceinline__ float inv_rms(float inv_n, float eps, Sum sum) {
  const float ss = sum(1.f);
  if (!isinf(ss)) return rsqrtf(fmaf(ss, inv_n, eps));
  constexpr float f = 5.42101086242752217e-20f;  // 2^-64
  return rsqrtf(fmaf(sum(f), inv_n, eps * f * f)) * f;
}
// v / s rounded once, 0 where the scale is 0 (a row of zeros, or so small that amax / 448 is)
__device__ __forceinline__ float over_scale(float v, float s) { return s == 0.f ? 0.f : __fdiv_rn(v, s); }

// ---------------------------------------------------------------- the queries of a call and their keys
// The page of a table that logical row j lies in
__device__ __forceinline__ int page_of(const PagedArgs& a, int j) {
  return (int)((__umulhi(a.by_page.m, (uint32_t)j) + (uint32_t)j) >> a.by_page.l);
}
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

// Tiles of a.tile keys.  shift == 0: the keys in a row.  Else (the tensor-core kernel) a selection's rows by themselves,
// then runs of 2^shift rows, which lie in one page each, some to a tile.
struct TileCut {
  int sel_tiles, runs0, runs1, runs2;  // runs of rows, of first tokens, of window tokens
  int w_run;                           // first run of the window
};
__device__ __forceinline__ TileCut cut_tiles(bool selected, const PagedQuery& k, int tile, int shift) {
  TileCut c;  // (tables hold at most 2^30 rows: no sum overflows)
  const int u = 1 << shift;
  c.sel_tiles = selected ? (k.n0 + tile - 1) / tile : 0;
  c.runs0 = selected ? 0 : (k.n0 + u - 1) >> shift;
  c.runs1 = (k.f + u - 1) >> shift;
  c.w_run = k.w0 >> shift;
  c.runs2 = k.nw > 0 ? ((k.w0 + k.nw - 1) >> shift) - c.w_run + 1 : 0;
  return c;
}

// report: raise the error bits of what is wrong with query q
__device__ __forceinline__ PagedQuery find_query(const PagedArgs& a, int q, bool report) {
  PagedQuery k;
  const int b = q / a.T, i = q - b * a.T;
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
        k.n0 = min(k.n_rows, (int)(((unsigned)k.p + 1u) / (unsigned)a.ratio));
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
    k.tiles = max(1, c.sel_tiles + (int)(((long long)c.runs0 + c.runs1 + c.runs2 + per - 1) / per));
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
// The tiles of all queries, one after another, are cut into equal runs, one a block: block c has tiles [c per, (c + 1) per).
// However ragged the batch, blocks end together, and one query of a long cache is spread over the device.  A run that
// covers a query whole writes its output; otherwise it leaves its part: slot 2 c + 1 if the query begins in the run, 2 c if
// it began before.  parts[q] says where a query's parts are.  Every block finds the plan itself (a few loads a query, spread
// over its threads): a kernel before it would cost more than that for the batches that count in microseconds.
struct PagedRun {
  int t0, t1;      // the run's tiles
  int pre;         // tiles before its first query
  PagedQuery k;    // that query
};

// Whole block (at most 1024 threads); `sm` in shared memory is the result.
__device__ __forceinline__ void paged_plan(const PagedArgs& a, PagedRun* sm, int* sums) {
  const int Q = a.B * a.T, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int each = (Q + nt - 1) / nt, q0 = min(Q, tid * each), q1 = min(Q, q0 + each);
  const bool lead = blockIdx.x == 0;
  int mine = 0;
  PagedQuery k;
  for (int q = q0; q < q1; ++q) {
    k = find_query(a, q, lead);
    mine += k.tiles;
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int pre = inc - mine, total = 0;
  for (int w = 0; w < nw; ++w) {
    pre += w < warp ? sums[w] : 0;
    total += sums[w];
  }
  // (a call has fewer than 2^31 tiles: the host refuses tables and batches that could hold more)
  const int per = max(a.min_tiles, (int)(((long long)total + gridDim.x - 1) / gridDim.x));
  const int t0 = (int)min((long long)total, (long long)blockIdx.x * per), t1 = (int)min((long long)total, (long long)t0 + per);
  if (tid == 0) {
    sm->t0 = t0;
    sm->t1 = t1;
  }
  for (int q = q0; q < q1; ++q) {
    if (each > 1) k = find_query(a, q, false);
    if (k.tiles > 0 && pre <= t0 && t0 < pre + k.tiles) {
      sm->pre = pre;
      sm->k = k;
    }
    if (lead) a.parts[q] = make_int2(pre / per, k.tiles > 0 ? (pre + k.tiles - 1) / per - pre / per + 1 : 0);
    pre += k.tiles;
  }
  __syncthreads();
}

}  // namespace csa
