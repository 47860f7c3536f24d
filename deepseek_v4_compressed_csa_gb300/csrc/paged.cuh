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
// Query q = b T + i sits at p = pos[b] + i.  Its keys, in this order:
//   n0 compressed rows: sel[q][0 .. n0), or rows 0 .. n0 - 1 without a selection;
//   f first tokens 0 .. f - 1 (those before its window);
//   nw window tokens w0 .. p.
struct PagedQuery {
  int b, p, n0, f, w0, nw;
  bool live;
};

// report: this thread raises the error bits of what it finds (one thread a query does)
__device__ __forceinline__ PagedQuery paged_query(const PagedArgs& a, int q, bool report) {
  PagedQuery k;
  k.b = q / a.T;
  const int i = q - k.b * a.T, p0 = a.pos[k.b], n = a.n_new ? a.n_new[k.b] : a.T;
  const bool ok = p0 >= 0 && p0 <= INT32_MAX - a.T && n >= 0 && n <= a.T;
  k.live = ok && i < n;
  k.p = p0 + i;
  k.n0 = k.f = k.w0 = k.nw = 0;
  int bits = ok ? 0 : CSA_DEV_STATE;
  if (k.live) {
    if (a.row_table) {
      int rows = a.n_rows[k.b];
      if (rows < 0) {
        bits |= CSA_DEV_STATE;
        rows = 0;
      }
      if (a.sel) {
        k.n0 = a.n_sel[q];
        if (k.n0 < 0 || k.n0 > a.topk) bits |= CSA_DEV_RANGE;
        k.n0 = min(max(k.n0, 0), a.topk);
      } else {
        k.n0 = min(rows, (int)(((unsigned)k.p + 1u) / (unsigned)a.ratio));
        const long long held = (long long)a.row_pages * a.P;  // rows that the table has room for
        if (k.n0 > held) {
          bits |= CSA_DEV_CAPACITY;
          k.n0 = (int)held;
        }
      }
    }
    if (a.token_table) {
      int last = k.p;
      const long long held = (long long)a.token_pages * a.P;
      if (last >= held) {
        bits |= CSA_DEV_CAPACITY;
        last = (int)held - 1;
      }
      k.w0 = k.p >= a.W ? k.p - a.W + 1 : 0;
      k.nw = max(0, last - k.w0 + 1);
      k.f = min(min(a.first, k.w0), last + 1);
    }
  }
  if (report && bits) atomicOr(a.err, bits);
  return k;
}

// Physical row of logical row j of sequence b's table, -1 where the table names no page of the pool.
__device__ __forceinline__ int paged_row(const int32_t* __restrict__ table, int pages, int b, int j, int P, int n_pages) {
  const int k = j / P, page = __ldg(table + (size_t)b * pages + k);
  return (unsigned)page < (unsigned)n_pages ? page * P + (j - k * P) : -1;
}

// Physical row of selected row k of query q (-1: out of range or in no page; both are reported).
__device__ __forceinline__ int paged_selected(const PagedArgs& a, const PagedQuery& k, int j, int n_rows) {
  int r = -1;
  if (j >= 0 && j < n_rows && j / a.P < a.row_pages) r = paged_row(a.row_table, a.row_pages, k.b, j, a.P, a.n_pages);
  if (r < 0) atomicOr(a.err, CSA_DEV_RANGE);
  return r;
}

// ---------------------------------------------------------------- work over the blocks
// The tiles (64 keys, or 32 in the portable kernel) of all queries, one after another, are cut into equal runs, one a
// block: block c has tiles [c per, (c + 1) per).  However ragged the batch, blocks end together, and one query of a long
// cache is spread over the device.  A run that covers a query whole writes its output; otherwise it leaves its part:
// slot 2 c + 1 if the query begins in the run, 2 c if it began before.  parts[q] says where a query's parts are.
struct PagedRun {
  int q, pre;     // the first query of the run, and the tiles before it
  int t0, t1;     // the run's tiles
};

// Whole block.  tiles(q): a query's tiles (at least one if it is live, else 0).  `sm` holds 33 ints + 2.  The plan is
// found anew by every block (a load or two per query, spread over its threads), so it needs no kernel before it.
template <typename Tiles>
__device__ __forceinline__ PagedRun paged_run(const PagedArgs& a, int* sm, Tiles tiles) {
  const int Q = a.B * a.T, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int each = (Q + nt - 1) / nt, q0 = min(Q, tid * each), q1 = min(Q, q0 + each);
  int mine = 0;
  for (int q = q0; q < q1; ++q) mine += tiles(q);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sm[warp] = inc;
  __syncthreads();
  if (tid == 0) {
    int s = 0;
    for (int w = 0; w < nw; ++w) {
      const int v = sm[w];
      sm[w] = s;
      s += v;
    }
    sm[32] = s;
  }
  __syncthreads();
  const int total = sm[32], per = max(a.min_tiles, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  int pre = sm[warp] + inc - mine;
  PagedRun r;
  // (a call has fewer than 2^31 tiles: the host refuses tables and batches that could hold more)
  r.t0 = (int)min((long long)total, (long long)blockIdx.x * per);
  r.t1 = (int)min((long long)total, (long long)r.t0 + per);
  for (int q = q0; q < q1; ++q) {
    const int n = tiles(q);
    if (n > 0 && pre <= r.t0 && r.t0 < pre + n) {
      sm[33] = q;
      sm[34] = pre;
    }
    if (blockIdx.x == 0) {
      paged_query(a, q, true);
      // where the merge finds the query's parts: block of the first one, and how many (0 or 1: nothing to merge)
      a.parts[q] = make_int2(pre / per, n > 0 ? (pre + n - 1) / per - pre / per + 1 : 0);
    }
    pre += n;
  }
  __syncthreads();
  const bool any = r.t0 < r.t1;
  r.q = any ? sm[33] : 0;
  r.pre = any ? sm[34] : r.t1;
  return r;
}

}  // namespace csa
