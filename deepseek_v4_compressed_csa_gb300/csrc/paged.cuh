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
// tiles: what the attention kernel cuts them into (at least one for a query that is there, 0 for none); n_rows bounds the
// selected rows.
struct alignas(16) PagedQuery {
  int p, n0, f, w0;
  int nw, n_rows, tiles, q;
};

__device__ __forceinline__ PagedQuery load_query(const PagedQuery* r) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(r)), b = __ldg(reinterpret_cast<const int4*>(r) + 1);
  PagedQuery k;
  k.p = a.x; k.n0 = a.y; k.f = a.z; k.w0 = a.w;
  k.nw = b.x; k.n_rows = b.y; k.tiles = b.z; k.q = b.w;
  return k;
}

// Physical row of logical row j of sequence b's table, -1 where the table names no page of the pool.
__device__ __forceinline__ int paged_row(const int32_t* __restrict__ table, int pages, int b, int j, int P, int n_pages) {
  const int k = j / P, page = __ldg(table + (size_t)b * pages + k);
  return (unsigned)page < (unsigned)n_pages ? page * P + (j - k * P) : -1;
}

// ---------------------------------------------------------------- work over the blocks
// The tiles of all queries, one after another, are cut into equal runs, one a block: block c has tiles [c per, (c + 1) per).
// However ragged the batch, blocks end together, and one query of a long cache is spread over the device.  A run that
// covers a query whole writes its output; otherwise it leaves its part: slot 2 c + 1 if the query begins in the run, 2 c if
// it began before.  parts[q] says where a query's parts are.
struct alignas(16) PagedRun {
  int t0, t1;      // the run's tiles
  int pre, pad;    // tiles before its first query
  PagedQuery k;    // that query
};

// Tiles of `tile` keys.  u == 1: the keys in a row.  Else (the tensor-core kernel) a selection's rows by themselves, then
// runs of u rows, which lie in one page each, tile / u of them to a tile.
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

}  // namespace csa
