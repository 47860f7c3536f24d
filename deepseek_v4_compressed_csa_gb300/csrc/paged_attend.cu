// Attention over a cache in pages and 8 bits: the plan of a call, the portable kernel (any head layout and size, bf16 and
// fp32), and the merge of queries that several blocks worked on.
//
//   l_k = scale q_h . key_k;  o_h = sum_k e^{l_k} key_k / (e^{sink_h} + sum_k e^{l_k});  out_h = RoPE^-1(o_h, p)
//
// over the keys of PagedQuery, key_k = scale_k code_k.  A block walks its run of tiles (paged.cuh) with a running maximum
// and sum per head; all arithmetic in fp32, the output rounded once.
#include "paged.cuh"
#include "tc.cuh"

namespace csa {

namespace {

// ---------------------------------------------------------------- the plan
// The last block: every query's keys and tiles, their sum, each block's run.  The others (tensor cores): the queries as
// two E4M3 parts each, q = 2^e (hi + lo / 16), a warp a row, in the order in which the attention kernel's lanes take them.
constexpr int kPlanThreads = 256;

// Query q's keys; what is wrong with them raises error bits.
__device__ __forceinline__ PagedQuery find_query(const PagedArgs& a, int q) {
  PagedQuery k;
  const int b = q / a.T, i = q - b * a.T, p0 = a.pos[b], n = a.n_new ? a.n_new[b] : a.T;
  const bool ok = p0 >= 0 && p0 <= INT32_MAX - a.T && n >= 0 && n <= a.T;
  int bits = ok ? 0 : CSA_DEV_STATE;
  k.q = q;
  k.p = p0 + i;
  k.n0 = k.f = k.w0 = k.nw = k.n_rows = k.tiles = 0;
  if (ok && i < n) {
    if (a.row_table) {
      k.n_rows = a.n_rows[b];
      if (k.n_rows < 0) {
        bits |= CSA_DEV_STATE;
        k.n_rows = 0;
      }
      const int held = a.row_pages * a.P;  // rows that the table has room for (at most 2^30)
      if (a.sel) {
        k.n0 = a.n_sel[q];
        if (k.n0 < 0 || k.n0 > a.topk) bits |= CSA_DEV_RANGE;
        k.n0 = min(max(k.n0, 0), a.topk);
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
    int tiles;
    if (a.shift == 0) {
      tiles = (int)(((long long)k.n0 + k.f + k.nw + a.tile - 1) / a.tile);
    } else {
      const TileCut c = cut_tiles(a.sel != nullptr, k, a.tile, a.shift);
      const int per = a.tile >> a.shift;
      tiles = c.sel_tiles + (int)(((long long)c.runs0 + c.runs1 + c.runs2 + per - 1) / per);
    }
    k.tiles = max(1, tiles);
  }
  if (bits) atomicOr(a.err, bits);
  return k;
}

__device__ __forceinline__ void store_query(PagedQuery* r, const PagedQuery& k) {
  reinterpret_cast<int4*>(r)[0] = make_int4(k.p, k.n0, k.f, k.w0);
  reinterpret_cast<int4*>(r)[1] = make_int4(k.nw, k.n_rows, k.tiles, k.q);
}

__device__ __forceinline__ void make_plan(const PagedArgs& a, int* sm) {
  const int Q = a.B * a.T, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (Q + kPlanThreads - 1) / kPlanThreads, q0 = min(Q, tid * each), q1 = min(Q, q0 + each);
  int mine = 0;
  PagedQuery k;
  for (int q = q0; q < q1; ++q) {
    k = find_query(a, q);
    store_query(a.queries + q, k);
    mine += k.tiles;
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sm[warp] = inc;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    before += w < warp ? sm[w] : 0;
    total += sm[w];
  }
  const int per = max(a.min_tiles, (total + kPagedBlocks - 1) / kPagedBlocks);
  int pre = before + inc - mine;
  for (int q = q0; q < q1; ++q) {
    if (each > 1) k = a.queries[q];
    if (k.tiles > 0) {
      const int c0 = pre / per, c1 = (pre + k.tiles - 1) / per;
      a.parts[q] = make_int2(c0, c1 - c0 + 1);
      for (int c = (pre + per - 1) / per; c <= c1; ++c) {  // the runs that begin in this query
        reinterpret_cast<int4*>(a.runs + c)[0] = make_int4(c * per, min(total, c * per + per), pre, 0);
        store_query(&a.runs[c].k, k);
      }
    } else {
      a.parts[q] = make_int2(0, 0);
    }
    pre += k.tiles;
  }
  for (int c = (total + per - 1) / per + tid; c < kPagedBlocks; c += kPlanThreads)
    reinterpret_cast<int4*>(a.runs + c)[0] = make_int4(0, 0, 0, 0);
}

// Row of the split queries' tile: a 32-row quarter holds 16 heads' hi parts, then their lo parts.
__device__ __forceinline__ void split_query_row(const PagedArgs& a, int row) {
  const int lane = threadIdx.x & 31, q = row >> 6, h = row & 63;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (size_t)row * 512) + 2 * lane;
  const uint4 v[2] = {src[0], src[1]};
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  // the largest magnitude by its bits: bf16 pairs compared as unsigned halves
  uint32_t mx = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = __vmaxu2(mx, w[e] & 0x7fff7fffu);
  mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
  // 2^-e with e = exponent - 7: values below 2^8, exact products; a row of denormals, or zeros, stays small; a row that
  // holds an infinity or a NaN becomes NaN by its product with 0
  const int be = max((int)(mx >> 7), 8);
  const float inv = be == 255 ? 0.f : __uint_as_float((uint32_t)(261 - be) << 23);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x0 = __uint_as_float(w[2 * e] << 16) * inv, x1 = __uint_as_float(w[2 * e] & 0xffff0000u) * inv;
    const float x2 = __uint_as_float(w[2 * e + 1] << 16) * inv, x3 = __uint_as_float(w[2 * e + 1] & 0xffff0000u) * inv;
    hi[e] = e4m3x4(x0, x1, x2, x3);
    const float2 b0 = e4m3x2_f(hi[e]), b1 = e4m3x2_f(hi[e] >> 16);
    lo[e] = e4m3x4((x0 - b0.x) * 16.f, (x1 - b0.y) * 16.f, (x2 - b1.x) * 16.f, (x3 - b1.y) * 16.f);
  }
  uint4* dst = reinterpret_cast<uint4*>(a.q8) + ((size_t)q * 32 + lane) * 128 + 32 * (h >> 4) + (h & 15);
  dst[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  dst[16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  // what a product of the parts stands for: 2^e, and the softmax scale with it
  if (lane == 0) a.q8_scale[row] = be == 255 ? NAN : __uint_as_float((uint32_t)(be - 7) << 23) * a.scale2;
}

__global__ void __launch_bounds__(kPlanThreads) k_plan_pages(const __grid_constant__ PagedArgs a) {
  pdl_trigger();  // (the attention kernel alone follows, and waits)
  __shared__ int sm[kPlanThreads / 32];
  pdl_wait();
  if (blockIdx.x == gridDim.x - 1) {
    make_plan(a, sm);
    return;
  }
  const int row = blockIdx.x * (kPlanThreads / 32) + (threadIdx.x >> 5);
  if (row < a.B * a.T * 64) split_query_row(a, row);
}

// ---------------------------------------------------------------- the portable kernel
constexpr int kSimtTile = 32;   // keys a tile: a lane each
constexpr int kSimtWarps = 8;   // heads at a time, a warp each
constexpr int kSimtMaxC = 4;    // chunks of 8 dims a lane: D <= 1024
constexpr int kSimtPad = 4;     // floats behind a key's row: lanes read their keys' chunks without bank conflicts
constexpr int kSimtSmemMax = (kSimtTile * (1024 + kSimtPad) + kSimtWarps * 1024) * 4;

__host__ __device__ constexpr int simt_smem(int D) { return (kSimtTile * (D + kSimtPad) + kSimtWarps * D) * 4; }

template <typename T>
__global__ void __launch_bounds__(32 * kSimtWarps) k_attend_pages_simt(const __grid_constant__ PagedArgs a) {
  pdl_trigger();  // (the merge alone follows, and waits)
  extern __shared__ __align__(16) float sm_pa[];
  __shared__ int s_row[kSimtTile];
  const int D = a.D, KS = D + kSimtPad, n8 = D >> 3;
  float* ks = sm_pa;                    // [kSimtTile][KS] keys
  float* qs = sm_pa + kSimtTile * KS;   // [kSimtWarps][D] queries of this group of heads
  pdl_wait();
  const PagedRun* run = a.runs + blockIdx.x;
  const int4 r4 = *reinterpret_cast<const int4*>(run);
  const int t0 = r4.x, t1 = r4.y;
  int pre = r4.z;
  if (t0 >= t1) return;
  PagedQuery k = load_query(&run->k);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll 1
  while (true) {
    const int q = k.q, b = q / a.T;
    const int begin = max(t0 - pre, 0), end = min(t1 - pre, k.tiles), nkeys = k.n0 + k.f + k.nw;
    const bool whole = begin == 0 && end == k.tiles;
    const int slot = 2 * blockIdx.x + (begin == 0 ? 1 : 0);
#pragma unroll 1
    for (int h0 = 0; h0 < a.H && begin < end; h0 += kSimtWarps) {
      const int h = h0 + warp;
      __syncthreads();
      for (int e = tid; e < kSimtWarps * n8; e += blockDim.x) {
        const int hh = e / n8, c = (e - hh * n8) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (h0 + hh < a.H) load8(static_cast<const T*>(a.q) + ((size_t)q * a.H + h0 + hh) * D + c, v);
        store8(qs + hh * D + c, v);
      }
      float m = -INFINITY, l = 0.f;
      float acc[kSimtMaxC][8];
#pragma unroll
      for (int c = 0; c < kSimtMaxC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[c][e] = 0.f;
#pragma unroll 1
      for (int t = begin; t < end; ++t) {
        const int k0 = t * kSimtTile, nk = min(kSimtTile, nkeys - k0);
        __syncthreads();
        if (tid < kSimtTile) {
          const int x = k0 + tid;
          int r = -1;
          if (x < k.n0) {
            const int j = a.sel ? __ldg(a.sel + (size_t)q * a.topk + x) : x;
            if (!a.sel || (j >= 0 && j < k.n_rows)) r = paged_row(a.row_table, a.row_pages, b, j, a.P, a.n_pages);
          } else if (x < nkeys) {
            const int y = x - k.n0;
            r = paged_row(a.token_table, a.token_pages, b, y < k.f ? y : k.w0 + (y - k.f), a.P, a.n_pages);
          }
          if (r < 0 && x < nkeys) atomicOr(a.err, CSA_DEV_RANGE);
          s_row[tid] = r;
        }
        __syncthreads();
        for (int e = tid; e < kSimtTile * n8; e += blockDim.x) {
          const int x = e / n8, c = (e - x * n8) * 8, r = s_row[x];
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (r >= 0) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(a.codes + (size_t)r * D + c));
            const float s = __ldg(a.scales + r);
            const float2 f[4] = {e4m3x2_f(u.x), e4m3x2_f(u.x >> 16), e4m3x2_f(u.y), e4m3x2_f(u.y >> 16)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[2 * i] = f[i].x * s;
              v[2 * i + 1] = f[i].y * s;
            }
          }
          store8(ks + x * KS + c, v);
        }
        __syncthreads();
        float dot = 0.f;
        const bool on = lane < nk && s_row[lane] >= 0;
        if (on) {
          const float* kr = ks + lane * KS;
          const float* qh = qs + warp * D;
          for (int c = 0; c < D; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(kr + c), y = *reinterpret_cast<const float4*>(qh + c);
            dot = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, dot))));
          }
        }
        const float lg = on ? dot * a.scale2 : -INFINITY;
        const float mn = fmaxf(m, warp_max(lg)), ref = mn == -INFINITY ? 0.f : mn;
        const float p = exp2f(lg - ref), f = exp2f(m - ref);
        l = fmaf(l, f, warp_sum(p));
        m = mn;
#pragma unroll
        for (int c = 0; c < kSimtMaxC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[c][e] *= f;
        for (int x = 0; x < nk; ++x) {
          const float px = __shfl_sync(0xffffffffu, p, x);
          const float* kr = ks + x * KS;
#pragma unroll
          for (int c = 0; c < kSimtMaxC; ++c) {
            if (lane + 32 * c < n8) {
              float v[8];
              load8(kr + 8 * (lane + 32 * c), v);
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[c][e] = fmaf(px, v[e], acc[c][e]);
            }
          }
        }
      }
      if (h >= a.H) continue;
      if (!whole) {
        const size_t at = (size_t)slot * a.H + h;
        if (lane == 0) a.ml[at] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < kSimtMaxC; ++c)
          if (lane + 32 * c < n8) store8(a.part + at * D + 8 * (lane + 32 * c), acc[c]);
        continue;
      }
      const float z2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
      const float M = fmaxf(m, z2), f = m == -INFINITY ? 0.f : exp2f(m - M);
      const float Z = l * f + (z2 == -INFINITY ? 0.f : exp2f(z2 - M));
      const float w = Z == 0.f ? 0.f : f / Z;  // (no key and no sink: zeros)
#pragma unroll
      for (int c = 0; c < kSimtMaxC; ++c) {
        const int d = 8 * (lane + 32 * c);
        if (d >= D) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[c][e] * w;
        if (a.inv_freq && d >= D - a.R) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float cs, sn;
            rope_cs(k.p, a.inv_freq, (d + e - (D - a.R)) >> 1, &cs, &sn);
            const float x0 = v[e], x1 = v[e + 1];
            v[e] = fmaf(x0, cs, x1 * sn);
            v[e + 1] = fmaf(-x0, sn, x1 * cs);
          }
        }
        store8(static_cast<T*>(a.out) + ((size_t)q * a.H + h) * D + d, v);
      }
    }
    pre += k.tiles;
    if (pre >= t1) return;
    k = load_query(a.queries + q + 1);
  }
}

// ---------------------------------------------------------------- merge of split queries
// With (m_s, l_s, acc_s) of the parts: M = max(z, m_s), Z = 2^{z - M} + sum_s l_s 2^{m_s - M},
// o = sum_s acc_s 2^{m_s - M} / Z (z the sink in powers of two).  A block of eight warps takes one head of a query (few
// queries: each has many parts) or eight; a head's warps take its parts in turn.  The weights are found first, from all
// parts' statistics at once, so that the sum over the accumulators is loads and products only, eight in flight.
constexpr int kMergeC = 8;       // 4-value columns a lane holds, 128 values apart: D <= 1024
constexpr int kMergeWarps = 8;

template <typename T, int kC>
__global__ void __launch_bounds__(32 * kMergeWarps) k_merge_pages(const __grid_constant__ PagedArgs a, int heads) {
  // no early trigger: what follows finds the outputs written
  extern __shared__ __align__(16) float sm_merge[];  // [kMergeWarps][kPagedBlocks] weights; heads == 1: [kMergeWarps][D] sums
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n4 = a.D >> 2;
  const int hh = heads == 1 ? 0 : warp, h = blockIdx.y * heads + hh;
  const int first = heads == 1 ? warp : 0, step = heads == 1 ? kMergeWarps : 1;
  float* wt = sm_merge + warp * kPagedBlocks;  // (a query has at most a part in every block)
  float4* sums = reinterpret_cast<float4*>(sm_merge + kMergeWarps * kPagedBlocks);
#pragma unroll 1
  for (int q = blockIdx.x; q < a.B * a.T; q += gridDim.x) {
    const int2 at = a.parts[q];
    if (at.y <= 1) continue;
    const bool on = h < a.H;
    float inv = 0.f;
    if (heads == 1) __syncthreads();  // (the query before has been read)
    if (on) {
      // every warp of a head finds all weights
      const float z2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
      float M = z2;
      for (int s = lane; s < at.y; s += 32) M = fmaxf(M, a.ml[(size_t)(2 * (at.x + s) + (s == 0)) * a.H + h].x);
      M = warp_max(M);
      float Z = 0.f;
      for (int s = lane; s < at.y; s += 32) {
        const float2 ml = a.ml[(size_t)(2 * (at.x + s) + (s == 0)) * a.H + h];
        const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);  // (a part without keys)
        wt[s] = f;
        Z = fmaf(ml.y, f, Z);
      }
      Z = warp_sum(Z) + (z2 == -INFINITY ? 0.f : exp2f(z2 - M));
      inv = Z == 0.f ? 0.f : 1.f / Z;
    }
    __syncwarp();
    float4 acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      constexpr int kAhead = kC <= 4 ? 4 : 2;
      for (int s0 = first; s0 < at.y; s0 += kAhead * step) {
        float4 x[kAhead][kC];
        float f[kAhead];
#pragma unroll
        for (int g = 0; g < kAhead; ++g) {
          const int s = min(s0 + g * step, at.y - 1);
          f[g] = s0 + g * step < at.y ? wt[s] : 0.f;
          const float* src = a.part + (size_t)(2 * (at.x + s) + (s == 0)) * a.H * a.D;
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int d = 4 * (lane + 32 * c), blk = a.cols == 128 ? c : 0;
            if (lane + 32 * c < n4)
              x[g][c] = __ldcg(reinterpret_cast<const float4*>(src + ((size_t)blk * a.H + h) * a.cols + (d - blk * 128)));
          }
        }
#pragma unroll
        for (int g = 0; g < kAhead; ++g) {
          if (f[g] == 0.f) continue;  // (what a part without keys holds counts for nothing)
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            if (lane + 32 * c < n4) {
              acc[c].x = fmaf(x[g][c].x, f[g], acc[c].x);
              acc[c].y = fmaf(x[g][c].y, f[g], acc[c].y);
              acc[c].z = fmaf(x[g][c].z, f[g], acc[c].z);
              acc[c].w = fmaf(x[g][c].w, f[g], acc[c].w);
            }
          }
        }
      }
    }
    if (heads == 1) {
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (lane + 32 * c < n4) sums[warp * n4 + lane + 32 * c] = acc[c];
      __syncthreads();
    }
    if (!on) continue;
    const int p = a.pos[q / a.T] + q % a.T;
    // a head's columns: by its warp from registers, or over the block's warps from their sums
    for (int c = 0; c < kC; ++c) {
      const int col = heads == 1 ? (int)threadIdx.x + 256 * c : lane + 32 * c;
      if (col >= n4) break;
      float4 v4;
      if (heads == 1) {
        v4 = sums[col];
        for (int w = 1; w < kMergeWarps; ++w) {
          const float4 x = sums[w * n4 + col];
          v4.x += x.x; v4.y += x.y; v4.z += x.z; v4.w += x.w;
        }
      } else {
        v4 = acc[0];
#pragma unroll
        for (int e = 1; e < kC; ++e)
          if (e == c) v4 = acc[e];
      }
      const int d = 4 * col;
      float v[4] = {v4.x * inv, v4.y * inv, v4.z * inv, v4.w * inv};
      if (a.inv_freq && d >= a.D - a.R) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float cs, sn;
          rope_cs(p, a.inv_freq, (d + e - (a.D - a.R)) >> 1, &cs, &sn);
          const float x0 = v[e], x1 = v[e + 1];
          v[e] = fmaf(x0, cs, x1 * sn);
          v[e + 1] = fmaf(-x0, sn, x1 * cs);
        }
      }
      T* o = static_cast<T*>(a.out) + ((size_t)q * a.H + h) * a.D + d;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = from_f<T>(v[e]);
    }
  }
}

template <typename T, int kC>
cudaError_t merge_c(const PagedArgs& a, cudaStream_t s) {
  const int Q = a.B * a.T;
  const int heads = Q <= 8 ? 1 : kMergeWarps;
  const int smem = (kMergeWarps * kPagedBlocks + (heads == 1 ? kMergeWarps * a.D : 0)) * 4;
  CSA_LAUNCH((k_merge_pages<T, kC>), dim3(min(Q, 4 * kPagedBlocks), (a.H + heads - 1) / heads), dim3(32 * kMergeWarps),
             smem, s, a, heads);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_merge(const PagedArgs& a, cudaStream_t s) {
  return a.D <= 128 ? merge_c<T, 1>(a, s) : a.D <= 512 ? merge_c<T, 4>(a, s) : merge_c<T, kMergeC>(a, s);
}

template <typename T>
cudaError_t attend_t(const Dims& L, PagedArgs a, cudaStream_t s) {
  const int Q = a.B * a.T;
  if (tc_paged_supported(L, a.P)) {
    a.tile = 64;
    a.shift = 3;  // the largest power of two that divides a page, at most a tile
    while (a.shift < 6 && a.P % (2 << a.shift) == 0) ++a.shift;
    a.min_tiles = 2;
    a.cols = 128;
    CSA_LAUNCH(k_plan_pages, dim3(Q * 64 / (kPlanThreads / 32) + 1), dim3(kPlanThreads), 0, s, a);
    const cudaError_t e = launch_tc_paged(a, s);
    if (e != cudaSuccess) return e;
  } else {
    a.tile = kSimtTile;
    a.shift = 0;
    a.min_tiles = 2;
    a.cols = a.D;
    CSA_LAUNCH(k_plan_pages, dim3(1), dim3(kPlanThreads), 0, s, a);
    allow_smem<kSimtSmemMax>(k_attend_pages_simt<T>);
    CSA_LAUNCH(k_attend_pages_simt<T>, dim3(kPagedBlocks), dim3(32 * kSimtWarps), simt_smem(a.D), s, a);
  }
  return launch_merge<T>(a, s);
}

}  // namespace

void carve_paged(Carver& c, const Dims& L, int Q, PagedArgs* a) {
  a->runs = c.take<PagedRun>(kPagedBlocks);
  a->queries = c.take<PagedQuery>(Q);
  a->parts = c.take<int2>(Q);
  a->ml = c.take<float2>((size_t)2 * kPagedBlocks * L.H);
  a->part = c.take<float>((size_t)2 * kPagedBlocks * L.H * L.D);
  if (tc_paged_supported(L, 8)) {
    a->q8 = c.take<uint8_t>((size_t)Q * 64 * 1024);
    a->q8_scale = c.take<float>((size_t)Q * 64);
  }
}

cudaError_t launch_attend_pages(const Dims& L, PagedArgs a, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? attend_t<__nv_bfloat16>(L, a, s) : attend_t<float>(L, a, s);
}

}  // namespace csa
