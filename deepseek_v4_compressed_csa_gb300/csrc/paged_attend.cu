// Attention over a cache in pages and 8 bits: the portable kernel (any head layout and size, bf16 and fp32), and the merge
// of queries that several blocks worked on.
//
//   l_k = scale q_h . key_k;  o_h = sum_k e^{l_k} key_k / (e^{sink_h} + sum_k e^{l_k});  out_h = RoPE^-1(o_h, p)
//
// over the keys of PagedQuery, key_k = scale_k code_k.  A block walks its run of tiles (paged.cuh) with a running maximum
// and sum per head; all arithmetic in fp32, the output rounded once.
#include <algorithm>

#include "paged.cuh"
#include "tc.cuh"

namespace csa {

namespace {

// ---------------------------------------------------------------- the portable kernel
// A tile's keys wait in shared memory as fp32; the next tile's codes are on their way in registers meanwhile, and the rows
// of the one after it are looked up.  A warp takes kN heads and 32 of the tile's 32 kN keys: a lane a key for the logits,
// then lanes share a key's dims (rows of up to 128 dims: several keys at a time) for the sums; the warps of a head are put
// together behind the last tile.  What bounds it is reading the keys from shared memory, twice a head: 60 queries of 1K keys
// (8 heads of 64 dims) take 38 us with a warp a head, 28 with a warp two, 23.5 with four.  But where a block has few tiles,
// most warps have no keys with four: one to three tiles (a window of 32) 6.4 us with two heads a warp, 7.0 with four, 6.8
// with one; one tile (15 queries of 250 keys, cut) 8.7 with one, 9.0 with two, 9.7 with four.
constexpr int kSimtWarps = 8;   // and heads at a time
constexpr int kSimtPad = 4;     // floats behind a key's row: lanes read their keys' chunks without bank conflicts
__host__ __device__ constexpr int simt_heads(int chunks) { return 4 / chunks; }  // the most heads a warp, and tiles at once
__host__ __device__ constexpr int simt_chunks(int D) { return D <= 256 ? 1 : D <= 512 ? 2 : 4; }
__host__ __device__ constexpr int simt_smem(int D) {
  return (32 * simt_heads(simt_chunks(D)) * (D + kSimtPad) + kSimtWarps * D) * 4;
}
constexpr int kSimtSmemMax = simt_smem(1024);
static_assert(simt_smem(256) <= kSimtSmemMax && simt_smem(512) <= kSimtSmemMax && kSimtSmemMax <= 232448, "shared memory");

// kC: chunks of 8 dims a lane holds (D <= 256 kC)
template <typename T, int kC, int kN>
__global__ void __launch_bounds__(32 * kSimtWarps, 1) k_attend_pages_simt(const __grid_constant__ PagedArgs a) {
  if (a.merge) pdl_trigger();  // (what follows otherwise finds the outputs written)
  extern __shared__ __align__(16) float sm_pa[];
  constexpr int kTile = 32 * kN;  // kN tiles of the plan at once
  __shared__ int s_row[2][kTile];
  __shared__ float2 s_ml[kN * kSimtWarps];
  __shared__ __align__(16) int s_plan[kPlanInts];
  __shared__ PagedRun s_run;
  constexpr int kPass = kTile / kSimtWarps;  // rows of a tile a thread copies (one of kC chunks of) at most
  const int D = a.D, KS = D + kSimtPad, n8 = D >> 3;
  float* ks = sm_pa;                    // [kTile][KS] keys
  float* qs = sm_pa + kTile * KS;       // [kSimtWarps][D] queries of this group of heads
  pdl_wait();
  paged_plan<kSimtWarps>(a, &s_run, s_plan);
  const int t0 = s_run.t0, t1 = s_run.t1;
  if (t0 >= t1) return;
  int pre = s_run.pre;
  PagedQuery k = s_run.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // lanes that share a key's dims, and keys at a time
  int share = 32;
  while (share > 1 && share / 2 >= n8) share /= 2;
  const int sub = lane & (share - 1), group = lane / share, groups = 32 / share;
  const int head0 = warp % (kSimtWarps / kN) * kN, key0 = warp / (kSimtWarps / kN) * 32;  // the warp's heads and keys
  const int row0 = warp * groups + group, rows = kSimtWarps * groups;  // rows that the block copies at once, and the lane's
#pragma unroll 1
  while (true) {
    const int q = k.q, b = k.b;
    const int begin = max(t0 - pre, 0), end = min(t1 - pre, k.tiles), stop = min(k.n0 + k.f + k.nw, 32 * end);
    const bool whole = begin == 0 && end == k.tiles;
    const int slot = 2 * blockIdx.x + (begin == 0 ? 1 : 0);
    if (begin == 0 && !whole && a.inv_freq)  // (for the merge: an angle costs a lane some hundred instructions)
      for (int i = tid; i < a.R / 2; i += blockDim.x) {
        float2 t;
        turn_cs(k.p, __ldg(a.inv_freq + i), &t.x, &t.y);
        a.turns[(size_t)blockIdx.x * (a.R / 2) + i] = t;
      }
    // key x of the query: its physical row, -1 for none (a thread a key of a tile)
    auto row_of = [&](int x) {
      if (x >= stop) return -1;
      int r = -1;
      if (x < k.n0) {
        const int j = a.sel ? __ldg(a.sel + (size_t)q * a.topk + x) : x;
        if (!a.sel || (j >= 0 && j < k.n_rows)) r = paged_row(a, a.row_table + (size_t)b * a.row_pages, j);
      } else {
        const int y = x - k.n0;
        r = paged_row(a, a.token_table + (size_t)b * a.token_pages, y < k.f ? y : k.w0 + (y - k.f));
      }
      if (r < 0) atomicOr(a.err, CSA_DEV_RANGE);
      return r;
    };
#pragma unroll 1
    for (int h0 = 0; h0 < a.H; h0 += kSimtWarps) {
      const int h = h0 + warp;
      __syncthreads();
      for (int e = tid; e < kSimtWarps * n8; e += blockDim.x) {
        const int hh = e / n8, c = (e - hh * n8) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (h0 + hh < a.H) load8(static_cast<const T*>(a.q) + ((size_t)q * a.H + h0 + hh) * D + c, v);
        store8(qs + hh * D + c, v);
      }
      if (tid < kTile) s_row[0][tid] = row_of(begin * 32 + tid);
      __syncthreads();
      uint2 code[kPass][kC];
      float scale[kPass];
      auto fetch = [&](int t, int buf) {  // the codes of the tiles from t on, whose rows are there
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
          if (row0 + i * rows >= min(kTile, 32 * (end - t))) break;
          const int r = s_row[buf][row0 + i * rows];
          scale[i] = r >= 0 ? __ldg(a.scales + r) : 0.f;
#pragma unroll
          for (int c = 0; c < kC; ++c)
            code[i][c] = r >= 0 && sub + 32 * c < n8
                             ? __ldg(reinterpret_cast<const uint2*>(a.codes + (size_t)r * D + 8 * (sub + 32 * c)))
                             : make_uint2(0u, 0u);
        }
      };
      fetch(begin, 0);
      float ms[kN], ls[kN], sums[kN][kC][8];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        ms[n] = -INFINITY;
        ls[n] = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) sums[n][c][e] = 0.f;
      }
#pragma unroll 1
      for (int t = begin, buf = 0; t < end; t += kN, buf ^= 1) {
        if (tid < kTile && t + kN < end) s_row[buf ^ 1][tid] = row_of((t + kN) * 32 + tid);
        __syncthreads();  // (the tiles before have been read; the next ones' rows are there)
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
          if (row0 + i * rows >= min(kTile, 32 * (end - t))) break;
          const float s = scale[i];
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            if (sub + 32 * c >= n8) continue;
            const uint2 u = code[i][c];
            const float2 f[4] = {e4m3x2_f(u.x), e4m3x2_f(u.x >> 16), e4m3x2_f(u.y), e4m3x2_f(u.y >> 16)};
            const float v[8] = {f[0].x * s, f[0].y * s, f[1].x * s, f[1].y * s, f[2].x * s, f[2].y * s, f[3].x * s, f[3].y * s};
            store8(ks + (row0 + i * rows) * KS + 8 * (sub + 32 * c), v);
          }
        }
        const bool on = s_row[buf][key0 + lane] >= 0;
        if (t + kN < end) fetch(t + kN, buf ^ 1);
        __syncthreads();
        const int nk = min(32, stop - t * 32 - key0);  // (rows behind the last hold zeros, and p is 0)
        if (nk <= 0) continue;
        float d2[kN][2];
#pragma unroll
        for (int n = 0; n < kN; ++n) d2[n][0] = d2[n][1] = 0.f;
        {
          const float* kr = ks + (key0 + lane) * KS;
          const float* qh = qs + head0 * D;
#pragma unroll 4
          for (int c = 0; c < D; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(kr + c);
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              const float4 y = *reinterpret_cast<const float4*>(qh + n * D + c);
              d2[n][0] = fmaf(x.x, y.x, d2[n][0]);
              d2[n][1] = fmaf(x.y, y.y, d2[n][1]);
              d2[n][0] = fmaf(x.z, y.z, d2[n][0]);
              d2[n][1] = fmaf(x.w, y.w, d2[n][1]);
            }
          }
        }
        float p[kN];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          p[n] = on ? (d2[n][0] + d2[n][1]) * a.scale2 : -INFINITY;
          const float mn = fmaxf(ms[n], warp_max(p[n])), ref = mn == -INFINITY ? 0.f : mn, f = exp2f(ms[n] - ref);
          p[n] = exp2f(p[n] - ref);
          ls[n] = fmaf(ls[n], f, warp_sum(p[n]));
          ms[n] = mn;
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) sums[n][c][e] *= f;
        }
#pragma unroll 2
        for (int x0 = 0; x0 < nk; x0 += groups) {
          const float* kr = ks + (key0 + x0 + group) * KS;
          float px[kN];
#pragma unroll
          for (int n = 0; n < kN; ++n) px[n] = __shfl_sync(0xffffffffu, p[n], x0 + group);
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            if (sub + 32 * c < n8) {
              float v[8];
              load8(kr + 8 * (sub + 32 * c), v);
#pragma unroll
              for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[n][c][e] = fmaf(px[n], v[e], sums[n][c][e]);
            }
          }
        }
      }
      // ---- the parts of a head: of the lanes that took other keys, then of the warps, through the tile's memory
      for (int o = share; o < 32; o <<= 1)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 8; ++e) sums[n][0][e] += __shfl_xor_sync(0xffffffffu, sums[n][0][e], o);
      float m = ms[0], l = ls[0], acc[kC][8];
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[c][e] = sums[0][c][e];
      if (kN > 1) {
        __syncthreads();  // (the last tile has been read)
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int at = key0 / 32 * kSimtWarps + head0 + n;  // [kN][kSimtWarps] parts
          if (lane == 0) s_ml[at] = make_float2(ms[n], ls[n]);
#pragma unroll
          for (int c = 0; c < kC; ++c)
            if (group == 0 && sub + 32 * c < n8) store8(ks + at * D + 8 * (sub + 32 * c), sums[n][c]);
        }
        __syncthreads();
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i) m = fmaxf(m, s_ml[i * kSimtWarps + warp].x);
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[c][e] = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float2 part = s_ml[i * kSimtWarps + warp];
          // (a part without keys has m = -inf and zeros, but for a NaN that it may hold)
          const float f = part.x == -INFINITY ? 1.f : exp2f(part.x - m);
          l = fmaf(part.y, f, l);
#pragma unroll
          for (int c = 0; c < kC; ++c)
            if (sub + 32 * c < n8) {
              float v[8];
              load8(ks + (i * kSimtWarps + warp) * D + 8 * (sub + 32 * c), v);
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[c][e] = fmaf(v[e], f, acc[c][e]);
            }
        }
      }
      if (h >= a.H || group > 0) continue;
      if (!whole) {
        const size_t at = (size_t)slot * a.H + h;
        if (lane == 0) a.ml[at] = make_float2(l == l ? m : l, l);  // (a NaN is one for the merge, too)
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (sub + 32 * c < n8) store8(a.part + at * D + 8 * (sub + 32 * c), acc[c]);
        continue;
      }
      const float z2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
      const float M = fmaxf(m, z2), f = m == -INFINITY ? 0.f : exp2f(m - M);
      const float Z = l * f + (z2 == -INFINITY ? 0.f : exp2f(z2 - M));
      const float w = Z == 0.f ? 0.f : f / Z;  // (no key and no sink: zeros)
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int d = 8 * (sub + 32 * c);
        if (d >= D) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[c][e] * w;
        if (a.inv_freq && d >= D - a.R) {
#pragma unroll 1
          for (int e = 0; e < 8; e += 2) {
            float cs, sn;
            turn_cs(k.p, __ldg(a.inv_freq + ((d + e - (D - a.R)) >> 1)), &cs, &sn);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              if (i != e) continue;
              const float x0 = v[i], x1 = v[i + 1];
              v[i] = fmaf(x0, cs, x1 * sn);
              v[i + 1] = fmaf(-x0, sn, x1 * cs);
            }
          }
        }
        store8(static_cast<T*>(a.out) + ((size_t)q * a.H + h) * D + d, v);
      }
    }
    pre += k.tiles;
    if (pre >= t1) return;
    k = next_query(a, q);
  }
}

template <typename T, int kC, int kN>
cudaError_t simt_c(const PagedArgs& a, cudaStream_t s) {
  allow_smem<kSimtSmemMax>(k_attend_pages_simt<T, kC, kN>);
  CSA_LAUNCH((k_attend_pages_simt<T, kC, kN>), dim3(kPagedBlocks), dim3(32 * kSimtWarps), simt_smem(a.D), s, a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- merge of split queries
// With (m_s, l_s, acc_s) of the parts: M = max(z, m_s), Z = 2^{z - M} + sum_s l_s 2^{m_s - M},
// o = sum_s acc_s 2^{m_s - M} / Z (z the sink in powers of two).  An item is 128 kC values of a head of a split query, 4 kC
// a lane; `share` warps take its parts in turn (one query of 129 parts, 17 MB: some 6 us).  What the kernel waits for is memory, two round trips (where the parts are; their
// statistics and the first accumulators together), if it has few enough instructions beside its loads (128 values an item
// cost 1500 a warp, 8.7 us for 8 queries of 18 parts) and blocks: one started a head of every query cost 8 us on 128 queries
// of which none was split.  So a block finds the split queries itself and walks their items, one in most calls: all
// accumulators of 8 queries or of one long one fit the device's registers.
constexpr int kMergeWarps = 8;
// Parts in flight a warp, 4 chunks registers each: all that a long query's warp has to take (the first of a second round
// cost 2 us), or as many as fit the registers of two blocks an SM
__host__ __device__ constexpr int merge_ahead(int chunks) { return chunks == 1 ? kPagedBlocks / kMergeWarps : 10; }

template <typename T, int kC>
__global__ void __launch_bounds__(32 * kMergeWarps, 2) k_merge_pages(const __grid_constant__ PagedArgs a, int share) {
  // no early trigger: what follows finds the outputs written
  // split queries: q, block of the first part, parts (at least two of the blocks each)
  __shared__ int4 s_list[kMergeWarps][kPagedBlocks];
  __shared__ int s_count[kMergeWarps];
  __shared__ float4 s_acc[kMergeWarps][32 * kC];
  __shared__ float s_wt[kMergeWarps][kPagedBlocks];  // weights of a warp's item's parts
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, Q = a.B * a.T;
  int n_split = 0;
  if (Q <= 32) {  // every warp writes the same list, its own for all it reads: no barrier
    const int2 at = lane < Q ? __ldcg(a.parts + lane) : make_int2(0, 0);
    const uint32_t on = __ballot_sync(0xffffffffu, at.y > 1);
    n_split = __popc(on);
    if (at.y > 1) s_list[warp][__popc(on & ((1u << lane) - 1))] = make_int4(lane, at.x, at.y, 0);
    __syncwarp();
  } else {
    for (int q0 = 0; q0 < Q; q0 += 32 * kMergeWarps) {
      const int2 at = q0 + tid < Q ? __ldcg(a.parts + q0 + tid) : make_int2(0, 0);
      const uint32_t on = __ballot_sync(0xffffffffu, at.y > 1);
      if (lane == 0) s_count[warp] = __popc(on);
      __syncthreads();
      int before = n_split;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        before += w < warp ? s_count[w] : 0;
        n_split += s_count[w];
      }
      if (at.y > 1) s_list[0][before + __popc(on & ((1u << lane) - 1))] = make_int4(q0 + tid, at.x, at.y, 0);
      __syncthreads();
    }
  }
  const int4* list = s_list[Q <= 32 ? warp : 0];
  const int chunks = (a.D + 128 * kC - 1) / (128 * kC), items = n_split * a.H * chunks, per = kMergeWarps / share;
  constexpr int kAhead = merge_ahead(kC), kL = (kPagedBlocks + 31) / 32;
  const int first = warp % share;
#pragma unroll 1
  for (int i0 = blockIdx.x * per; i0 < items; i0 += gridDim.x * per) {
    const int item = min(i0 + warp / share, items - 1);  // (a warp behind the last repeats it)
    const int hq = item / chunks, lq = hq / a.H, h = hq - lq * a.H, d0 = 128 * kC * (item - hq * chunks) + 4 * lane;
    const int4 at = list[lq];
    // part s of the query: slot 2 (block + s), the first one the slot behind; a lane's columns: 4 values, 128 apart
    const size_t one = (size_t)a.H * a.D, step = 2 * one * share;
    const float* src = a.part + 2 * one * (at.y + first) + (first == 0 ? one : 0);
    size_t off[kC];
    bool on[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int d = d0 + 128 * c, blk = a.cols == a.D ? 0 : d >> 5;  // (blocks of 32 dims, or all)
      on[c] = d < a.D;
      off[c] = ((size_t)blk * a.H + h) * a.cols + (d - blk * 32);
    }
    float4 x[kAhead][kC];
    auto fetch = [&](int s0, const float* p) {
#pragma unroll
      for (int g = 0; g < kAhead; ++g) {
        if (s0 + g * share < at.z) {
#pragma unroll
          for (int c = 0; c < kC; ++c)
            if (on[c]) x[g][c] = __ldcg(reinterpret_cast<const float4*>(p + off[c]));
        }
        p += s0 + g * share == 0 ? step - one : step;
      }
      return p;
    };
    const float2* stat = a.ml + (size_t)2 * at.y * a.H + h;
    float2 ml[kL];  // (all at once)
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const int s = lane + 32 * i;
      ml[i] = s < at.z ? __ldcg(stat + (size_t)2 * s * a.H + (s == 0 ? a.H : 0)) : make_float2(-INFINITY, 0.f);
    }
    src = fetch(first, src);
    // the weights (every warp of an item finds them)
    const float z2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
    float M = z2, Z = 0.f;
#pragma unroll
    for (int i = 0; i < kL; ++i) M = fmaxf(M, ml[i].x);
    M = warp_max(M);
    float* wt = s_wt[warp];
    __syncwarp();  // (the weights of the item before have been read)
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      if (32 * i >= at.z) break;
      const float f = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - M);  // (a part without keys)
      if (lane + 32 * i < at.z) wt[lane + 32 * i] = f;
      Z = fmaf(ml[i].y, f, Z);
    }
    Z = warp_sum(Z) + (z2 == -INFINITY ? 0.f : exp2f(z2 - M));
    __syncwarp();
    float4 acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s0 = first; s0 < at.z; s0 += kAhead * share) {
      if (s0 > first) src = fetch(s0, src);
#pragma unroll
      for (int g = 0; g < kAhead; ++g) {
        const int s = s0 + g * share;
        const float f = s < at.z ? wt[s] : 0.f;
        if (f == 0.f) continue;  // (what a part without keys holds counts for nothing)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          acc[c].x = fmaf(x[g][c].x, f, acc[c].x);
          acc[c].y = fmaf(x[g][c].y, f, acc[c].y);
          acc[c].z = fmaf(x[g][c].z, f, acc[c].z);
          acc[c].w = fmaf(x[g][c].w, f, acc[c].w);
        }
      }
    }
    if (share > 1) {
      __syncthreads();  // (the items before have been read)
#pragma unroll
      for (int c = 0; c < kC; ++c) s_acc[warp][lane + 32 * c] = acc[c];
      __syncthreads();
      if (first != 0) continue;
      for (int g = 1; g < share; ++g)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const float4 v = s_acc[warp + g][lane + 32 * c];
          acc[c].x += v.x; acc[c].y += v.y; acc[c].z += v.z; acc[c].w += v.w;
        }
    }
    const float inv = Z == 0.f ? 0.f : 1.f / Z;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if (!on[c]) continue;
      const int d = d0 + 128 * c;
      float v[4] = {acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv};
      if (a.inv_freq && d >= a.D - a.R) {
        const float4 t = __ldcg(reinterpret_cast<const float4*>(a.turns + (size_t)at.y * (a.R / 2) + ((d - (a.D - a.R)) >> 1)));
        const float x0 = v[0], x2 = v[2];
        v[0] = fmaf(x0, t.x, v[1] * t.y);
        v[1] = fmaf(-x0, t.y, v[1] * t.x);
        v[2] = fmaf(x2, t.z, v[3] * t.w);
        v[3] = fmaf(-x2, t.w, v[3] * t.z);
      }
      T* o = static_cast<T*>(a.out) + ((size_t)at.x * a.H + h) * a.D + d;
      if constexpr (sizeof(T) == 2) {
        uint2 u;
        reinterpret_cast<__nv_bfloat162*>(&u)[0] = __floats2bfloat162_rn(v[0], v[1]);
        reinterpret_cast<__nv_bfloat162*>(&u)[1] = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(o) = u;
      } else {
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

template <typename T, int kC>
cudaError_t merge_c(const PagedArgs& a, cudaStream_t s) {
  const int Q = a.B * a.T;
  // few queries have many parts each (about blocks / queries): as many warps share an item as take them at once, while the
  // items find room on the device at once (two blocks an SM)
  const long long items = (long long)min(Q, kPagedBlocks) * a.H * ((a.D + 128 * kC - 1) / (128 * kC)), room = 2LL * kPagedBlocks;
  int share = 1;
  while (share < kMergeWarps && share * merge_ahead(kC) * Q < kPagedBlocks && 2 * share * items <= room * kMergeWarps) share *= 2;
  const long long per = kMergeWarps / share;
  CSA_LAUNCH((k_merge_pages<T, kC>), dim3((unsigned)min((items + per - 1) / per, room)), dim3(32 * kMergeWarps),
             0, s, a, share);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_merge(const PagedArgs& a, cudaStream_t s) {
  // items enough for every SM: a quarter of the Flash row's values for up to four queries, else half
  return a.D <= 128 || a.B * a.T <= 4 ? merge_c<T, 1>(a, s) : merge_c<T, 2>(a, s);
}

// The most tiles that a query of the call may have, by what its sizes say
long long most_tiles(const PagedArgs& a) {
  const long long u = 1 << a.shift, per = a.tile >> a.shift;
  long long n = 0, runs = 0;
  if (a.sel) n += (a.topk + a.tile - 1) / a.tile;
  else if (a.row_table) runs += ((long long)a.row_pages * a.P + u - 1) / u;
  if (a.token_table) {
    const long long room = (long long)a.token_pages * a.P, f = a.first < room ? a.first : room, w = a.W < room ? a.W : room;
    runs += (f + u - 1) / u + (w + u - 1) / u + 1;
  }
  return n + (runs + per - 1) / per;
}

// Whether queries stay whole: then no merge follows.  Cutting one saves it the tiles that other blocks take (a tile: 0.9 us on
// the tensor cores, elsewhere 0.4 us and 1 more per 150 dims for every 8 heads) and costs the parts and their merge, more for
// more queries.  Measured, us whole / cut, selections of so many tiles each:
//   tensor cores, 1 query: 6 tiles 14.0 / 14.8, 7 15.5 / 15.0; 20: 8 16.9 / 17.8, 11 19.6 / 19.0; 40: 14 25.0 / 26.8,
//     16 27.1 / 27.6, 20 31.7 / 29.9; 70: 8 20.4 / 28.9, 20 32.0 / 35.4, 24 36.2 / 37.1; 128: 11 25.3 / 26.7, 24 37.5 / 39.8;
//   fp32, 8 heads of 64, 1 query: 4 tiles 8.2 / 8.7, 6 10.6 / 8.7; 40: 8 12.6 / 13.2, 11 15.7 / 13.6; 70: 8 12.7 / 12.8,
//     16 19.2 / 16.1; bf16, 32 heads of 512, 1 query: 1 tile 42 / 43, 2 56 / 43; 70: 4 102 / 61; 110: 4 102 / 103.
// Where lengths differ a long query holds its block up, by 15 us at most.
bool stay_whole(const PagedArgs& a, bool tc, long long most) {
  if (a.row_table && !a.sel) return false;  // (as long as the table at most, and mostly not)
  const int Q = a.B * a.T, each = Q < kPagedBlocks ? kPagedBlocks / Q : 1;  // pieces a query
  const double tile = tc ? 0.9 : (a.H + 7) / 8 * (0.4 + a.D / 150.0), merge = tc ? 4 + Q / 9.0 : 3 + Q / 40.0;
  const long long piece = std::max((most + each - 1) / each, tc ? 2LL : 1LL);
  return tile * (most - piece) <= merge && tile * most <= 15;
}

template <typename T>
cudaError_t attend_t(const Dims& L, PagedArgs a, cudaStream_t s) {
  const bool tc = tc_paged_supported(L, a.P);
  a.tile = tc ? 64 : 32;
  a.shift = tc ? 3 : 0;  // of a run: the largest power of two that divides a page, at most a tile
  while (tc && a.shift < 6 && a.P % (2 << a.shift) == 0) ++a.shift;
  a.cols = tc ? 32 : a.D;
  const long long most = most_tiles(a);
  a.merge = !stay_whole(a, tc, most);
  a.min_tiles = a.merge ? tc ? 2 : 1 : (int)most;
  cudaError_t e;
  if (tc) {
    e = launch_tc_paged(a, s);
  } else if (simt_chunks(a.D) == 1) {
    const long long tiles = a.merge ? (most * a.B * a.T + kPagedBlocks - 1) / kPagedBlocks : most;  // a block's, at most
    e = tiles <= 1 ? simt_c<T, 1, 1>(a, s) : tiles <= 3 ? simt_c<T, 1, 2>(a, s) : simt_c<T, 1, 4>(a, s);
  } else {
    e = simt_chunks(a.D) == 2 ? simt_c<T, 2, 2>(a, s) : simt_c<T, 4, 1>(a, s);
  }
  if (e != cudaSuccess) return e;
  return a.merge ? launch_merge<T>(a, s) : cudaSuccess;
}

}  // namespace

void carve_paged(Carver& c, const Dims& L, int Q, PagedArgs* a) {
  a->parts = c.take<int2>(Q);
  a->ml = c.take<float2>((size_t)2 * kPagedBlocks * L.H);
  a->turns = c.take<float2>((size_t)kPagedBlocks * (L.R / 2));
  a->part = c.take<float>((size_t)2 * kPagedBlocks * L.H * L.D);
}

cudaError_t launch_attend_pages(const Dims& L, PagedArgs a, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? attend_t<__nv_bfloat16>(L, a, s) : attend_t<float>(L, a, s);
}

}  // namespace csa
