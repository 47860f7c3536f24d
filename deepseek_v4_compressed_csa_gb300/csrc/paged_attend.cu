// Attention over a cache in pages and 8 bits: the portable kernel (any head layout and size, bf16 and fp32), and the merge
// of queries that several blocks worked on.
//
//   l_k = scale q_h . key_k;  o_h = sum_k e^{l_k} key_k / (e^{sink_h} + sum_k e^{l_k});  out_h = RoPE^-1(o_h, p)
//
// over the keys of PagedQuery, key_k = scale_k code_k.  A block walks its run of tiles (paged.cuh) with a running maximum
// and sum per head; all arithmetic in fp32, the output rounded once.
#include "paged.cuh"
#include "tc.cuh"

namespace csa {

namespace {

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
  __shared__ int s_row[kSimtTile], s_sums[kSimtWarps];
  __shared__ PagedRun s_run;
  const int D = a.D, KS = D + kSimtPad, n8 = D >> 3;
  float* ks = sm_pa;                    // [kSimtTile][KS] keys
  float* qs = sm_pa + kSimtTile * KS;   // [kSimtWarps][D] queries of this group of heads
  pdl_wait();
  paged_plan(a, &s_run, s_sums);
  const int t0 = s_run.t0, t1 = s_run.t1;
  if (t0 >= t1) return;
  int pre = s_run.pre;
  PagedQuery k = s_run.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll 1
  while (true) {
    const int q = k.q, b = k.b;
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
            if (!a.sel || (j >= 0 && j < k.n_rows)) r = paged_row(a, a.row_table + (size_t)b * a.row_pages, j);
          } else if (x < nkeys) {
            const int y = x - k.n0;
            r = paged_row(a, a.token_table + (size_t)b * a.token_pages, y < k.f ? y : k.w0 + (y - k.f));
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
    k = next_query(a, q);
  }
}

// ---------------------------------------------------------------- merge of split queries
// With (m_s, l_s, acc_s) of the parts: M = max(z, m_s), Z = 2^{z - M} + sum_s l_s 2^{m_s - M},
// o = sum_s acc_s 2^{m_s - M} / Z (z the sink in powers of two).  A block of eight warps takes one head of a query (up to 8
// queries: each has many parts) or eight; a head's warps take its parts in turn.  The weights are found first, from all
// parts' statistics at once, so that the sum over the accumulators is loads and products only, several parts in flight;
// the angles of the rotation are found meanwhile, once a block.
constexpr int kMergeWarps = 8;

// kC: 4-value columns a lane holds, 128 values apart; kAhead: parts in flight
template <typename T, int kC, int kAhead, bool kOneHead>
__global__ void __launch_bounds__(32 * kMergeWarps) k_merge_pages(const __grid_constant__ PagedArgs a) {
  // no early trigger: what follows finds the outputs written
  extern __shared__ __align__(16) float sm_merge[];  // [kMergeWarps][kPagedBlocks] weights; [R / 2] angles; sums
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n4 = a.D >> 2;
  const int h = kOneHead ? blockIdx.y : blockIdx.y * kMergeWarps + warp;
  const int first = kOneHead ? warp : 0, step = kOneHead ? kMergeWarps : 1;
  float* wt = sm_merge + warp * kPagedBlocks;  // (a query has at most a part in every block)
  float2* cs = reinterpret_cast<float2*>(sm_merge + kMergeWarps * kPagedBlocks);
  float4* sums = reinterpret_cast<float4*>(sm_merge + kMergeWarps * kPagedBlocks + a.R);  // kOneHead: [kMergeWarps][D]
  const bool on = h < a.H;
#pragma unroll 1
  for (int q = blockIdx.x; q < a.B * a.T; q += gridDim.x) {
    const int2 at = a.parts[q];
    if (at.y <= 1) continue;
    __syncthreads();  // (the query before has been read)
    if (a.inv_freq) {
      const int p = a.pos[q / a.T] + q % a.T;
      for (int i = tid; i < a.R / 2; i += 32 * kMergeWarps) rope_cs(p, a.inv_freq, i, &cs[i].x, &cs[i].y);
    }
    auto slot = [&](int s) { return (size_t)(2 * (at.x + s) + (s == 0)); };
    float inv = 0.f;
    if (on) {
      const float z2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
      constexpr int kL = (kPagedBlocks + 31) / 32;
      float2 ml[kL];
      float M = z2;
#pragma unroll
      for (int i = 0; i < kL; ++i) {
        const int s = lane + 32 * i;
        ml[i] = s < at.y ? a.ml[slot(s) * a.H + h] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kL; ++i) M = fmaxf(M, ml[i].x);
      M = warp_max(M);
      float Z = 0.f;
#pragma unroll
      for (int i = 0; i < kL; ++i) {
        const int s = lane + 32 * i;
        const float f = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - M);  // (a part without keys)
        if (s < at.y) wt[s] = f;
        Z = fmaf(ml[i].y, f, Z);
      }
      Z = warp_sum(Z) + (z2 == -INFINITY ? 0.f : exp2f(z2 - M));
      inv = Z == 0.f ? 0.f : 1.f / Z;
    }
    __syncwarp();
    float4 acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
#pragma unroll 1
      for (int s0 = first; s0 < at.y; s0 += kAhead * step) {
        float4 x[kAhead][kC];
        float f[kAhead];
#pragma unroll
        for (int g = 0; g < kAhead; ++g) {
          const int s = min(s0 + g * step, at.y - 1);
          f[g] = s0 + g * step < at.y ? wt[s] : 0.f;
          const float* src = a.part + slot(s) * a.H * a.D;
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int d = 4 * (lane + 32 * c), blk = a.cols == a.D ? 0 : d >> 5;  // (blocks of 32 dims, or all)
            if (lane + 32 * c < n4)
              x[g][c] = __ldcg(reinterpret_cast<const float4*>(src + ((size_t)blk * a.H + h) * a.cols + (d - blk * 32)));
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
      if (kOneHead) {
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (lane + 32 * c < n4) sums[warp * n4 + lane + 32 * c] = acc[c];
      }
    }
    __syncthreads();  // (the sums, the angles)
    if (!on) continue;
    auto write = [&](int col, float4 v4) {
      const int d = 4 * col;
      float v[4] = {v4.x * inv, v4.y * inv, v4.z * inv, v4.w * inv};
      if (a.inv_freq && d >= a.D - a.R) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 t = cs[(d + e - (a.D - a.R)) >> 1];
          const float x0 = v[e], x1 = v[e + 1];
          v[e] = fmaf(x0, t.x, x1 * t.y);
          v[e + 1] = fmaf(-x0, t.y, x1 * t.x);
        }
      }
      T* o = static_cast<T*>(a.out) + ((size_t)q * a.H + h) * a.D + d;
      if constexpr (sizeof(T) == 2) {
        uint2 u;
        reinterpret_cast<__nv_bfloat162*>(&u)[0] = __floats2bfloat162_rn(v[0], v[1]);
        reinterpret_cast<__nv_bfloat162*>(&u)[1] = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(o) = u;
      } else {
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      }
    };
    if (kOneHead) {  // the head's columns over all threads
      for (int col = tid; col < n4; col += 32 * kMergeWarps) {
        float4 v4 = sums[col];
        for (int w = 1; w < kMergeWarps; ++w) {
          const float4 x = sums[w * n4 + col];
          v4.x += x.x; v4.y += x.y; v4.z += x.z; v4.w += x.w;
        }
        write(col, v4);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (lane + 32 * c < n4) write(lane + 32 * c, acc[c]);
    }
  }
}

template <typename T, int kC>
cudaError_t merge_c(const PagedArgs& a, cudaStream_t s) {
  const int Q = a.B * a.T, smem = (kMergeWarps * kPagedBlocks + a.R) * 4;
  if (Q <= 8) {
    constexpr int kSmem = (kMergeWarps * kPagedBlocks + 1024 + kMergeWarps * 1024) * 4;
    static_assert(kSmem <= 48 * 1024, "the sums fit what every kernel may take");
    CSA_LAUNCH((k_merge_pages<T, kC, kC <= 4 ? 4 : 2, true>), dim3(Q, a.H), dim3(32 * kMergeWarps),
               smem + kMergeWarps * a.D * 4, s, a);
  } else {
    CSA_LAUNCH((k_merge_pages<T, kC, 2, false>), dim3(min(Q, 4 * kPagedBlocks), (a.H + kMergeWarps - 1) / kMergeWarps),
               dim3(32 * kMergeWarps), smem, s, a);
  }
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_merge(const PagedArgs& a, cudaStream_t s) {
  return a.D <= 128 ? merge_c<T, 1>(a, s) : a.D <= 512 ? merge_c<T, 4>(a, s) : merge_c<T, 8>(a, s);
}

template <typename T>
cudaError_t attend_t(const Dims& L, PagedArgs a, cudaStream_t s) {
  a.min_tiles = 2;
  if (tc_paged_supported(L, a.P)) {
    a.tile = 64;
    a.shift = 3;  // the largest power of two that divides a page, at most a tile
    while (a.shift < 6 && a.P % (2 << a.shift) == 0) ++a.shift;
    a.cols = 32;
    const cudaError_t e = launch_tc_paged(a, s);
    if (e != cudaSuccess) return e;
  } else {
    a.tile = kSimtTile;
    a.shift = 0;
    a.cols = a.D;
    allow_smem<kSimtSmemMax>(k_attend_pages_simt<T>);
    CSA_LAUNCH(k_attend_pages_simt<T>, dim3(kPagedBlocks), dim3(32 * kSimtWarps), simt_smem(a.D), s, a);
  }
  return launch_merge<T>(a, s);
}

}  // namespace

void carve_paged(Carver& c, const Dims& L, int Q, PagedArgs* a) {
  a->parts = c.take<int2>(Q);
  a->ml = c.take<float2>((size_t)2 * kPagedBlocks * L.H);
  a->part = c.take<float>((size_t)2 * kPagedBlocks * L.H * L.D);
}

cudaError_t launch_attend_pages(const Dims& L, PagedArgs a, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? attend_t<__nv_bfloat16>(L, a, s) : attend_t<float>(L, a, s);
}

}  // namespace csa
