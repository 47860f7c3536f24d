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

constexpr int kSimtTile = 32;   // keys a tile: a lane each
constexpr int kSimtWarps = 8;   // heads at a time, a warp each
constexpr int kSimtMaxC = 4;    // chunks of 8 dims a lane: D <= 1024
constexpr int kSimtPad = 4;     // floats behind a key's row: lanes read their keys' chunks without bank conflicts
constexpr int kSimtSmemMax = (kSimtTile * (1024 + kSimtPad) + kSimtWarps * 1024) * 4 + 1024;

__host__ __device__ constexpr int simt_smem(int D) { return (kSimtTile * (D + kSimtPad) + kSimtWarps * D) * 4; }

__device__ __forceinline__ int simt_tiles(const PagedArgs& a, int q) {
  const PagedQuery k = paged_query(a, q, false);
  return k.live ? max(1, (k.n0 + k.f + k.nw + kSimtTile - 1) / kSimtTile) : 0;
}

template <typename T>
__global__ void __launch_bounds__(32 * kSimtWarps) k_attend_pages_simt(const __grid_constant__ PagedArgs a) {
  pdl_trigger();  // (the merge alone follows, and waits)
  extern __shared__ __align__(16) float sm_pa[];
  __shared__ int sm_plan[35];
  __shared__ int s_row[kSimtTile];
  const int D = a.D, KS = D + kSimtPad, n8 = D >> 3;
  float* ks = sm_pa;                    // [kSimtTile][KS] keys
  float* qs = sm_pa + kSimtTile * KS;   // [kSimtWarps][D] queries of this group of heads
  pdl_wait();
  const PagedRun run = paged_run(a, sm_plan, [&](int q) { return simt_tiles(a, q); });
  if (run.t0 >= run.t1) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int pre = run.pre;
#pragma unroll 1
  for (int q = run.q; pre < run.t1; ++q) {
    const int n = simt_tiles(a, q);
    if (n == 0) continue;
    const PagedQuery k = paged_query(a, q, false);
    const int begin = max(run.t0 - pre, 0), end = min(run.t1 - pre, n), nkeys = k.n0 + k.f + k.nw;
    const int n_rows = a.sel ? a.n_rows[k.b] : 0;
    const bool whole = begin == 0 && end == n;
    const int slot = 2 * blockIdx.x + (begin == 0 ? 1 : 0);
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
            r = a.sel ? paged_selected(a, k, __ldg(a.sel + (size_t)q * a.topk + x), n_rows)
                      : paged_row(a.row_table, a.row_pages, k.b, x, a.P, a.n_pages);
          } else if (x < nkeys) {
            const int y = x - k.n0;
            r = paged_row(a.token_table, a.token_pages, k.b, y < k.f ? y : k.w0 + (y - k.f), a.P, a.n_pages);
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
    pre += n;
  }
}

// ---------------------------------------------------------------- merge of split queries
// With (m_s, l_s, acc_s) of the parts: M = max(z, m_s), Z = 2^{z - M} + sum_s l_s 2^{m_s - M},
// o = sum_s acc_s 2^{m_s - M} / Z (z the sink in powers of two).  Block (query, heads): a head by 1 or 8 warps, which take
// its parts in turn; a lane holds 4-value columns 128 apart.
constexpr int kMergeC = 8;  // columns a lane: D <= 1024
constexpr int kMergeWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kMergeWarps) k_merge_pages(const __grid_constant__ PagedArgs a, int heads) {
  // no early trigger: what follows finds the outputs written
  extern __shared__ __align__(16) float4 sm_acc[];  // [kMergeWarps][D / 4] (heads == 1)
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n4 = a.D >> 2;
  const int h = blockIdx.y * heads + (heads == 1 ? 0 : warp), first = heads == 1 ? warp : 0, step = heads == 1 ? kMergeWarps : 1;
#pragma unroll 1
  for (int q = blockIdx.x; q < a.B * a.T; q += gridDim.x) {
    const int2 at = a.parts[q];
    if (at.y <= 1) continue;
    float m = -INFINITY, l = 0.f;
    float4 acc[kMergeC];
#pragma unroll
    for (int c = 0; c < kMergeC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h < a.H) {
      for (int s = first; s < at.y; s += step) {
        const size_t row = (size_t)(2 * (at.x + s) + (s == 0 ? 1 : 0)) * a.H + h;
        const float2 ml = a.ml[row];
        float4 x[kMergeC];
#pragma unroll
        for (int c = 0; c < kMergeC; ++c)
          if (lane + 32 * c < n4) x[c] = reinterpret_cast<const float4*>(a.part + row * a.D)[lane + 32 * c];
        if (ml.x == -INFINITY) continue;  // a part without keys
        const float mn = fmaxf(m, ml.x), f0 = exp2f(m - mn), f1 = exp2f(ml.x - mn);
        m = mn;
        l = fmaf(l, f0, ml.y * f1);
#pragma unroll
        for (int c = 0; c < kMergeC; ++c) {
          if (lane + 32 * c < n4) {
            acc[c].x = fmaf(acc[c].x, f0, x[c].x * f1);
            acc[c].y = fmaf(acc[c].y, f0, x[c].y * f1);
            acc[c].z = fmaf(acc[c].z, f0, x[c].z * f1);
            acc[c].w = fmaf(acc[c].w, f0, x[c].w * f1);
          }
        }
      }
    }
    if (heads == 1) {
      __syncthreads();  // (the query before has been read)
      for (int c = 0; c < kMergeC; ++c)
        if (lane + 32 * c < n4) sm_acc[warp * n4 + lane + 32 * c] = acc[c];
      if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
      }
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < kMergeWarps; ++w) {
          if (s_m[w] == -INFINITY) continue;
          const float mn = fmaxf(m, s_m[w]), f0 = exp2f(m - mn), f1 = exp2f(s_m[w] - mn);
          m = mn;
          l = fmaf(l, f0, s_l[w] * f1);
#pragma unroll
          for (int c = 0; c < kMergeC; ++c) {
            if (lane + 32 * c < n4) {
              const float4 x = sm_acc[w * n4 + lane + 32 * c];
              acc[c].x = fmaf(acc[c].x, f0, x.x * f1);
              acc[c].y = fmaf(acc[c].y, f0, x.y * f1);
              acc[c].z = fmaf(acc[c].z, f0, x.z * f1);
              acc[c].w = fmaf(acc[c].w, f0, x.w * f1);
            }
          }
        }
      }
    }
    if (h >= a.H || (heads == 1 && warp != 0)) continue;
    const float z2 = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
    const float M = fmaxf(m, z2), f = m == -INFINITY ? 0.f : exp2f(m - M);
    const float Z = l * f + (z2 == -INFINITY ? 0.f : exp2f(z2 - M));
    const float w = Z == 0.f ? 0.f : f / Z;
    const int p = a.pos[q / a.T] + q % a.T;
#pragma unroll
    for (int c = 0; c < kMergeC; ++c) {
      const int d = 4 * (lane + 32 * c);
      if (d >= a.D) continue;
      float v[4] = {acc[c].x * w, acc[c].y * w, acc[c].z * w, acc[c].w * w};
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

template <typename T>
cudaError_t launch_merge(const PagedArgs& a, cudaStream_t s) {
  const int Q = a.B * a.T;
  // few queries have many parts each: a head by a block's eight warps
  const int heads = Q <= 8 ? 1 : kMergeWarps;
  const size_t smem = heads == 1 ? (size_t)kMergeWarps * a.D * sizeof(float) : 0;
  CSA_LAUNCH(k_merge_pages<T>, dim3(min(Q, 4 * kPagedBlocks), (a.H + heads - 1) / heads), dim3(32 * kMergeWarps), smem, s,
             a, heads);
  return cudaGetLastError();
}

template <typename T>
cudaError_t attend_t(const Dims& L, PagedArgs a, cudaStream_t s) {
  if (tc_paged_supported(L, a.n_pages, a.P)) {
    const cudaError_t e = launch_tc_paged(L, a, kPagedBlocks, s);
    if (e != cudaSuccess) return e;
  } else {
    a.min_tiles = 2;
    allow_smem<kSimtSmemMax>(k_attend_pages_simt<T>);
    CSA_LAUNCH(k_attend_pages_simt<T>, dim3(kPagedBlocks), dim3(32 * kSimtWarps), simt_smem(a.D), s, a);
  }
  return launch_merge<T>(a, s);
}

}  // namespace

void carve_paged(Carver& c, const Dims& L, int Q, PagedArgs* a) {
  a->part = c.take<float>((size_t)2 * kPagedBlocks * L.H * L.D);
  a->ml = c.take<float2>((size_t)2 * kPagedBlocks * L.H);
  a->parts = c.take<int2>(Q);
}

cudaError_t launch_attend_pages(const Dims& L, PagedArgs a, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? attend_t<__nv_bfloat16>(L, a, s) : attend_t<float>(L, a, s);
}

}  // namespace csa
