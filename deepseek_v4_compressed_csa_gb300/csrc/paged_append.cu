// Latent rows into the pages of a cache: RMS norm, rotation at the row's position, 8 bits with a scale per row.
//
//   y = x (mean(x^2) + eps)^-1/2 w, its last R values rotated;  codes = E4M3(y / s), s = max |y| / 448
//
// in fp32, rounded once, to the codes.  A warp a row, which stays in its registers; the page is looked up while the row
// is on its way.  A row costs 3 bytes a value: some thousand rows take as long as the launch (32 rows of 512 values 2.7 us,
// 4096 rows 4.3, 1.5 TB/s; with the weights read after the norm and the page before it 3.0 and 4.4, cold 4.5 against 3.7).
#include "paged.cuh"

namespace csa {

namespace {

constexpr int kApWarps = 4;

template <typename T, int kChunks>  // chunks of 8 values a lane holds: D <= 256 kChunks
__global__ void __launch_bounds__(32 * kApWarps) k_append_pages(const __grid_constant__ PagedAppend a) {
  // no early trigger: what follows finds the rows in their pages
  extern __shared__ __align__(16) float2 cs_all[];  // [kApWarps][R / 2] cos, sin
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n = (long long)blockIdx.x * kApWarps + warp;
  if (n >= (long long)a.B * a.T) return;
  const int b = (int)(n / a.T), i = (int)(n - (long long)b * a.T), n8 = a.D >> 3;
  const T* x = static_cast<const T*>(a.rows) + b * a.stride_b + i * a.stride_t;
  float v[kChunks][8];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
    if (lane + 32 * c < n8) load8(x + 8 * (lane + 32 * c), v[c]);
  }
  const int p0 = a.pos[b], count = a.n_new ? a.n_new[b] : a.T;
  if (p0 < 0 || p0 > INT32_MAX - a.T || count < 0 || count > a.T) {
    if (i == 0 && lane == 0) atomicOr(a.err, CSA_DEV_STATE);
    return;
  }
  if (i >= count) return;
  const int p = p0 + i, k = p / a.P;
  if (k >= a.pages) {
    if (lane == 0) atomicOr(a.err, CSA_DEV_CAPACITY);
    return;
  }
  // (what else is read is on its way while the row is worked on: the page is needed last)
  const int page = __ldg(a.table + (size_t)b * a.pages + k);
  float w[kChunks][8];
  const bool weighted = a.norm && a.weight;
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    if (weighted && lane + 32 * c < n8) load8_nc(a.weight + 8 * (lane + 32 * c), w[c]);
  if (a.inv_freq) {
    float2* cs = cs_all + warp * (a.R / 2);
    for (int f = lane; f < a.R / 2; f += 32) turn_cs(p, __ldg(a.inv_freq + f), &cs[f].x, &cs[f].y);
    __syncwarp();
  }
  if (a.norm) {
    const float inv = inv_rms(1.0f / (float)a.D, a.eps, [&](float f) {
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[c][e] * f, v[c][e] * f, ss);
      return warp_sum(ss);
    });
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= inv;
  }
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int d = 8 * (lane + 32 * c);
    if (d >= a.D) continue;
    if (weighted) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= w[c][e];
    }
    if (a.inv_freq && d >= a.D - a.R) {
      const float2* cs = cs_all + warp * (a.R / 2) + ((d - (a.D - a.R)) >> 1);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 t = cs[e >> 1];
        const float x0 = v[c][e], x1 = v[c][e + 1];
        v[c][e] = fmaf(x0, t.x, -x1 * t.y);
        v[c][e + 1] = fmaf(x0, t.y, x1 * t.x);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v[c][e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((unsigned)page >= (unsigned)a.n_pages) {
    if (lane == 0) atomicOr(a.err, CSA_DEV_RANGE);
    return;
  }
  const float s = __fdiv_rn(amax, 448.f);
  const size_t row = (size_t)page * a.P + (p - k * a.P);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int d = 8 * (lane + 32 * c);
    if (d >= a.D) continue;
    uint2 u;
    u.x = e4m3x4(over_scale(v[c][0], s), over_scale(v[c][1], s), over_scale(v[c][2], s), over_scale(v[c][3], s));
    u.y = e4m3x4(over_scale(v[c][4], s), over_scale(v[c][5], s), over_scale(v[c][6], s), over_scale(v[c][7], s));
    *reinterpret_cast<uint2*>(a.codes + row * a.D + d) = u;
  }
  if (lane == 0) a.scales[row] = s;
}

template <typename T>
cudaError_t append_t(const PagedAppend& t, cudaStream_t s) {
  const dim3 grid((unsigned)(((long long)t.B * t.T + kApWarps - 1) / kApWarps)), block(32 * kApWarps);
  const size_t smem = t.inv_freq ? (size_t)kApWarps * (t.R / 2) * sizeof(float2) : 0;
  if (t.D <= 256) CSA_LAUNCH((k_append_pages<T, 1>), grid, block, smem, s, t);
  else if (t.D <= 512) CSA_LAUNCH((k_append_pages<T, 2>), grid, block, smem, s, t);
  else CSA_LAUNCH((k_append_pages<T, 4>), grid, block, smem, s, t);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_pages(const Dims& L, const PagedAppend& t, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? append_t<__nv_bfloat16>(t, s) : append_t<float>(t, s);
}

}  // namespace csa
