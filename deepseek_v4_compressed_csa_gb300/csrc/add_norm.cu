// The residual's addition, its RMS norm and the norm in 8 bits, in one pass over the rows.
//
//   h = x + residual;  y = h (mean(h^2) + eps)^-1/2 w;  codes = E4M3(y / s), s = max |y| of a group / 448
//
// in fp32: the sum is normed as it is, before h is rounded for the stream; y is rounded to the model dtype and, apart
// from that, to the codes.  Bound by memory: 4 model-dtype tensors and one of bytes, each touched once; a row stays in
// registers between its square sum and its outputs.
#include "paged.cuh"

namespace csa {

namespace {

constexpr int kAnThreads = 512;  // the most for a row: four chunks of 8 values a thread cover 16384

template <typename T>
struct AnArgs {
  const T *x, *residual;
  const float* weight;
  T *out, *residual_out;
  uint8_t* codes;
  float* scales;
  long long N, x_stride, r_stride;
  int X, group, lanes;  // lanes: threads that hold a group (a power of two up to 32), 0: the whole row
  float inv_x, eps;
};

__device__ __forceinline__ float max_nan_lanes(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A row by one warp (kWarpRow: blockDim.y rows a block, X <= 256 kChunks) or by a block; kChunks chunks of 8 values a thread.
template <typename T, int kChunks, bool kWarpRow>
__global__ void __launch_bounds__(kAnThreads) k_add_norm(const __grid_constant__ AnArgs<T> a) {
  // no early trigger: the compress calls read x before their own wait
  __shared__ float red[32];
  pdl_wait();
  const int tid = threadIdx.x, n8 = a.X >> 3, nt = blockDim.x;
  const long long row = kWarpRow ? (long long)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
  if (kWarpRow && row >= a.N) return;
  const T* x = a.x + row * a.x_stride;
  const T* r = a.residual ? a.residual + row * a.r_stride : nullptr;
  float v[kChunks][8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = tid + i * nt;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    if (c < n8) load8(x + 8 * c, v[i]);
  }
  if (r) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = tid + i * nt;
      if (c < n8) {
        float w[8];
        load8(r + 8 * c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += w[e];
      }
    }
  }
  if (a.residual_out) {
    T* h = a.residual_out + row * a.X;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = tid + i * nt;
      if (c < n8) store8(h + 8 * c, v[i]);
    }
  }
  const float inv = inv_rms(a.inv_x, a.eps, [&](float f) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e] * f, v[i][e] * f, ss);
    return kWarpRow ? warp_sum(ss) : block_sum(ss, red);
  });
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = tid + i * nt;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= inv;
    if (a.weight && c < n8) {
      float w[8];
      load8_nc(a.weight + 8 * c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
    }
  }
  if (a.out) {
    T* o = a.out + row * a.X;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = tid + i * nt;
      if (c < n8) store8(o + 8 * c, v[i]);
    }
  }
  if (!a.codes) return;
  float amax[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    amax[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax[i] = max_nan(amax[i], fabsf(v[i][e]));
  }
  if (a.lanes) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) amax[i] = max_nan_lanes(amax[i], a.lanes);
  } else {
    float m = amax[0];
#pragma unroll
    for (int i = 1; i < kChunks; ++i) m = max_nan(m, amax[i]);
    m = max_nan_lanes(m, 32);
    if (!kWarpRow) {
      __syncthreads();  // (red: the square sum's)
      if ((tid & 31) == 0) red[tid >> 5] = m;
      __syncthreads();
      m = max_nan_lanes((tid & 31) < (nt >> 5) ? red[tid & 31] : 0.f, 32);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) amax[i] = m;
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = tid + i * nt;
    if (c >= n8) continue;
    const float s = __fdiv_rn(amax[i], 448.f);
    uint2 k;
    k.x = e4m3x4(over_scale(v[i][0], s), over_scale(v[i][1], s), over_scale(v[i][2], s), over_scale(v[i][3], s));
    k.y = e4m3x4(over_scale(v[i][4], s), over_scale(v[i][5], s), over_scale(v[i][6], s), over_scale(v[i][7], s));
    *reinterpret_cast<uint2*>(a.codes + row * a.X + 8 * c) = k;
    if (a.lanes ? c % a.lanes == 0 : c == 0) a.scales[row * (a.X / a.group) + 8 * c / a.group] = s;
  }
}

template <typename T>
cudaError_t add_norm_t(const Dims& L, const AddNorm& t, cudaStream_t s) {
  AnArgs<T> a{};
  a.x = static_cast<const T*>(t.x);
  a.residual = static_cast<const T*>(t.residual);
  a.weight = t.weight;
  a.out = static_cast<T*>(t.out);
  a.residual_out = static_cast<T*>(t.residual_out);
  a.codes = t.codes; a.scales = t.scales;
  a.N = t.N; a.x_stride = t.x_stride; a.r_stride = t.r_stride;
  a.X = t.X; a.group = t.group;
  a.lanes = t.codes && t.group <= 256 && t.group != t.X ? t.group / 8 : 0;
  a.inv_x = 1.0f / (float)t.X;
  a.eps = L.eps;
  const int n8 = t.X / 8;
  if (n8 <= 64) {
    const dim3 block(32, 8), grid((unsigned)((t.N + 7) / 8));
    if (n8 <= 32) CSA_LAUNCH((k_add_norm<T, 1, true>), grid, block, 0, s, a);
    else CSA_LAUNCH((k_add_norm<T, 2, true>), grid, block, 0, s, a);
    return cudaGetLastError();
  }
  const dim3 grid((unsigned)t.N);
  if (n8 <= kAnThreads) CSA_LAUNCH((k_add_norm<T, 1, false>), grid, dim3((n8 + 31) / 32 * 32), 0, s, a);
  else if (n8 <= 2 * kAnThreads) CSA_LAUNCH((k_add_norm<T, 2, false>), grid, dim3(kAnThreads), 0, s, a);
  else CSA_LAUNCH((k_add_norm<T, 4, false>), grid, dim3(kAnThreads), 0, s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_norm(const Dims& L, const AddNorm& t, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? add_norm_t<__nv_bfloat16>(L, t, s) : add_norm_t<float>(L, t, s);
}

}  // namespace csa
