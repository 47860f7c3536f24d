// The residual's addition, its RMS norm and the norm in 8 bits, in one pass over the rows.
//
//   h = x + residual;  y = h (mean(h^2) + eps)^-1/2 w;  codes = E4M3(y / s), s = max |y| of a group / 448
//
// in fp32: the sum is normed as it is, before h is rounded for the stream; y is rounded to the model dtype and, apart
// from that, to the codes (by the scale's reciprocal: a quotient within two roundings).  Bound by memory: 4 model-dtype
// tensors and one of bytes, each touched once; a row stays in registers between its square sum and its outputs.  What else
// costs is instructions, 16.7M values of a chunk of 4096 tokens by some twenty each: a division a value took 6 us of 31.
// Blocks walk rows; the next row is on its way while one is worked on.
#include "paged.cuh"

namespace csa {

namespace {

constexpr int kSms = 152;
constexpr int kAnThreads = 512;  // the most for a row: four chunks of 8 values a thread cover 16384
// Threads an SM holds of blocks with so many chunks a thread (what their registers are bounded for).  4096 tokens of 4096
// values: 512 threads with one chunk, three blocks an SM, 26.6 us (5.7 TB/s); two blocks 27.9, four 28.6 (spills); 256
// threads with two chunks 31.0.
constexpr int an_resident(int chunks, int bytes) { return chunks == 1 ? (bytes == 2 ? 1536 : 1024) : chunks == 2 && bytes == 2 ? 1024 : 512; }

template <typename T>
struct AnArgs {
  const T *x, *residual;
  const float* weight;
  T *out, *residual_out;
  uint8_t* codes;
  float* scales;
  long long N, x_stride, r_stride;
  int X, lanes;         // lanes: threads that hold a group (a power of two up to 32), 0: the whole row
  int group_log2;
  float inv_x, eps;
};

// 8 values as loaded
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 v; };
template <> struct Raw8<float> { float4 a, b; };
__device__ __forceinline__ void raw_load(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p) { r.v = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void raw_load(Raw8<float>& r, const float* p) {
  r.a = reinterpret_cast<const float4*>(p)[0];
  r.b = reinterpret_cast<const float4*>(p)[1];
}
__device__ __forceinline__ void raw_get(const Raw8<__nv_bfloat16>& r, float* o) {
  const uint32_t u[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(u[i] << 16);
    o[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void raw_get(const Raw8<float>& r, float* o) {
  o[0] = r.a.x; o[1] = r.a.y; o[2] = r.a.z; o[3] = r.a.w;
  o[4] = r.b.x; o[5] = r.b.y; o[6] = r.b.z; o[7] = r.b.w;
}

__device__ __forceinline__ float max_nan_lanes(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A row by one warp (kWarpRow: blockDim.y rows a block, X <= 256 kChunks) or by a block; kChunks chunks of 8 values a thread.
template <typename T, int kChunks, bool kWarpRow>
__global__ void __launch_bounds__(kAnThreads, an_resident(kChunks, sizeof(T)) / kAnThreads) k_add_norm(const __grid_constant__ AnArgs<T> a) {
  // no early trigger: the compress calls read x before their own wait
  __shared__ float red[2][32];
  pdl_wait();
  const int tid = threadIdx.x, n8 = a.X >> 3, nt = kWarpRow ? 32 : blockDim.x;
  const long long step = kWarpRow ? (long long)gridDim.x * blockDim.y : gridDim.x;
  long long row = kWarpRow ? (long long)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
  Raw8<T> rx[kChunks], rr[kChunks];
  auto fetch = [&](long long n) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = tid + i * nt;
      if (c < n8) {
        raw_load(rx[i], a.x + n * a.x_stride + 8 * c);
        if (a.residual) raw_load(rr[i], a.residual + n * a.r_stride + 8 * c);
      }
    }
  };
  if (row < a.N) fetch(row);
  int buf = 0;
#pragma unroll 1
  for (; row < a.N; row += step) {
    float v[kChunks][8];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      if (tid + i * nt < n8) {
        raw_get(rx[i], v[i]);
        if (a.residual) {
          float u[8];
          raw_get(rr[i], u);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += u[e];
        }
      }
    }
    // (in place, too: an output's row is written once its own has been read, and no other row is)
    if (row + step < a.N) fetch(row + step);
    if (a.residual_out) {
      T* h = a.residual_out + row * a.X;
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        if (tid + i * nt < n8) store8(h + 8 * (tid + i * nt), v[i]);
    }
    const float inv = inv_rms(a.inv_x, a.eps, [&](float f) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e] * f, v[i][e] * f, ss);
      ss = warp_sum(ss);
      if (kWarpRow) return ss;
      buf ^= 1;  // (two buffers: the next sums are written while some warp still reads these)
      if ((tid & 31) == 0) red[buf][tid >> 5] = ss;
      __syncthreads();
      return warp_sum((tid & 31) < (nt >> 5) ? red[buf][tid & 31] : 0.f);
    });
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= inv;
      if (a.weight && tid + i * nt < n8) {
        float w[8];
        load8_nc(a.weight + 8 * (tid + i * nt), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
      }
    }
    if (a.out) {
      T* o = a.out + row * a.X;
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        if (tid + i * nt < n8) store8(o + 8 * (tid + i * nt), v[i]);
    }
    if (!a.codes) continue;
    float amax[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      amax[i] = fabsf(v[i][0]);
#pragma unroll
      for (int e = 1; e < 8; ++e) amax[i] = max_nan(amax[i], fabsf(v[i][e]));
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
        buf ^= 1;
        if ((tid & 31) == 0) red[buf][tid >> 5] = m;
        __syncthreads();
        m = max_nan_lanes((tid & 31) < (nt >> 5) ? red[buf][tid & 31] : 0.f, 32);
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
      if (s < 1e-30f) {  // (its reciprocal would leave fp32's range, or the scale is 0; a NaN goes the other way)
        k.x = e4m3x4(over_scale(v[i][0], s), over_scale(v[i][1], s), over_scale(v[i][2], s), over_scale(v[i][3], s));
        k.y = e4m3x4(over_scale(v[i][4], s), over_scale(v[i][5], s), over_scale(v[i][6], s), over_scale(v[i][7], s));
      } else {
        const float r = __frcp_rn(s);
        k.x = e4m3x4(v[i][0] * r, v[i][1] * r, v[i][2] * r, v[i][3] * r);
        k.y = e4m3x4(v[i][4] * r, v[i][5] * r, v[i][6] * r, v[i][7] * r);
      }
      *reinterpret_cast<uint2*>(a.codes + row * a.X + 8 * c) = k;
      if (a.lanes ? (c & (a.lanes - 1)) == 0 : c == 0)
        a.scales[a.lanes ? row * (a.X >> a.group_log2) + (8 * c >> a.group_log2) : row] = s;
    }
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
  a.X = t.X;
  a.lanes = t.codes && t.group <= 256 && t.group != t.X ? t.group / 8 : 0;
  while ((1 << a.group_log2) < t.group) ++a.group_log2;
  a.inv_x = 1.0f / (float)t.X;
  a.eps = L.eps;
  const int n8 = t.X / 8;
  auto blocks = [&](long long rows, int threads, int chunks) {
    return dim3((unsigned)min(rows, (long long)kSms * (an_resident(chunks, sizeof(T)) / threads)));
  };
  if (n8 <= 64) {
    const dim3 block(32, 8);
    if (n8 <= 32) CSA_LAUNCH((k_add_norm<T, 1, true>), blocks((t.N + 7) / 8, 256, 1), block, 0, s, a);
    else CSA_LAUNCH((k_add_norm<T, 2, true>), blocks((t.N + 7) / 8, 256, 2), block, 0, s, a);
    return cudaGetLastError();
  }
  const int chunks = n8 <= kAnThreads ? 1 : n8 <= 2 * kAnThreads ? 2 : 4, threads = ((n8 + chunks - 1) / chunks + 31) / 32 * 32;
  const dim3 grid = blocks(t.N, threads, chunks), block(threads);
  if (chunks == 1) CSA_LAUNCH((k_add_norm<T, 1, false>), grid, block, 0, s, a);
  else if (chunks == 2) CSA_LAUNCH((k_add_norm<T, 2, false>), grid, block, 0, s, a);
  else CSA_LAUNCH((k_add_norm<T, 4, false>), grid, block, 0, s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_norm(const Dims& L, const AddNorm& t, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? add_norm_t<__nv_bfloat16>(L, t, s) : add_norm_t<float>(L, t, s);
}

}  // namespace csa
