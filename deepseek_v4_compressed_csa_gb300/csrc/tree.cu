// Verifying a tree of drafted tokens: the portable kernels (any head layout and size, bf16 and fp32).
//
// Definitions (include/csa.h): a node's row, scores and output are what sequential decoding along the node's path
// would give; nothing of the tree enters the cache before commit.
#include "tree.cuh"

#include "fp8_row.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa {

namespace {

// ---------------------------------------------------------------- norm and rotation
// y = x rsqrt(mean(x^2) + eps) w, then the last R dims of the row turned by the token's position.  One pass: a row
// is read once into registers, its square sum reduced in fp32 inside the lanes that hold it, and written once, rounded
// once.  Bound by memory (2 x the tensors' bytes) only while a row costs few instructions: a row of up to 256 values
// sits in 2^k lanes (several rows a warp), a longer one in a warp, 8 values a lane and chunk, sums and products run as
// packed pairs, and a block takes a whole token, so that its angles (sines of up to 10^5 rad, some hundred instructions
// each) are found once, its rows requested into L2 meanwhile; with few tokens a token's rows are split over blocks.  4096
// tokens of 64 x 512, 512 and 64 x 128 values: 112 us, 6.1 TB/s (without the requests 128 us; two row groups in flight a
// warp in place of one 118 us, the next one's loads before a group's arithmetic 120 us; two tokens a block 4% more).
constexpr int kNrParts = 4;
constexpr int kNrWarps = 8;
constexpr int kNrAhead = 128 * 1024;  // bytes of a token's tensor that are prefetched

template <typename T>
struct NrPart {
  const T* x;
  T* out;
  const float* w;
  int heads, dim, norm, lpr_log2;  // lpr: lanes that hold a row (a power of two, at most 32)
  float inv_dim;
  long long x_stride;              // elements between tokens
};
template <typename T>
struct NrArgs {
  NrPart<T> part[kNrParts];
  int n_parts, R, T_;
  const int32_t* parent;
  const int32_t* pos;
  const float* inv_freq;
  float eps;
  int32_t* err;
};

// 8 values as loaded
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 v; };
template <> struct Raw8<float> { float4 a, b; };
__device__ __forceinline__ void raw_load(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p) {
  r.v = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void raw_load(Raw8<float>& r, const float* p) {
  r.a = reinterpret_cast<const float4*>(p)[0];
  r.b = reinterpret_cast<const float4*>(p)[1];
}
__device__ __forceinline__ void raw_get(const Raw8<__nv_bfloat16>& r, float2 (&o)[4]) {
  const uint32_t u[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ void raw_get(const Raw8<float>& r, float2 (&o)[4]) {
  o[0] = make_float2(r.a.x, r.a.y); o[1] = make_float2(r.a.z, r.a.w);
  o[2] = make_float2(r.b.x, r.b.y); o[3] = make_float2(r.b.z, r.b.w);
}

// This warp's rows of one tensor for one token; kChunks: 8-value chunks a lane holds of a row (more than one: a row
// takes the warp).
template <typename T, int kChunks>
__device__ __forceinline__ void norm_rope_part(const NrPart<T>& pt, int tok, int first, int step, int R, float eps,
                                               bool rotate, const float2* cs) {
  const int lane = threadIdx.x & 31, lg = kChunks > 1 ? 5 : pt.lpr_log2, sub = lane & ((1 << lg) - 1);
  const int rpw = 32 >> lg, n8 = pt.dim >> 3, r0 = pt.dim - R, heads = pt.heads, dim = pt.dim, norm = pt.norm;
  const float* w = pt.w;
  const float inv_dim = pt.inv_dim;
  const T* x = pt.x + (size_t)tok * pt.x_stride + sub * 8;
  T* out = pt.out + (size_t)tok * heads * dim + sub * 8;
  const int h0 = lane >> lg;
  for (int g = first; g * rpw < heads; g += step) {
    const int h = g * rpw + h0;
    Raw8<T> raw[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (h < heads && sub + 32 * i < n8) raw_load(raw[i], x + (size_t)h * dim + 256 * i);
    float2 v[kChunks][4];
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (h < heads && sub + 32 * i < n8) {
        raw_get(raw[i], v[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s2 = __ffma2_rn(v[i][e], v[i][e], s2);
      }
    }
    if (norm) {
      float ss = s2.x + s2.y;
      if (kChunks > 1) {
        ss = warp_sum(ss);
      } else {
        for (int o = 1 << lg >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      }
      const float inv = rsqrtf(fmaf(ss, inv_dim, eps));
      const float2 inv2 = make_float2(inv, inv);
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = __fmul2_rn(v[i][e], inv2);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = sub + 32 * i;
      if (h >= heads || c >= n8) continue;
      if (norm && w) {
        const float4 wa = __ldg(reinterpret_cast<const float4*>(w + 8 * c));
        const float4 wb = __ldg(reinterpret_cast<const float4*>(w + 8 * c) + 1);
        v[i][0] = __fmul2_rn(v[i][0], make_float2(wa.x, wa.y));
        v[i][1] = __fmul2_rn(v[i][1], make_float2(wa.z, wa.w));
        v[i][2] = __fmul2_rn(v[i][2], make_float2(wb.x, wb.y));
        v[i][3] = __fmul2_rn(v[i][3], make_float2(wb.z, wb.w));
      }
      if (rotate && 8 * c >= r0) {
        const float4* t = reinterpret_cast<const float4*>(cs + ((8 * c - r0) >> 1));
        const float4 t0 = t[0], t1 = t[1];
        const float2 a[4] = {make_float2(t0.x, t0.y), make_float2(t0.z, t0.w), make_float2(t1.x, t1.y),
                             make_float2(t1.z, t1.w)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[i][e] = make_float2(fmaf(v[i][e].x, a[e].x, -v[i][e].y * a[e].y),
                                fmaf(v[i][e].x, a[e].y, v[i][e].y * a[e].x));
      }
      store8(out + (size_t)h * dim + 256 * i, reinterpret_cast<const float*>(v[i]));
    }
  }
}

// Block (token, share): the token's row groups blockIdx.y * kNrWarps + warp, and so on by kNrWarps * gridDim.y.  kLong:
// some row is longer than 512 values (an instance of its own, for its registers).
template <typename T, bool kLong>
__global__ void __launch_bounds__(32 * kNrWarps, kLong ? 2 : 3) k_norm_rope(const __grid_constant__ NrArgs<T> a) {
  // no early trigger: kernels of later calls read queries and keys before their own wait
  extern __shared__ __align__(16) float2 cs[];  // [R / 2] cos, sin
  __shared__ int s_depth;
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok = blockIdx.x, b = tok / a.T_, i = tok - b * a.T_;
  const bool rotate = a.inv_freq != nullptr;
  // a block with the whole token: its rows are on their way into L2 while the angles are found
  if (gridDim.y == 1)
    for (int k = 0; k < a.n_parts; ++k) {
      const NrPart<T>& pt = a.part[k];
      const char* x = reinterpret_cast<const char*>(pt.x + (size_t)tok * pt.x_stride);
      for (int o = tid * 128; o < min(pt.heads * pt.dim * (int)sizeof(T), kNrAhead); o += 32 * kNrWarps * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(x + o));
    }
  if (warp == 0) {
    int depth = i;
    if (a.parent) {
      bool bad = false;
      depth = __popcll(tree_path_warp(a.parent + (size_t)b * a.T_, a.T_, i, bad)) - 1;
      if (bad && lane == 0) atomicOr(a.err, CSA_DEV_STATE);
    }
    if (depth >= 0 && rotate) {
      const int p0 = a.pos[b];
      if (p0 < 0 || p0 > INT32_MAX - depth) {
        if (lane == 0) atomicOr(a.err, CSA_DEV_STATE);
        depth = -1;
      } else {
        for (int k = lane; k < a.R / 2; k += 32) rope_cs(p0 + depth, a.inv_freq, k, &cs[k].x, &cs[k].y);
      }
    }
    if (lane == 0) s_depth = depth;
  }
  __syncthreads();
  if (s_depth < 0) return;
  const int first = blockIdx.y * kNrWarps + warp, step = kNrWarps * gridDim.y;
#pragma unroll 1
  for (int k = 0; k < a.n_parts; ++k) {
    const NrPart<T>& pt = a.part[k];
    if (pt.dim <= 256) norm_rope_part<T, 1>(pt, tok, first, step, a.R, a.eps, rotate, cs);
    else if (pt.dim <= 512) norm_rope_part<T, 2>(pt, tok, first, step, a.R, a.eps, rotate, cs);
    else if (kLong) norm_rope_part<T, 4>(pt, tok, first, step, a.R, a.eps, rotate, cs);
  }
}

template <typename T>
cudaError_t norm_rope_t(const Dims& L, const csa_rows* rows, int n, int B, int T_, const int32_t* parent,
                        const int32_t* pos, const float* inv_freq, int32_t* err, cudaStream_t s) {
  NrArgs<T> a{};
  a.n_parts = n;
  a.R = L.R; a.T_ = T_; a.parent = parent; a.pos = pos; a.inv_freq = inv_freq; a.eps = L.eps; a.err = err;
  int most = 1, longest = 0;
  for (int k = 0; k < n; ++k) {
    NrPart<T>& p = a.part[k];
    p.x = static_cast<const T*>(rows[k].x);
    p.out = static_cast<T*>(rows[k].out);
    p.w = rows[k].weight;
    p.heads = rows[k].heads;
    p.dim = rows[k].dim;
    p.norm = rows[k].norm;
    p.inv_dim = 1.0f / (float)p.dim;
    p.x_stride = rows[k].x_stride > 0 ? rows[k].x_stride : (long long)p.heads * p.dim;
    p.lpr_log2 = 0;
    while ((1 << p.lpr_log2) < 32 && (1 << p.lpr_log2) < p.dim / 8) ++p.lpr_log2;
    const int rpw = 32 >> p.lpr_log2;
    most = max(most, (p.heads + rpw - 1) / rpw);
    longest = max(longest, p.dim);
  }
  // few tokens: the rows of a token over as many blocks as give every SM eight, up to one warp per row group
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int ntok = B * T_, split = min((most + kNrWarps - 1) / kNrWarps, (8 * sms + ntok - 1) / ntok);
  const dim3 grid(ntok, max(1, split));
  const size_t smem = L.R * sizeof(float);
  if (longest > 512) CSA_LAUNCH((k_norm_rope<T, true>), grid, dim3(32 * kNrWarps), smem, s, a);
  else CSA_LAUNCH((k_norm_rope<T, false>), grid, dim3(32 * kNrWarps), smem, s, a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- rows that the tree's paths complete
template <typename T>
struct TreePool {
  const T* frontier;  // [B, F, 2 L d]
  const T* src;       // [B, T, 2 L d] the projections of every slot, or (src == proj) the nodes' in place
  T* proj;            // [B, T, 2 L d] the draft buffer that keeps the nodes'
  T* rows;            // [B, T, d], or fp8 rows
  const float* ape;
  const float* norm_w;
  int d, fp8;
};

__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }

// Block (g, b, pool): the g-th node of sequence b that completes a window along its path: the row that the compressor
// would emit, entries before pos from the frontier ring, from pos on the path's nodes.  Arithmetic and roundings are
// those of the committed rows (compress.cu: the pooled value, its norm and its rotation each in the model dtype), so
// that from equal projections an accepted row is the row decoding would have written (the projections' sums are split
// in another way than decoding's, tc_tree_project.cu, and may round to the neighbouring value).  A thread takes two neighbouring channels, and eight
// entries' loads are in flight together.  Latency-bound: what depends on the tree alone (the path, the rows' addresses,
// weights, angles) stands before the programmatic wait, behind the projections; what is left adds 3 us to 8 nodes'
// projections, 7 us to those of 512.
template <typename T>
__global__ void __launch_bounds__(256) k_tree_pool(const __grid_constant__ TreePool<T> pa,
                                                   const __grid_constant__ TreePool<T> pi, int T_, int ratio, int lanes,
                                                   int R, int F, float eps, const int32_t* __restrict__ parent,
                                                   const int32_t* __restrict__ pos,
                                                   const float* __restrict__ inv_freq, int32_t* err) {
  pdl_trigger();
  extern __shared__ __align__(16) float sm_tp[];  // [d] pooled, then normed; 32 reduction slots
  __shared__ uint64_t s_masks[kTreeMax];
  __shared__ int s_par[kTreeMax], s_path[kTreeMax], s_list[kTreeMax], s_count[2];
  const TreePool<T>& tp = blockIdx.z ? pi : pa;
  const int d = tp.d, Ld = lanes * d, rowlen = 2 * Ld;
  float* u = sm_tp;
  float* red = u + d;
  const int b = blockIdx.y, p0 = pos[b], tid = threadIdx.x;
  const bool pos_ok = tree_pos_ok(p0);
  const bool consistent = tree_masks_block(parent + (size_t)b * T_, T_, s_masks, s_par);
  if (tid < kTreeMax) {  // the completing nodes in order (two warps)
    const uint64_t m = s_masks[tid];
    const bool closes = pos_ok && m != 0 && (p0 + __popcll(m)) % ratio == 0;
    const unsigned mine = __ballot_sync(0xffffffffu, closes);
    if ((tid & 31) == 0) s_count[tid >> 5] = __popc(mine);
    if (blockIdx.x == 0 && ((tid == 0 && !consistent) || (!pos_ok && m != 0))) atomicOr(err, CSA_DEV_STATE);
    s_par[tid] = closes ? __popc(mine & ((1u << (tid & 31)) - 1u)) : -1;
  }
  __syncthreads();
  if (tid < kTreeMax && s_par[tid] >= 0) s_list[s_par[tid] + (tid < 32 ? 0 : s_count[0])] = tid;
  const bool works = pos_ok && (int)blockIdx.x < s_count[0] + s_count[1], copies = pos_ok && tp.src != tp.proj;
  // One block waits in any case: a grid that ended before the projections would let the next call's wait pass early.
  if (!works && !copies && blockIdx.x + blockIdx.y + blockIdx.z > 0) return;
  const T* src = tp.src + (size_t)b * T_ * rowlen;
  const T* fr = tp.frontier + (size_t)b * F * rowlen;
  if (copies) {
    pdl_wait();  // (the projections of every slot lie in the workspace)
    if (s_masks[blockIdx.x] != 0)
      for (int e = tid * 8; e < rowlen; e += blockDim.x * 8)
        copy8<T>(tp.proj + ((size_t)b * T_ + blockIdx.x) * rowlen + e, src + (size_t)blockIdx.x * rowlen + e);
  }
  if (!works) {
    pdl_wait();
    return;
  }
  __syncthreads();
  const int i = s_list[blockIdx.x];
  const uint64_t mask = s_masks[i];
  if (tid < kTreeMax && ((mask >> tid) & 1)) s_path[__popcll(mask & ((1ull << tid) - 1))] = tid;
  __syncthreads();
  const int p = p0 + __popcll(mask) - 1;
  const int j = (p + 1) / ratio - 1;
  const int t_lo = lanes == 2 ? max(0, (j - 1) * ratio) : j * ratio;
  const int t_hi = (j + 1) * ratio;
  const int c0 = 2 * tid;
  float2 w0 = make_float2(0.f, 0.f);
  float cs0 = 1.f, sn0 = 0.f;
  if (c0 < d) {
    w0 = load2(tp.norm_w + c0);
    if (c0 >= d - R) rope_cs(j * ratio, inv_freq, (c0 - (d - R)) >> 1, &cs0, &sn0);
  }
  // committed entries and the position table on their way into L2 (a line a request)
  for (int e = tid; e < (t_hi - t_lo) * 2; e += blockDim.x) {
    const int t = t_lo + (e >> 1), at = ((lanes == 2 && t >= j * ratio) ? d : 0) + (e & 1) * Ld;
    if (t < p0)
      for (int k = 0; k < d; k += 128 / (int)sizeof(T))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(fr + (size_t)(t % F) * rowlen + at + k));
    if ((e & 1) == 0)
      for (int k = 0; k < d; k += 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(tp.ape + (size_t)(t % ratio) * Ld + at + k));
  }
  pdl_wait();
  float ss = 0.f;
  for (int c = 2 * threadIdx.x; c < d; c += 2 * blockDim.x) {
    float2 m = make_float2(-INFINITY, -INFINITY), num = make_float2(0.f, 0.f), den = make_float2(0.f, 0.f);
    // (a remainder per entry would be most of the loop's instructions: the ring slot and the phase run along)
    int slot = t_lo % F, phase = 0, at = (lanes == 2 && t_lo >= j * ratio ? d : 0) + c;
    for (int t0 = t_lo; t0 < t_hi; t0 += 8) {
      float2 sv[8], kv[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int t = t0 + k;
        sv[k] = make_float2(-INFINITY, -INFINITY);
        kv[k] = make_float2(0.f, 0.f);
        if (t < t_hi) {
          const T* row = (t < p0 ? fr + (size_t)slot * rowlen : src + (size_t)s_path[t - p0] * rowlen) + at;
          kv[k] = load2(row);
          const float2 g = load2(row + Ld), w = load2(tp.ape + phase * Ld + at);
          sv[k] = make_float2(g.x + w.x, g.y + w.y);
          if (++slot == F) slot = 0;
          if (++phase == ratio) {
            phase = 0;
            if (lanes == 2) at += d;
          }
        }
      }
      float2 cm = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) cm = make_float2(fmaxf(cm.x, sv[k].x), fmaxf(cm.y, sv[k].y));
      const float ax = (m.x == -INFINITY) ? 0.f : expf(m.x - cm.x), ay = (m.y == -INFINITY) ? 0.f : expf(m.y - cm.y);
      num = make_float2(num.x * ax, num.y * ay);
      den = make_float2(den.x * ax, den.y * ay);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float ex = (sv[k].x == -INFINITY) ? 0.f : expf(sv[k].x - cm.x);
        const float ey = (sv[k].y == -INFINITY) ? 0.f : expf(sv[k].y - cm.y);
        den = make_float2(den.x + ex, den.y + ey);
        num = make_float2(fmaf(ex, kv[k].x, num.x), fmaf(ey, kv[k].y, num.y));
      }
      m = cm;
    }
    const float x = rnd<T>(num.x / den.x), y = rnd<T>(num.y / den.y);
    u[c] = x;
    u[c + 1] = y;
    ss = fmaf(x, x, fmaf(y, y, ss));
  }
  ss = block_sum(ss, red);
  const float inv = 1.0f / sqrtf(ss / (float)d + eps);
  T* dst = tp.rows + ((size_t)b * T_ + i) * d;
  for (int c = 2 * threadIdx.x; c < d; c += 2 * blockDim.x) {  // (the thread's own channels, a rotated pair whole)
    const float2 w = c == c0 ? w0 : load2(tp.norm_w + c);
    float x = rnd<T>(u[c] * inv * w.x), y = rnd<T>(u[c + 1] * inv * w.y);
    if (c >= d - R) {
      float cs = cs0, sn = sn0;
      if (c != c0) rope_cs(j * ratio, inv_freq, (c - (d - R)) >> 1, &cs, &sn);
      const float x0 = x, y0 = y;
      x = fmaf(x0, cs, -y0 * sn);
      y = fmaf(x0, sn, y0 * cs);
    }
    if (tp.fp8) {
      u[c] = rnd<T>(x);
      u[c + 1] = rnd<T>(y);
    } else {
      store2(dst + c, x, y);
    }
  }
  if (tp.fp8) {
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      float q[4] = {u[4 * lane], u[4 * lane + 1], u[4 * lane + 2], u[4 * lane + 3]};
      float scale;
      const uint32_t packed = fp8_rotate_quantize(q, lane, &scale);
      fp8_row_store(reinterpret_cast<uint8_t*>(tp.rows) + ((size_t)b * T_ + i) * kFp8RowBytes, lane, packed, scale);
    }
  }
}

// ---------------------------------------------------------------- index scores
// Block (node, column share): one warp per column in turn, a lane per head.
template <typename T>
__global__ void __launch_bounds__(256) k_tree_scores(const T* __restrict__ iq, const T* __restrict__ iw, int Hi, int Di,
                                                     const T* __restrict__ ikeys, int cap,
                                                     const T* __restrict__ rows, const int32_t* __restrict__ parent,
                                                     int T_, const int32_t* __restrict__ n_rows,
                                                     const int32_t* __restrict__ pos, int ratio, float wscale,
                                                     float* __restrict__ scores, int32_t* err) {
  pdl_trigger();
  extern __shared__ float sm_ts[];  // [8 warps][Di] key rows
  __shared__ NodeView sv;
  __shared__ int s_ok;
  pdl_wait();
  const int q = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    NodeView v;
    const bool ok = node_view(v, parent, T_, pos, n_rows, cap, ratio, q, err);
    if (lane == 0) {
      sv = v;
      s_ok = ok;
    }
  }
  __syncthreads();
  if (!s_ok) return;
  const int ncol = sv.n + T_;
  float* key = sm_ts + warp * Di;
  const T* qb = iq + (size_t)q * Hi * Di;
  for (int c = blockIdx.y * 8 + warp; c < ncol; c += 8 * gridDim.y) {
    const int node = c - sv.n;
    float s = -INFINITY;
    if (node < 0 || ((sv.closers >> node) & 1)) {
      const T* kr = node < 0 ? ikeys + ((size_t)sv.b * cap + c) * Di : rows + ((size_t)sv.b * T_ + node) * Di;
      __syncwarp();
      for (int e = lane; e < Di; e += 32) key[e] = to_f(kr[e]);
      __syncwarp();
      float tot = 0.f;
      for (int h = lane; h < Hi; h += 32) {
        float d = 0.f;
        for (int e = 0; e < Di; e += 8) {
          float v[8];
          load8_nc(qb + (size_t)h * Di + e, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) d = fmaf(v[k], key[e + k], d);
        }
        tot = fmaf(to_f(iw[(size_t)q * Hi + h]) * wscale, fmaxf(d, 0.f), tot);
      }
      s = warp_sum(tot);
    }
    if (lane == 0) scores[(size_t)q * (cap + T_) + c] = s;
  }
}

// ---------------------------------------------------------------- attention
template <typename T>
struct TreeAttnArgs {
  const T* q;       // [Q, H, D] normalised and rotated
  const T* kv;      // [B, T, D] the nodes' latent rows
  const T* window;  // [B, Wr, D]
  const T* pool;    // [B, cap, D]
  const T* rows;    // [B, T, D] rows that the tree's paths complete
  const int32_t* sel;  // [Q, topk] columns, or null: every visible one
  const TreeNode* nodes;
  const float* sink;
  const float* inv_freq;
  int T_, H, D, R, W, Wr, cap, topk;
  float scale;
  T* out;
};

// One warp per node: the records of a call without a selection.  early: the attention behind it reads nothing ahead of its
// own wait (the persistent kernel; 0.6 us of 64 for 128 nodes); otherwise it starts only once all work before this kernel
// is complete, as behind a selection (indexer.cu, TopkTree).
__global__ void __launch_bounds__(256) k_tree_nodes(const int32_t* __restrict__ parent, int T_, int Q,
                                                    const int32_t* __restrict__ pos,
                                                    const int32_t* __restrict__ n_rows, int cap, int ratio,
                                                    TreeNode* __restrict__ nodes, int early, int32_t* err) {
  if (early) pdl_trigger();
  pdl_wait();
  if (!early) pdl_trigger();
  const int q = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (q >= Q) return;
  NodeView v;
  const bool ok = node_view(v, parent, T_, pos, n_rows, cap, ratio, q, err);
  if ((threadIdx.x & 31) == 0) {
    TreeNode r{};
    r.nsel = -1;
    if (ok) {
      r.mask = v.mask; r.closers = v.closers; r.p = v.p; r.p0 = v.p0; r.n = v.n;
      r.nsel = v.n + __popcll(v.closers);
    }
    nodes[q] = r;
  }
}

// Block (node, head): chunks of 64 keys (selected rows, then the window's tokens), logits one warp per key, then
// each thread accumulates its dims; the running maximum and sum in fp32, the sink once at the end.
template <typename T>
__global__ void __launch_bounds__(128) k_tree_attend(TreeAttnArgs<T> a) {
  pdl_trigger();
  constexpr int kKeys = 64, kMaxC = 8;
  extern __shared__ float sm_ta[];  // [D] query
  __shared__ const T* kp[kKeys];
  __shared__ float lg[kKeys];
  pdl_wait();
  const int h = blockIdx.y, q = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TreeNode sv = a.nodes[q];
  if (sv.nsel < 0) return;
  const int b = q / a.T_, nsel = sv.nsel, nwin = min(a.W, sv.p + 1), nkeys = nsel + nwin;
  float* qs = sm_ta;
  for (int e = tid; e < a.D; e += 128) qs[e] = to_f(a.q[((size_t)q * a.H + h) * a.D + e]);
  float acc[kMaxC];
#pragma unroll
  for (int c = 0; c < kMaxC; ++c) acc[c] = 0.f;
  float m = a.sink[h], l = 1.f;  // the sink is a key without a value
  for (int k0 = 0; k0 < nkeys; k0 += kKeys) {
    __syncthreads();
    const int nk = min(kKeys, nkeys - k0);
    if (tid < nk) {
      const int k = k0 + tid;
      const T* r;
      if (k < nsel) {
        int c = a.sel ? a.sel[(size_t)q * a.topk + k] : (k < sv.n ? k : sv.n + tree_node_at(sv.closers, k - sv.n));
        r = c < sv.n ? a.pool + ((size_t)b * a.cap + c) * a.D : a.rows + ((size_t)b * a.T_ + (c - sv.n)) * a.D;
      } else {
        const int t = sv.p - nwin + 1 + (k - nsel);
        r = t < sv.p0 ? a.window + ((size_t)b * a.Wr + t % a.Wr) * a.D
                      : a.kv + ((size_t)b * a.T_ + tree_node_at(sv.mask, t - sv.p0)) * a.D;
      }
      kp[tid] = r;
    }
    __syncthreads();
    for (int k = warp; k < nk; k += 4) {
      float d = 0.f;
      for (int e = lane * 8; e < a.D; e += 256) {
        float v[8];
        load8(kp[k] + e, v);
#pragma unroll
        for (int x = 0; x < 8; ++x) d = fmaf(qs[e + x], v[x], d);
      }
      d = warp_sum(d);
      if (lane == 0) lg[k] = d * a.scale;
    }
    __syncthreads();
    float mx = m;
    for (int k = 0; k < nk; ++k) mx = fmaxf(mx, lg[k]);
    const float al = m == -INFINITY ? 0.f : expf(m - mx);
    l *= al;
#pragma unroll
    for (int c = 0; c < kMaxC; ++c) acc[c] *= al;
    for (int k = 0; k < nk; ++k) {
      const float pk = lg[k] == -INFINITY ? 0.f : expf(lg[k] - mx);
      l += pk;
#pragma unroll
      for (int c = 0; c < kMaxC; ++c)
        if (tid + 128 * c < a.D) acc[c] = fmaf(pk, to_f(kp[k][tid + 128 * c]), acc[c]);
    }
    m = mx;
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int c = 0; c < kMaxC; ++c) {
    const int e = tid + 128 * c;
    if (128 * c >= a.D) break;  // the same in every thread
    float v = acc[c] * inv;
    const float partner = __shfl_xor_sync(0xffffffffu, v, 1);
    if (e < a.D) {
      if (e >= a.D - a.R) {
        float cs, sn;
        rope_cs(sv.p, a.inv_freq, (e - (a.D - a.R)) >> 1, &cs, &sn);
        v = (e & 1) ? fmaf(-partner, sn, v * cs) : fmaf(v, cs, partner * sn);
      }
      a.out[((size_t)q * a.H + h) * a.D + e] = from_f<T>(v);
    }
  }
}

// ---------------------------------------------------------------- commit
template <typename T>
struct CommitPool {
  const T* proj;
  T* frontier;
  const char* rows;
  char* pool;
  const int32_t* n_rows;
  int32_t* n_rows_out;
  int rowlen, row_bytes, cap;
};
template <typename T>
struct CommitArgs {
  const int32_t* parent;
  const int32_t* leaf;
  const int32_t* pos;
  int32_t* pos_out;
  const T* kv;
  T* window;
  CommitPool<T> pool[2];
  int npool, T_, D, Wr, F, ratio;
  int32_t* err;
};

// A cluster of kCommitCtas blocks per sequence: the accepted path's rows from the draft buffers into the window ring,
// the frontier rings and the pools, a warp per (token, destination), then the new position and row counts.  The
// position may be replaced in place, so every block has read it (a cluster barrier) before the first one writes.
// Nothing is written before the checks.  Latency-bound: a few hundred KB at most, so the copies are spread over enough
// warps that each makes one round trip or two.
// No early trigger: kernels of the next step read positions and ring rows before their own wait.
constexpr int kCommitCtas = 8, kCommitWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kCommitWarps) k_tree_commit(const __grid_constant__ CommitArgs<T> a) {
  __shared__ uint64_t masks[kTreeMax];
  __shared__ int par[kTreeMax], path[kTreeMax];
  pdl_wait();
  const int b = blockIdx.x / kCommitCtas, rank = blockIdx.x % kCommitCtas, tid = threadIdx.x;
  const int leaf = a.leaf[b], p0 = a.pos[b];
  int rows[2] = {0, 0};
  for (int k = 0; k < a.npool; ++k) rows[k] = a.pool[k].n_rows[b];
  const bool tree_ok = tree_masks_block(a.parent + (size_t)b * a.T_, a.T_, masks, par);
  int bad = 0;
  if (!tree_pos_ok(p0) || !tree_ok || leaf < -1 || leaf >= a.T_ || (leaf >= 0 && masks[leaf] == 0)) bad = CSA_DEV_STATE;
  const uint64_t m = bad || leaf < 0 ? 0 : masks[leaf];
  const int n = __popcll(m), end = p0 + n;
  for (int k = 0; k < a.npool; ++k) {
    if (!bad && rows[k] != p0 / a.ratio) bad = CSA_DEV_STATE;
    if (!bad && end / a.ratio > a.pool[k].cap) bad = CSA_DEV_CAPACITY;
  }
  if (tid < n && !bad) path[tid] = tree_node_at(m, tid);
  tc::cluster_sync();
  if (rank == 0 && tid == 0) {
    if (bad) atomicOr(a.err, bad);
    a.pos_out[b] = bad ? p0 : end;
    for (int k = 0; k < a.npool; ++k) a.pool[k].n_rows_out[b] = bad ? rows[k] : end / a.ratio;
  }
  if (bad) return;
  const int lane = tid & 31, kinds = 1 + 2 * a.npool;  // window, then a frontier and a pool per pool
  for (int e = rank * kCommitWarps + (tid >> 5); e < n * kinds; e += kCommitCtas * kCommitWarps) {
    const int k = e / kinds, kind = e - k * kinds, t = p0 + k;
    const size_t row = (size_t)b * a.T_ + path[k];
    const char* src;
    char* dst;
    int bytes;
    if (kind == 0) {
      if (t < end - a.Wr) continue;  // a later token of the path takes the slot
      bytes = a.D * (int)sizeof(T);
      src = reinterpret_cast<const char*>(a.kv + row * a.D);
      dst = reinterpret_cast<char*>(a.window + ((size_t)b * a.Wr + t % a.Wr) * a.D);
    } else {
      const CommitPool<T>& cp = a.pool[(kind - 1) >> 1];
      if (kind & 1) {
        if (t < end - a.F) continue;
        bytes = cp.rowlen * (int)sizeof(T);
        src = reinterpret_cast<const char*>(cp.proj + row * cp.rowlen);
        dst = reinterpret_cast<char*>(cp.frontier + ((size_t)b * a.F + t % a.F) * cp.rowlen);
      } else {
        if ((t + 1) % a.ratio) continue;
        bytes = cp.row_bytes;
        src = cp.rows + row * cp.row_bytes;
        dst = cp.pool + ((size_t)b * cp.cap + (t + 1) / a.ratio - 1) * cp.row_bytes;
      }
    }
    for (int o = lane * 16; o < bytes; o += 4 * 512) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (o + 512 * u < bytes) v[u] = *reinterpret_cast<const uint4*>(src + o + 512 * u);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (o + 512 * u < bytes) *reinterpret_cast<uint4*>(dst + o + 512 * u) = v[u];
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const Dims& L, const csa_rows* rows, int n, int B, int T, const int32_t* parent,
                             const int32_t* pos, const float* inv_freq, int32_t* err, cudaStream_t s) {
  if (L.dtype == CSA_BF16) return norm_rope_t<__nv_bfloat16>(L, rows, n, B, T, parent, pos, inv_freq, err, s);
  return norm_rope_t<float>(L, rows, n, B, T, parent, pos, inv_freq, err, s);
}

void* carve_compress_tree(Carver& c, const Dims& L, int d, int B, int T) {
  if (tc_tree_project_supported(L, d)) return nullptr;
  return c.take<char>((size_t)B * T * 2 * L.lanes * d * esize(L.dtype));
}

template <typename T>
static cudaError_t compress_tree_t(const Dims& L, const TreeCompress* pools, int npool, const void* x, int B, int T_,
                                   const int32_t* parent, const int32_t* pos, const float* inv_freq, int32_t* err,
                                   cudaStream_t s) {
  TreePool<T> tp[2];
  // pools on the tensor cores share a grid; the others are projected one by one into the workspace
  TreeCompress tc_pools[2];
  int ntc = 0;
  for (int k = 0; k < npool; ++k) {
    const TreeCompress& c = pools[k];
    const int d = c.comp->d;
    const bool on_tc = tc_tree_project_supported(L, d);
    if (on_tc) {
      tc_pools[ntc++] = c;
    } else {
      const cudaError_t e = launch_project_simt(L, d, x, B * T_, c.comp->wkv, c.comp->wgate, c.ws, s);
      if (e != cudaSuccess) return e;
    }
    tp[k] = TreePool<T>{static_cast<const T*>(c.frontier), static_cast<const T*>(on_tc ? c.proj : c.ws),
                        static_cast<T*>(c.proj), static_cast<T*>(c.rows), c.comp->ape, c.comp->norm_w, d,
                        L.ikey_fp8 && d == L.Di && k == 1};
  }
  if (ntc > 0) {
    const cudaError_t e = launch_tc_tree_project(L, tc_pools, ntc, x, B, T_, parent, pos, err, s);
    if (e != cudaSuccess) return e;
  }
  if (npool == 1) tp[1] = tp[0];
  const int dm = max(tp[0].d, tp[1].d);
  CSA_LAUNCH(k_tree_pool<T>, dim3(T_, B, npool), dim3(256), ((size_t)dm + 32) * sizeof(float), s, tp[0], tp[1], T_,
             L.ratio, L.lanes, L.R, L.F, L.eps, parent, pos, inv_freq, err);
  return cudaGetLastError();
}

cudaError_t launch_compress_tree(const Dims& L, const TreeCompress* pools, int npool, const void* x, int B, int T,
                                 const int32_t* parent, const int32_t* pos, const float* inv_freq, int32_t* err,
                                 cudaStream_t s) {
  if (L.dtype == CSA_BF16)
    return compress_tree_t<__nv_bfloat16>(L, pools, npool, x, B, T, parent, pos, inv_freq, err, s);
  return compress_tree_t<float>(L, pools, npool, x, B, T, parent, pos, inv_freq, err, s);
}

template <typename T>
static cudaError_t index_scores_tree_t(const Dims& L, const void* iq, const void* iw, int B, int T_,
                                       const int32_t* parent, const void* ikeys, int cap, const void* rows,
                                       const int32_t* n_rows, const int32_t* pos, float* scores, int32_t* err,
                                       cudaStream_t s) {
  const float wscale = (float)(1.0 / sqrt((double)L.Di * (double)L.Hi));
  CSA_LAUNCH(k_tree_scores<T>, dim3(B * T_, min(1024, (cap + T_ + 63) / 64)), dim3(256),
             8 * (size_t)L.Di * sizeof(float), s, static_cast<const T*>(iq), static_cast<const T*>(iw), L.Hi, L.Di,
             static_cast<const T*>(ikeys), cap, static_cast<const T*>(rows), parent, T_, n_rows, pos, L.ratio, wscale, scores, err);
  return cudaGetLastError();
}

cudaError_t launch_index_scores_tree(const Dims& L, const void* iq, const void* iw, int B, int T,
                                     const int32_t* parent, const void* ikeys, int cap, const void* rows,
                                     const int32_t* n_rows, const int32_t* pos, float* scores, void* ws, int32_t* err,
                                     cudaStream_t s) {
  if (tc_tree_scores_supported(L, B, cap))
    return launch_tc_tree_scores(L, iq, iw, B, T, parent, ikeys, cap, rows, n_rows, pos, scores, ws, err, s);
  if (L.ikey_fp8) return cudaErrorNotSupported;  // (a pool of 2^31 rows)
  if (L.dtype == CSA_BF16)
    return index_scores_tree_t<__nv_bfloat16>(L, iq, iw, B, T, parent, ikeys, cap, rows, n_rows, pos, scores, err, s);
  return index_scores_tree_t<float>(L, iq, iw, B, T, parent, ikeys, cap, rows, n_rows, pos, scores, err, s);
}

TreeAttendWs carve_attend_tree(Carver& c, const Dims& L, int B, int T, int cap) {
  TreeAttendWs w{};
  (void)cap;
  w.nodes = c.take<TreeNode>((size_t)B * T);
  if (L.has_indexer()) w.sel = c.take<int32_t>((size_t)B * T * L.topk);
  return w;
}

template <typename T>
static cudaError_t attend_tree_t(const Dims& L, const TreeAttend& t, int32_t* err, cudaStream_t s) {
  const int Q = t.B * t.T;
  TreeAttnArgs<T> a{};
  // Tensor-core shapes.  Few nodes: S splits of one 160-row tile each, a cluster per query, while all clusters run at
  // once; eight of half a tile where four would do (8 nodes of 640 keys: 22.5 us instead of 23.4).  More nodes or keys
  // (S = 0): tc_tree_attend.cu.
  const bool codes_fit = (long long)t.B * t.cap < INT32_MAX && (long long)t.B * L.Wr < (1 << 28);
  const bool on_tc = tc_attend_supported(L) && codes_fit;
  int S = 0;
  if (on_tc) {
    const long long n_max = t.scores ? L.topk : (long long)t.cap + t.T;
    S = 1;
    while (S <= 4 && ((L.W + S - 1) / S + (n_max + S - 1) / S > 160 || Q > tc_attend_tree_split_max(S))) S *= 2;
    if (S > 4) S = 0;
    if (S == 4 && L.W + n_max >= 8 * 80 && Q <= tc_attend_tree_split_max(8)) S = 8;
  }
  if (t.scores) {
    int32_t* sel = t.sel_out ? t.sel_out : t.ws.sel;
    cudaError_t e = launch_topk_tree(L, t.scores, t.B, t.T, t.parent, t.cap, t.n_rows, t.pos, sel, t.ws.nodes, err, s);
    if (e != cudaSuccess) return e;
    a.sel = sel;
  } else {
    CSA_LAUNCH(k_tree_nodes, dim3((Q + 7) / 8), dim3(256), 0, s, t.parent, t.T, Q, t.pos, t.n_rows, t.cap, L.ratio,
               t.ws.nodes, on_tc && S == 0, err);
  }
  if (S > 0) return launch_tc_attend_tree_split(L, t, a.sel, S, err, s);
  if (on_tc) return launch_tc_attend_tree(L, t, a.sel, err, s);
  a.q = static_cast<const T*>(t.q); a.kv = static_cast<const T*>(t.kv); a.window = static_cast<const T*>(t.window);
  a.pool = static_cast<const T*>(t.pool); a.rows = static_cast<const T*>(t.rows);
  a.nodes = t.ws.nodes; a.sink = t.sink; a.inv_freq = t.inv_freq;
  a.T_ = t.T; a.H = L.H; a.D = L.D; a.R = L.R; a.W = L.W; a.Wr = L.Wr; a.cap = t.cap; a.topk = L.topk;
  a.scale = L.scale; a.out = static_cast<T*>(t.out);
  CSA_LAUNCH(k_tree_attend<T>, dim3(Q, L.H), dim3(128), L.D * sizeof(float), s, a);
  return cudaGetLastError();
}

cudaError_t launch_attend_tree(const Dims& L, const TreeAttend& t, int32_t* err, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? attend_tree_t<__nv_bfloat16>(L, t, err, s) : attend_tree_t<float>(L, t, err, s);
}

template <typename T>
static cudaError_t commit_tree_t(const Dims& L, const TreeCommit& c, int32_t* err, cudaStream_t s) {
  CommitArgs<T> a{};
  a.parent = c.parent; a.leaf = c.leaf; a.pos = c.pos; a.pos_out = c.pos_out;
  a.kv = static_cast<const T*>(c.kv); a.window = static_cast<T*>(c.window);
  a.npool = c.npool; a.T_ = c.T; a.D = L.D; a.Wr = L.Wr; a.F = L.F; a.ratio = L.ratio; a.err = err;
  for (int k = 0; k < c.npool; ++k) {
    const int d = k ? L.Di : L.D;
    a.pool[k] = CommitPool<T>{static_cast<const T*>(c.proj[k]), static_cast<T*>(c.frontier[k]),
                              static_cast<const char*>(c.rows[k]), static_cast<char*>(c.pool[k]), c.n_rows[k],
                              c.n_rows_out[k], 2 * L.lanes * d,
                              k && L.ikey_fp8 ? kFp8RowBytes : d * (int)sizeof(T), c.cap[k]};
  }
  const cudaError_t e = launch_pdl_cluster(k_tree_commit<T>, dim3(c.B * kCommitCtas), dim3(32 * kCommitWarps), 0, s,
                                           kCommitCtas, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_commit_tree(const Dims& L, const TreeCommit& c, int32_t* err, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? commit_tree_t<__nv_bfloat16>(L, c, err, s) : commit_tree_t<float>(L, c, err, s);
}

}  // namespace csa
