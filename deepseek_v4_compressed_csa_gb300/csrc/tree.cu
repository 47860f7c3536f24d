// Verifying a tree of drafted tokens: the portable kernels (any head layout and size, bf16 and fp32).
//
// Definitions (include/csa.h): a node's row, scores and output are what sequential decoding along the node's path
// would give; nothing of the tree enters the cache before commit.
#include "tree.cuh"

#include "fp8_row.cuh"
#include "kernels.h"

namespace csa {

namespace {

// ---------------------------------------------------------------- norm and rotation
// y = x rsqrt(mean(x^2) + eps) w, then the last R dims of the row turned by the token's position.  One pass: a row
// is read once into registers (fp32), its square sum reduced inside the lanes that hold it, and written once,
// rounded once.  Bound by memory: 2 x the tensors' bytes.
constexpr int kNrParts = 4;
constexpr int kNrThreads = 256;

template <typename T>
struct NrPart {
  const T* x;
  T* out;
  const float* w;
  int heads, dim, norm, lpr_log2;  // lpr: lanes that hold a row (a power of two, at most 32)
  long long x_stride;              // elements between tokens
};
template <typename T>
struct NrArgs {
  NrPart<T> part[kNrParts];
  int n_parts, rows, R, T_, B;     // rows: row groups (one warp pass each) of a token over all parts
  int groups_per_block;
  int first[kNrParts + 1];         // first row group of each part
  const int32_t* parent;
  const int32_t* pos;
  const float* inv_freq;
  float eps;
  int32_t* err;
};

template <typename T, int kChunks>
__device__ __forceinline__ void norm_rope_rows(const NrPart<T>& pt, int tok, int row, int R, float eps, bool rotate,
                                               const float* rc, const float* rs) {
  const int lane = threadIdx.x & 31, lpr = 1 << pt.lpr_log2, sub = lane & (lpr - 1);
  const int h = row + (lane >> pt.lpr_log2);
  const bool live = h < pt.heads;
  const int n8 = pt.dim >> 3;
  const T* src = pt.x + (size_t)tok * pt.x_stride + (size_t)h * pt.dim;
  float v[kChunks][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = sub + i * lpr;
    if (live && c < n8) {
      load8(src + 8 * c, v[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
  }
  float inv = 1.f;
  if (pt.norm) {
    for (int o = lpr >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    inv = 1.0f / sqrtf(ss / (float)pt.dim + eps);
  }
  T* dst = pt.out + ((size_t)tok * pt.heads + h) * pt.dim;
  const int r0 = pt.dim - R;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = sub + i * lpr;
    if (!live || c >= n8) continue;
    if (pt.norm) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= inv;
      if (pt.w) {
        float w[8];
        load8_nc(pt.w + 8 * c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
      }
    }
    if (rotate && 8 * c >= r0) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const int k = (8 * c + e - r0) >> 1;
        const float a = v[i][e], b = v[i][e + 1];
        v[i][e] = fmaf(a, rc[k], -b * rs[k]);
        v[i][e + 1] = fmaf(a, rs[k], b * rc[k]);
      }
    }
    store8(dst + 8 * c, v[i]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kNrThreads) k_norm_rope(NrArgs<T> a) {
  // no early trigger: kernels of later calls read queries and keys before their own wait
  extern __shared__ float sm_nr[];
  float* rc = sm_nr;
  float* rs = sm_nr + a.R / 2;
  __shared__ int s_depth;
  pdl_wait();
  const int tok = blockIdx.x, b = tok / a.T_, i = tok - b * a.T_;
  int depth = i;
  if (a.parent) {
    if (threadIdx.x < 32) {
      bool bad = false;
      const uint64_t m = tree_path_warp(a.parent + (size_t)b * a.T_, a.T_, i, bad);
      if (threadIdx.x == 0) {
        s_depth = __popcll(m) - 1;
        if (bad) atomicOr(a.err, CSA_DEV_STATE);
      }
    }
    __syncthreads();
    depth = s_depth;
    if (depth < 0) return;
  }
  const bool rotate = a.inv_freq != nullptr;
  if (rotate) {
    const int p = a.pos[b] + depth;
    if (a.pos[b] < 0) {
      if (threadIdx.x == 0) atomicOr(a.err, CSA_DEV_STATE);
      return;
    }
    for (int k = threadIdx.x; k < a.R / 2; k += blockDim.x) rope_cs(p, a.inv_freq, k, rc + k, rs + k);
    __syncthreads();
  }
  const int g1 = min(a.rows, (int)(blockIdx.y + 1) * a.groups_per_block);
  for (int g = blockIdx.y * a.groups_per_block + (threadIdx.x >> 5); g < g1; g += kNrThreads / 32) {
    int k = 0;
    while (k + 1 < a.n_parts && g >= a.first[k + 1]) ++k;
    const NrPart<T>& pt = a.part[k];
    const int row = (g - a.first[k]) << (5 - pt.lpr_log2);
    const int chunks = ((pt.dim >> 3) + (1 << pt.lpr_log2) - 1) >> pt.lpr_log2;
    if (chunks == 1) norm_rope_rows<T, 1>(pt, tok, row, a.R, a.eps, rotate, rc, rs);
    else if (chunks == 2) norm_rope_rows<T, 2>(pt, tok, row, a.R, a.eps, rotate, rc, rs);
    else norm_rope_rows<T, 4>(pt, tok, row, a.R, a.eps, rotate, rc, rs);
  }
}

template <typename T>
cudaError_t norm_rope_t(const Dims& L, const csa_rows* rows, int n, int B, int T_, const int32_t* parent,
                        const int32_t* pos, const float* inv_freq, int32_t* err, cudaStream_t s) {
  NrArgs<T> a{};
  a.n_parts = n;
  a.R = L.R; a.T_ = T_; a.B = B; a.parent = parent; a.pos = pos; a.inv_freq = inv_freq; a.eps = L.eps; a.err = err;
  int groups = 0;
  for (int k = 0; k < n; ++k) {
    NrPart<T>& p = a.part[k];
    p.x = static_cast<const T*>(rows[k].x);
    p.out = static_cast<T*>(rows[k].out);
    p.w = rows[k].weight;
    p.heads = rows[k].heads;
    p.dim = rows[k].dim;
    p.norm = rows[k].norm;
    p.x_stride = rows[k].x_stride > 0 ? rows[k].x_stride : (long long)p.heads * p.dim;
    p.lpr_log2 = 0;
    while ((1 << p.lpr_log2) < 32 && (1 << p.lpr_log2) < p.dim / 8) ++p.lpr_log2;
    a.first[k] = groups;
    groups += (p.heads + (32 >> p.lpr_log2) - 1) / (32 >> p.lpr_log2);
  }
  a.first[n] = groups;
  a.rows = groups;
  a.groups_per_block = kNrThreads / 32;
  const int gy = (groups + a.groups_per_block - 1) / a.groups_per_block;
  CSA_LAUNCH(k_norm_rope<T>, dim3(B * T_, gy), dim3(kNrThreads), L.R * sizeof(float), s, a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- rows that the tree's paths complete
template <typename T>
struct TreePool {
  const T* frontier;  // [B, F, 2 L d]
  const T* src;       // [B, T, 2 L d] the projections of every slot
  T* proj;            // [B, T, 2 L d] the draft buffer that keeps the nodes'
  T* rows;            // [B, T, d], or fp8 rows
  const float* ape;
  const float* norm_w;
  int d, fp8;
};

// Block (i, b, pool): node i of sequence b.  If its token completes window j along its path, the row that the
// compressor would emit: entries before pos from the frontier ring, from pos on the path's nodes.  Arithmetic and
// roundings are those of the committed rows (compress.cu), so that an accepted row is the row decoding would have
// written.
template <typename T>
__global__ void __launch_bounds__(256) k_tree_pool(TreePool<T> pa, TreePool<T> pi, int T_, int ratio, int lanes, int R,
                                                   int F, float eps, const int32_t* __restrict__ parent,
                                                   const int32_t* __restrict__ pos,
                                                   const float* __restrict__ inv_freq, int32_t* err) {
  pdl_trigger();
  extern __shared__ float sm_tp[];  // [d] pooled, [d] normed, 32 reduction slots
  __shared__ uint64_t s_mask;
  __shared__ int s_path[kTreeMax];
  const bool second = blockIdx.z != 0;
  const T* __restrict__ frontier = second ? pi.frontier : pa.frontier;
  const T* __restrict__ src = second ? pi.src : pa.src;
  T* proj = second ? pi.proj : pa.proj;
  T* rows = second ? pi.rows : pa.rows;
  const float* __restrict__ ape = second ? pi.ape : pa.ape;
  const float* __restrict__ norm_w = second ? pi.norm_w : pa.norm_w;
  const int d = second ? pi.d : pa.d, fp8 = second ? pi.fp8 : pa.fp8;
  float* u = sm_tp;
  float* y = u + d;
  float* red = y + d;
  pdl_wait();
  const int i = blockIdx.x, b = blockIdx.y, p0 = pos[b];
  if (threadIdx.x < 32) {
    bool bad = false;
    const uint64_t m = tree_path_warp(parent + (size_t)b * T_, T_, i, bad);
    if (threadIdx.x == 0) {
      s_mask = p0 < 0 ? 0 : m;
      if (bad || p0 < 0) atomicOr(err, CSA_DEV_STATE);
      int k = 0;
      for (uint64_t r = m; r; r &= r - 1) s_path[k++] = __ffsll((long long)r) - 1;
    }
  }
  __syncthreads();
  if (s_mask == 0) return;
  const int Ld = lanes * d, rowlen = 2 * Ld, p = p0 + __popcll(s_mask) - 1;
  const T* pj = src + (size_t)b * T_ * rowlen;
  for (int e = threadIdx.x * 8; e < rowlen; e += blockDim.x * 8)
    copy8<T>(proj + ((size_t)b * T_ + i) * rowlen + e, pj + (size_t)i * rowlen + e);
  if ((p + 1) % ratio != 0) return;
  const int j = (p + 1) / ratio - 1;
  const T* fr = frontier + (size_t)b * F * rowlen;
  const int t_lo = lanes == 2 ? max(0, (j - 1) * ratio) : j * ratio;
  const int t_hi = (j + 1) * ratio;
  float ss = 0.f;
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float m = -INFINITY, num = 0.f, den = 0.f;
    for (int t0 = t_lo; t0 < t_hi; t0 += 8) {
      float sv[8], kv[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int t = t0 + k;
        sv[k] = -INFINITY;
        kv[k] = 0.f;
        if (t < t_hi) {
          const int l = (lanes == 2 && t >= j * ratio) ? 1 : 0;
          const T* row = t < p0 ? fr + (size_t)(t % F) * rowlen : pj + (size_t)s_path[t - p0] * rowlen;
          kv[k] = to_f(row[l * d + c]);
          sv[k] = to_f(row[Ld + l * d + c]) + __ldg(ape + (size_t)(t % ratio) * Ld + l * d + c);
        }
      }
      float cm = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) cm = fmaxf(cm, sv[k]);
      const float al = (m == -INFINITY) ? 0.f : expf(m - cm);
      num *= al;
      den *= al;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float e = (sv[k] == -INFINITY) ? 0.f : expf(sv[k] - cm);
        den += e;
        num = fmaf(e, kv[k], num);
      }
      m = cm;
    }
    const float uc = rnd<T>(num / den);
    u[c] = uc;
    ss = fmaf(uc, uc, ss);
  }
  ss = block_sum(ss, red);
  const float inv = 1.0f / sqrtf(ss / (float)d + eps);
  for (int c = threadIdx.x; c < d; c += blockDim.x) y[c] = rnd<T>(u[c] * inv * __ldg(norm_w + c));
  __syncthreads();
  T* dst = rows + ((size_t)b * T_ + i) * d;
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float v = y[c];
    if (c >= d - R) {
      const int k = (c - (d - R)) >> 1;
      float cs, sn;
      rope_cs(j * ratio, inv_freq, k, &cs, &sn);
      const float x0 = y[d - R + 2 * k], x1 = y[d - R + 2 * k + 1];
      v = ((c - (d - R)) & 1) ? fmaf(x0, sn, x1 * cs) : fmaf(x0, cs, -x1 * sn);
    }
    if (fp8)
      u[c] = rnd<T>(v);
    else
      dst[c] = from_f<T>(v);
  }
  if (fp8) {
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      float q[4] = {u[4 * lane], u[4 * lane + 1], u[4 * lane + 2], u[4 * lane + 3]};
      float scale;
      const uint32_t packed = fp8_rotate_quantize(q, lane, &scale);
      fp8_row_store(reinterpret_cast<uint8_t*>(rows) + ((size_t)b * T_ + i) * kFp8RowBytes, lane, packed, scale);
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

// One warp per node: the records of a call without a selection.
__global__ void __launch_bounds__(256) k_tree_nodes(const int32_t* __restrict__ parent, int T_, int Q,
                                                    const int32_t* __restrict__ pos,
                                                    const int32_t* __restrict__ n_rows, int cap, int ratio,
                                                    TreeNode* __restrict__ nodes, int32_t* err) {
  pdl_trigger();
  pdl_wait();
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

// One block per sequence: the accepted path's rows from the draft buffers into the window ring, the frontier rings
// and the pools, then the new position and row counts.  Nothing is written before the checks.
// No early trigger: kernels of the next step read positions and ring rows before their own wait.
template <typename T>
__global__ void __launch_bounds__(512) k_tree_commit(CommitArgs<T> a) {
  __shared__ uint64_t masks[kTreeMax];
  __shared__ int par[kTreeMax], path[kTreeMax];
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x;
  const bool tree_ok = tree_masks_block(a.parent + (size_t)b * a.T_, a.T_, masks, par);
  const int leaf = a.leaf[b], p0 = a.pos[b];
  int bad = 0;
  if (p0 < 0 || !tree_ok || leaf < -1 || leaf >= a.T_ || (leaf >= 0 && masks[leaf] == 0)) bad = CSA_DEV_STATE;
  const uint64_t m = bad || leaf < 0 ? 0 : masks[leaf];
  const int n = __popcll(m), end = p0 + n;
  for (int k = 0; k < a.npool; ++k) {
    if (!bad && a.pool[k].n_rows[b] != p0 / a.ratio) bad = CSA_DEV_STATE;
    if (!bad && end / a.ratio > a.pool[k].cap) bad = CSA_DEV_CAPACITY;
  }
  if (bad && tid == 0) atomicOr(a.err, bad);
  if (tid < n && !bad) path[tid] = tree_node_at(m, tid);
  __syncthreads();  // every thread has read the positions and counts before thread 0 may replace them
  if (tid == 0) {
    a.pos_out[b] = bad ? p0 : end;
    for (int k = 0; k < a.npool; ++k) a.pool[k].n_rows_out[b] = bad ? a.pool[k].n_rows[b] : end / a.ratio;
  }
  if (bad) return;
  auto copy = [&](char* dst, const char* src, int bytes) {
    for (int e = tid * 16; e < bytes; e += blockDim.x * 16)
      *reinterpret_cast<uint4*>(dst + e) = *reinterpret_cast<const uint4*>(src + e);
  };
  for (int k = 0; k < n; ++k) {
    const int t = p0 + k, node = path[k];
    const size_t row = (size_t)b * a.T_ + node;
    if (t >= end - a.Wr)  // a later token of the path takes the slot otherwise
      copy(reinterpret_cast<char*>(a.window + ((size_t)b * a.Wr + t % a.Wr) * a.D),
           reinterpret_cast<const char*>(a.kv + row * a.D), a.D * (int)sizeof(T));
    for (int g = 0; g < a.npool; ++g) {
      const CommitPool<T>& cp = a.pool[g];
      if (t >= end - a.F)
        copy(reinterpret_cast<char*>(cp.frontier + ((size_t)b * a.F + t % a.F) * cp.rowlen),
             reinterpret_cast<const char*>(cp.proj + row * cp.rowlen), cp.rowlen * (int)sizeof(T));
      if ((t + 1) % a.ratio == 0)
        copy(cp.pool + ((size_t)b * cp.cap + (t + 1) / a.ratio - 1) * cp.row_bytes, cp.rows + row * cp.row_bytes,
             cp.row_bytes);
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const Dims& L, const csa_rows* rows, int n, int B, int T, const int32_t* parent,
                             const int32_t* pos, const float* inv_freq, int32_t* err, cudaStream_t s) {
  if (L.dtype == CSA_BF16) return norm_rope_t<__nv_bfloat16>(L, rows, n, B, T, parent, pos, inv_freq, err, s);
  return norm_rope_t<float>(L, rows, n, B, T, parent, pos, inv_freq, err, s);
}

template <typename T>
static cudaError_t compress_tree_t(const Dims& L, const TreeCompress* pools, int npool, const void* x, int B, int T_,
                                   const int32_t* parent, const int32_t* pos, const float* inv_freq, int32_t* err,
                                   cudaStream_t s) {
  TreePool<T> tp[2];
  for (int k = 0; k < npool; ++k) {
    const TreeCompress& c = pools[k];
    const int d = c.comp->d;
    // every slot is projected into the workspace; the pooling kernel keeps the nodes' rows
    cudaError_t e = tc_project_supported(L, d)
                        ? launch_tc_project(L, d, x, B * T_, c.comp->wkv, c.comp->wgate, c.ws.proj, c.ws.part,
                                            c.ws.tickets, true, err, s)
                        : launch_project_simt(L, d, x, B * T_, c.comp->wkv, c.comp->wgate, c.ws.proj, s);
    if (e != cudaSuccess) return e;
    tp[k] = TreePool<T>{static_cast<const T*>(c.frontier), static_cast<const T*>(c.ws.proj), static_cast<T*>(c.proj), static_cast<T*>(c.rows),
                        c.comp->ape, c.comp->norm_w, d, L.ikey_fp8 && d == L.Di && k == 1};
  }
  if (npool == 1) tp[1] = tp[0];
  const int dm = max(tp[0].d, tp[1].d);
  CSA_LAUNCH(k_tree_pool<T>, dim3(T_, B, npool), dim3(256), (2 * (size_t)dm + 32) * sizeof(float), s, tp[0], tp[1], T_,
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
  CSA_LAUNCH(k_tree_scores<T>, dim3(B * T_, min(1024, (cap + T_ + 63) / 64)), dim3(256), 8 * (size_t)L.Di * sizeof(float), s,
             static_cast<const T*>(iq), static_cast<const T*>(iw), L.Hi, L.Di, static_cast<const T*>(ikeys), cap,
             static_cast<const T*>(rows), parent, T_, n_rows, pos, L.ratio, wscale, scores, err);
  return cudaGetLastError();
}

cudaError_t launch_index_scores_tree(const Dims& L, const void* iq, const void* iw, int B, int T,
                                     const int32_t* parent, const void* ikeys, int cap, const void* rows,
                                     const int32_t* n_rows, const int32_t* pos, float* scores, int32_t* err,
                                     cudaStream_t s) {
  if (tc_tree_scores_supported(L, B, cap))
    return launch_tc_tree_scores(L, iq, iw, B, T, parent, ikeys, cap, rows, n_rows, pos, scores, err, s);
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
  if (t.scores) {
    int32_t* sel = t.sel_out ? t.sel_out : t.ws.sel;
    cudaError_t e = launch_topk_tree(L, t.scores, t.B, t.T, t.parent, t.cap, t.n_rows, t.pos, sel, t.ws.nodes, err, s);
    if (e != cudaSuccess) return e;
    a.sel = sel;
  } else {
    CSA_LAUNCH(k_tree_nodes, dim3((Q + 7) / 8), dim3(256), 0, s, t.parent, t.T, Q, t.pos, t.n_rows, t.cap, L.ratio,
               t.ws.nodes, err);
  }
  // Tensor-core shapes.  Few nodes: S splits of one 160-row tile each, a cluster per query, while every split has an
  // SM.  More: a CTA per query streaming its tiles.
  const bool codes_fit = (long long)t.B * t.cap < INT32_MAX && (long long)t.B * L.Wr < (1 << 28);
  if (tc_attend_supported(L) && codes_fit) {
    int sms = 0, dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int n_max = t.scores ? L.topk : t.cap + t.T;
    for (int S = 1; S <= 4; S *= 2)
      if ((L.W + S - 1) / S + (n_max + S - 1) / S <= 160 && (long)Q * S <= sms && (S == 1 || tc_attend_decode_cluster(S)))
        return launch_tc_attend_tree_split(L, t, a.sel, S, err, s);
    return launch_tc_attend_tree(L, t, a.sel, err, s);
  }
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
  CSA_LAUNCH(k_tree_commit<T>, dim3(c.B), dim3(512), 0, s, a);
  return cudaGetLastError();
}

cudaError_t launch_commit_tree(const Dims& L, const TreeCommit& c, int32_t* err, cudaStream_t s) {
  return L.dtype == CSA_BF16 ? commit_tree_t<__nv_bfloat16>(L, c, err, s) : commit_tree_t<float>(L, c, err, s);
}

}  // namespace csa
