// Internal interface between the C-ABI entry points (api.cu) and the kernel
// translation units.  Host-side only declarations; no torch types anywhere.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/csa.h"

namespace csa {

// Validated layer dimensions.
struct Dims {
  int dtype, H, D, R, W, ratio, Hi, Di, topk, X;
  float scale, eps;
  int lanes;     // 2 when ratio == 4 (overlapping windows), else 1
  int rollback;  // tokens csa_trim may rewind
  int Wr;        // window ring slots: W + rollback (a query attends its last W tokens)
  int F;         // frontier ring slots: 2 ratio (ratio 4) or ratio, + rollback (the journal)
  int ikey_fp8;  // index keys as fp8 rows (CSA_FP8_ROW_BYTES each: 128 E4M3 codes of the rotated row, fp32 scale)
  bool has_indexer() const { return ratio == 4; }
};

// Carves 256-byte aligned sub-buffers out of the caller's workspace; with a
// null base it only measures.
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename E> E* take(size_t n) {
    off = (off + 255) & ~size_t(255);
    E* p = base ? reinterpret_cast<E*>(base + off) : nullptr;
    off += n * sizeof(E);
    return p;
  }
};

inline size_t esize(int dtype) { return dtype == CSA_BF16 ? 2 : 4; }

// Number of kernels this library has enqueued in this process (diagnostics).
void count_launches(int n);

// Launch with programmatic stream serialization (see pdl_trigger / pdl_wait).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The same with thread-block clusters of cluster_x consecutive blocks (grid.x a multiple of cluster_x).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                      int cluster_x, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster_x;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Lets `kernel` be launched with up to kBytes of dynamic shared memory.  The limit belongs to the function on the device,
// not to a launch: set to one call's need, it would fall under a larger call's that another host thread is about to
// launch.  So it is a constant, the most that any call takes.
template <int kBytes, typename... KArgs>
inline void allow_smem(void (*kernel)(KArgs...)) {
  static_assert(kBytes <= 232448, "shared memory per block");
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
}

// Clusters of S blocks that the current device runs at once.  A cluster stays within one GPC, so that is less than
// SMs / S blocks (of one block an SM, 23 clusters of 6 and 15 of 7 on 152 SMs): a grid of more has a second wave.
template <typename... KArgs>
inline int max_clusters(void (*kernel)(KArgs...), int threads, size_t smem, int S) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(S);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();  // leave no sticky error behind
    return 0;
  }
  return n;
}

#define CSA_LAUNCH(...)                           \
  do {                                            \
    cudaError_t csa_e_ = launch_pdl(__VA_ARGS__); \
    if (csa_e_ != cudaSuccess) return csa_e_;     \
  } while (0)

// ---- compress.cu
struct CompressWs {
  int32_t* flags;  // [B] 1 = sequence valid for this call
  void* proj;      // [B*T, 2*L*d] model dtype: kv | gate of every new token
  float* part;     // tensor-core projection: split-K partials (or null)
  int* tickets;    // tensor-core projection: per-tile arrival counters (or null)
};
CompressWs carve_compress(Carver& c, const Dims& L, int d, int B, int T);
// The attention pool (ca, workspace wa) and the index pool (ci, wi) of one call's tokens.
cudaError_t launch_compress_pair(const Dims& L, const csa_compressor& ca, const csa_compressor& ci, const void* x,
                                 int B, int T, const int32_t* pos, void* fa, void* pa, int cap_a, int32_t* na,
                                 void* fi, void* pi, int cap_i, int32_t* ni, const float* inv_freq,
                                 const CompressWs& wa, const CompressWs& wi, int32_t* err, cudaStream_t s);
cudaError_t launch_compress(const Dims& L, const csa_compressor& comp, const void* x, int B, int T,
                            const int32_t* pos, void* frontier, void* pool, int cap, int32_t* n_rows,
                            const float* inv_freq, const CompressWs& ws, int32_t* err, cudaStream_t s);
// A packed variable-length batch: x [N, X], sequence b's chunk = rows cu[b] .. cu[b+1]-1 at positions pos[b] ..;
// ws carved for B sequences and N tokens (carve_compress(c, L, d, B, ceil(N / B)) is not enough: use
// carve_compress_varlen).  A sequence whose row-table entries are inconsistent is flagged CSA_DEV_STATE and left.
cudaError_t launch_compress_varlen(const Dims& L, const csa_compressor& comp, const void* x, int B,
                                   const int32_t* cu, int N, int T_max, const int32_t* pos, void* frontier,
                                   void* pool, int cap, int32_t* n_rows, const float* inv_freq,
                                   const CompressWs& ws, int32_t* err, cudaStream_t s);
CompressWs carve_compress_varlen(Carver& c, const Dims& L, int d, int B, int N);

// The projection of ntok tokens into proj [ntok, 2*L*d] on the SIMT path (any type and size).
cudaError_t launch_project_simt(const Dims& L, int d, const void* x, int ntok, const void* wkv, const void* wgate,
                                void* proj, cudaStream_t s);

// ---- indexer.cu
struct IndexWs {
  float* qr;      // [Q, Hi, Di] roped index queries (model-dtype values held as fp32)
  float* scores;  // [Q, cap]
};
IndexWs carve_index(Carver& c, const Dims& L, int Q, int cap);
// The indexer in two stages around `ready` (an event recorded after the index pool's compress call for the same
// token, possibly on another stream; null: no wait): the scan of the rows complete before the token, then,
// after the event, the rows that call may have written and the selection.  Decode, tensor-core shapes only;
// otherwise the whole call waits for the event and runs as launch_index_topk.
cudaError_t launch_index_topk_overlapped(const Dims& L, const void* iq, const void* iw, int Q, const void* ikeys,
                                         int cap, const int32_t* n_rows, const int32_t* pos, const float* inv_freq,
                                         int32_t* sel, int32_t* n_sel, const IndexWs& ws, int32_t* err,
                                         cudaStream_t s, cudaEvent_t ready);
// Scores and top-k for Q queries.  Query q belongs to sequence bseq(q) at position p(q): without pos, 0 and
// pos0 + q (one chunk); with pos, q / t and pos[q / t] + q % t, t = max(1, pos0) (decode, verify blocks); with
// cu (a packed variable-length batch of pos0 sequences, row table cu [pos0 + 1]), the b with cu[b] <= q <
// cu[b+1] and pos[b] + q - cu[b].  Its visible rows are min(n_rows[bseq], (p+1)/ratio).  sel [Q, topk], n_sel [Q].
cudaError_t launch_index_topk(const Dims& L, const void* iq, const void* iw, int Q, const void* ikeys, int cap,
                              const int32_t* n_rows, const int32_t* pos, int pos0, const float* inv_freq,
                              int32_t* sel, int32_t* n_sel, const IndexWs& ws, int32_t* err, cudaStream_t s,
                              const int32_t* cu = nullptr);

// ---- tc_project.cu (tensor-core compressor projections; bf16)
bool tc_project_supported(const Dims& L, int d);
void carve_tc_project(Carver& c, const Dims& L, int d, int ntok, float** part, int** tickets);
// K splits the projection of ntok tokens uses (1: proj is written directly).
int tc_project_splits(const Dims& L, int d, int ntok);
// Padded token count (rows of each split's partial block).
int tc_project_cols(const Dims& L, int d, int ntok);
// fixup = false (splits > 1): the fp32 partials [splits, ntok (padded), 2*L*d] are left for the consumer.
cudaError_t launch_tc_project(const Dims& L, int d, const void* x, int ntok, const void* wkv, const void* wgate,
                              void* proj, float* part, int* tickets, bool fixup, int32_t* err, cudaStream_t s);
// The index pool's and the attention pool's single-token projections as one grid (partials only; the pooling
// kernel sums them).  plan_project_pair picks the split counts (false: use two launches).
bool plan_project_pair(const Dims& L, int d0, int d1, int ntok, int* s0, int* s1);
cudaError_t launch_tc_project_pair(const Dims& L, int d0, const void* wkv0, const void* wg0, float* part0, int d1,
                                   const void* wkv1, const void* wg1, float* part1, const void* x, int ntok, int s0,
                                   int s1, int32_t* err, cudaStream_t s);

// ---- tc_indexer.cu (tensor-core scores; bf16, Hi = 64, Di = 128)
bool tc_index_supported(const Dims& L);
size_t tc_index_ws(const Dims& L, int Q);
// scores[q][j] for every q whose visible rows exceed topk; keys of query q are
// ikeys[pos ? q : 0]; ws needs tc_index_ws() bytes.
// overlap (decode only): score only rows < floor(pos/ratio) without reading n_rows, and leave the roped
// queries (bf16 [Q,64,128]) and scaled head weights (fp32 [Q,64]) at the start of ws for the selection stage.
cudaError_t launch_tc_index_scores(const Dims& L, const void* iq, const void* iw, int Q, const void* ikeys, int Bk,
                                   int cap, const int32_t* n_rows, const int32_t* pos, int pos0,
                                   const float* inv_freq, void* ws, float* scores, int32_t* err, cudaStream_t s,
                                   bool overlap = false, const int32_t* cu = nullptr, bool fp8 = false);

// ---- tc_attend.cu (tensor-core attention; bf16, H = 64, D = 512, R = 64)
bool tc_attend_supported(const Dims& L);
// Q queries (decode: pos[q], ring[q], pool[q]; prefill: pos == null, positions pos0 + q, batch 1, chunk rows
// kvr), S key splits per query: S > 1 writes (m, l, acc) partials, S == 1 the final output.
// Decode passes kv_new: the CTA that owns the new token's row ropes it and writes its ring slot.
cudaError_t launch_tc_attend(const Dims& L, const void* q, const void* pool, void* ring, const void* kvr,
                             const void* kv_new, const int32_t* sel, const int32_t* n_sel, const int32_t* n_rows,
                             const int32_t* pos, int pos0, int cap, const float* sink, const float* inv_freq, int Q,
                             int S, float* part_ml, float* part_acc, void* out, int32_t* err, cudaStream_t s);
// Merge of decode split partials for H % 8 == 0, D == 512 (one warp per head, 16 dims per lane).
// qps: consecutive queries per sequence (query q at pos[q / qps] + q % qps).
cudaError_t launch_tc_merge(const Dims& L, const float* part_ml, const float* part_acc, int S, int Q,
                            const float* sink, const int32_t* pos, const float* inv_freq, void* out, cudaStream_t s,
                            int qps = 1);

// ---- attend.cu: pos[b] += by for b < B
cudaError_t launch_advance_positions(int32_t* pos, int B, int by, cudaStream_t s);
// n rows of 128 bf16 values (src) -> n fp8 index rows of kFp8RowBytes (dst)
cudaError_t launch_index_rows_fp8(const void* src, long long n, void* dst, cudaStream_t s);
// ---- attend.cu: csa_trim (rewind B sequences by n_back tokens within the rollback margin)
cudaError_t launch_trim(const Dims& L, int B, const int32_t* n_back, int32_t* pos, int32_t* n_rows_a,
                        int32_t* n_rows_i, int32_t* hw, int32_t* err, cudaStream_t s);

// ---- tc_attend_prefill.cu (tensor-core chunked-prefill attention; bf16, H = 64, D = 512, R = 64)
// T queries of one sequence at positions pos0 + q; the chunk's roped rows kvr [T, D], the ring before the
// chunk, pool [cap, D]; persistent CTAs (one per SM) finalise the output.  Requires tc_attend_supported(L).
// With device positions (verify blocks): query q of sequence q / qps at pos[q / qps] + q % qps over pool
// [B, cap, D] and ring [B, Wr, D], every window token (the block's included) read from the ring; kvr unused.
// With a row table cu (a packed variable-length batch of qps chunks, T = N rows): query q of sequence b at
// pos[b] + q - cu[b]; tokens before pos[b] from the ring, the chunk's own from kvr [N, D] (roped).
cudaError_t launch_tc_attend_prefill(const Dims& L, const void* q, const void* pool, const void* ring,
                                     const void* kvr, const int32_t* sel, const int32_t* n_sel,
                                     const int32_t* n_rows, int pos0, int cap, const float* sink,
                                     const float* inv_freq, int T, void* out, int32_t* err, cudaStream_t s,
                                     const int32_t* pos = nullptr, int qps = 1, const int32_t* cu = nullptr);

// ---- tc_attend_decode.cu (tensor-core decode attention; bf16, H = 64, D = 512, R = 64)
bool tc_attend_decode_supported(const Dims& L);
// Key splits per query for Q queries over a window of W rows and at most n_max selected rows: each split's window
// share plus selection share fits one 160-row tile, more splits while every CTA still fits one wave; 0 when
// max_splits cannot hold enough splits.
int tc_attend_decode_splits(int Q, int W, int n_max, int max_splits);
// One CTA per (query, split).  S > 1 writes (m, l, acc) partials (merge follows), S == 1 the final output.
// Decode (qps 1): the new token kv_new[b] is roped in-kernel and written to ring slot pos[b] % Wr.  Verify blocks
// (qps tokens per sequence, kv_in_ring): query q belongs to sequence q / qps at pos[q / qps] + q % qps and every
// block token is already in the ring.
cudaError_t launch_tc_attend_decode(const Dims& L, const void* q, const void* pool, void* ring, const void* kv_new,
                                    const int32_t* sel, const int32_t* n_sel, const int32_t* n_rows,
                                    const int32_t* pos, int cap, const float* sink, const float* inv_freq, int Q,
                                    int S, float* part_ml, float* part_acc, void* out, int32_t* err, cudaStream_t s,
                                    int qps = 1, bool kv_in_ring = false, bool cluster = false);
// Whether S splits can merge inside a cluster (S in {2, 4} and the device places such clusters): the decode
// kernel then writes the output itself and no merge kernel runs.
bool tc_attend_decode_cluster(int S);

// ---- attend.cu
struct AttendWs {
  void* qr;        // [Q, H, D] roped queries, model dtype
  void* kvr;       // [T, D] roped chunk kv (prefill only)
  float* part_ml;  // [Q, S, H, 2] split partial (max, sum)
  float* part_acc; // [Q, S, H, D] split partial accumulators
  int S;           // splits per query
};
int attend_splits(const Dims& L, bool prefill, bool all_rows, int cap);
AttendWs carve_attend(Carver& c, const Dims& L, int Q, int S, int T);
// Decode: Q = B sequences, positions pos[b], window rings window[b].
cudaError_t launch_attend_decode(const Dims& L, const void* q, const void* kv_new, const float* sink, int B,
                                 void* window, const void* pool, int cap, const int32_t* n_rows, const int32_t* sel,
                                 const int32_t* n_sel, const int32_t* pos, const float* inv_freq, void* out,
                                 const AttendWs& ws, int32_t* err, cudaStream_t s);
// Prefill: T queries of one sequence at pos0 + t.  sel/n_sel from the indexer (or null: all visible rows).
cudaError_t launch_attend_prefill(const Dims& L, const void* q, const void* kv_new, const float* sink, int T,
                                  int pos0, void* window, const void* pool, int cap, const int32_t* n_rows,
                                  const int32_t* sel, const int32_t* n_sel, const float* inv_freq, void* out,
                                  const AttendWs& ws, int32_t* err, cudaStream_t s);

// A packed variable-length batch of B prefill chunks (row table cu [B + 1], N rows, the longest T_max): the rows
// are roped at their positions into ws.kvr, every query attends, then each sequence's last min(T_b, Wr) rows
// enter its ring.  Tensor-core shapes only.
cudaError_t launch_attend_prefill_varlen(const Dims& L, const void* q, const void* kv_new, const float* sink, int B,
                                         const int32_t* cu, int N, int T_max, void* window, const void* pool, int cap,
                                         const int32_t* n_rows, const int32_t* sel, const int32_t* n_sel,
                                         const int32_t* pos, const float* inv_freq, void* out, const AttendWs& ws,
                                         int32_t* err, cudaStream_t s);

// Verify blocks: T tokens per sequence appended to the window ring (roped), then each attended by its own query.
cudaError_t launch_attend_verify(const Dims& L, const void* q, const void* kv_new, const float* sink, int B, int T,
                                 void* window, const void* pool, int cap, const int32_t* n_rows, const int32_t* sel,
                                 const int32_t* n_sel, const int32_t* pos, const float* inv_freq, void* out,
                                 const AttendWs& ws, int32_t* err, cudaStream_t s);

// ---- tree.cu (a tree of drafted tokens; parent [B, T], T <= 64)
cudaError_t launch_norm_rope(const Dims& L, const csa_rows* rows, int n, int B, int T, const int32_t* parent,
                             const int32_t* pos, const float* inv_freq, int32_t* err, cudaStream_t s);
// One pool of a compress call: the committed frontier, and the draft buffers proj [B, T, 2*L*d] and rows [B, T, d].
// ws: [B*T, 2*L*d] of the model dtype for the SIMT projection, which projects unused slots too (null where the
// tensor-core projection applies).
struct TreeCompress {
  const csa_compressor* comp;
  const void* frontier;
  void* proj;
  void* rows;
  void* ws;
};
void* carve_compress_tree(Carver& c, const Dims& L, int d, int B, int T);
// ---- tc_tree_project.cu: the projections of all pools into the draft buffers (bf16; whole 128-feature tiles)
bool tc_tree_project_supported(const Dims& L, int d);
cudaError_t launch_tc_tree_project(const Dims& L, const TreeCompress* pools, int npool, const void* x, int B, int T,
                                   const int32_t* parent, const int32_t* pos, int32_t* err, cudaStream_t s);
cudaError_t launch_compress_tree(const Dims& L, const TreeCompress* pools, int npool, const void* x, int B, int T,
                                 const int32_t* parent, const int32_t* pos, const float* inv_freq, int32_t* err,
                                 cudaStream_t s);
cudaError_t launch_index_scores_tree(const Dims& L, const void* iq, const void* iw, int B, int T,
                                     const int32_t* parent, const void* ikeys, int cap, const void* rows,
                                     const int32_t* n_rows, const int32_t* pos, float* scores, void* ws, int32_t* err,
                                     cudaStream_t s);
// ---- tc_tree_scores.cu (the same on the tensor cores; bf16, Hi = 64, Di = 128, keys in bf16 or fp8 rows)
bool tc_tree_scores_supported(const Dims& L, int B, int cap);
size_t tree_scores_ws(const Dims& L, int B, int T);
cudaError_t launch_tc_tree_scores(const Dims& L, const void* iq, const void* iw, int B, int T, const int32_t* parent,
                                  const void* ikeys, int cap, const void* rows, const int32_t* n_rows,
                                  const int32_t* pos, float* scores, void* ws, int32_t* err, cudaStream_t s);
// What the attention kernels read of a node: its path and the path's completing nodes as masks, its position, the
// committed length and rows of its sequence, and its keys' count from the pool and the draft rows (nsel < 0: an
// unused slot, or a node that an error skips).
struct TreeNode {
  unsigned long long mask, closers;
  int32_t p, p0, n, nsel;
};
// ---- indexer.cu: the selection of every node (sel [B*T, topk], columns of scores [B*T, cap + T]; nodes [B*T])
cudaError_t launch_topk_tree(const Dims& L, const float* scores, int B, int T, const int32_t* parent, int cap,
                             const int32_t* n_rows, const int32_t* pos, int32_t* sel, TreeNode* nodes, int32_t* err,
                             cudaStream_t s);
// ---- tree_topk.cu: the same by a block of 256 threads per node with its keys in shared memory, where
// topk_tree_small_blocks says so (more nodes than SMs and up to 64 KB of keys, or few nodes and up to 33 KB)
bool topk_tree_small_blocks(int Q, int cap, int T, int sms);
cudaError_t launch_topk_tree_small(const Dims& L, const float* scores, int B, int T, const int32_t* parent, int cap,
                                  const int32_t* n_rows, const int32_t* pos, int32_t* sel, TreeNode* nodes,
                                  int32_t* err, cudaStream_t s);
struct TreeAttendWs {
  int32_t* sel;    // [B*T, topk] when the caller wants no selection (null without an indexer)
  TreeNode* nodes; // [B*T]
};
TreeAttendWs carve_attend_tree(Carver& c, const Dims& L, int B, int T, int cap);
struct TreeAttend {
  const void *q, *kv, *window, *pool, *rows;
  const float *scores, *sink, *inv_freq;
  const int32_t *parent, *n_rows, *pos;
  void* out;
  int32_t* sel_out;
  int B, T, cap;
  TreeAttendWs ws;
};
cudaError_t launch_attend_tree(const Dims& L, const TreeAttend& t, int32_t* err, cudaStream_t s);
// The same on the tensor cores (tc_attend_supported shapes), the node records already in t.ws: a CTA per query
// streaming its tiles (tc_tree_attend.cu), or S = 1, 2, 4 or 8 splits per query merged in a cluster (tc_attend_decode.cu).
cudaError_t launch_tc_attend_tree(const Dims& L, const TreeAttend& t, const int32_t* sel, int32_t* err,
                                  cudaStream_t s);
// queries that launch_tc_attend_tree_split works on at once with S splits each
int tc_attend_tree_split_max(int S);
cudaError_t launch_tc_attend_tree_split(const Dims& L, const TreeAttend& t, const int32_t* sel, int S, int32_t* err,
                                        cudaStream_t s);
// Pool 0: the attention pool; pool 1 (npool == 2): the index pool.
struct TreeCommit {
  const int32_t *parent, *leaf, *pos;
  int32_t* pos_out;
  const void* kv;
  void* window;
  const void *proj[2], *rows[2];
  void *frontier[2], *pool[2];
  const int32_t* n_rows[2];
  int32_t* n_rows_out[2];
  int cap[2], npool, B, T;
};
cudaError_t launch_commit_tree(const Dims& L, const TreeCommit& c, int32_t* err, cudaStream_t s);

// ---- add_norm.cu: h = x + residual, its RMS norm, and the norm in 8 bits
struct AddNorm {
  const void *x, *residual;   // [N, X], rows x_stride, r_stride elements apart; residual may be null
  const float* weight;        // [X] or null
  void *out, *residual_out;   // [N, X] or null
  uint8_t* codes;             // [N, X] or null
  float* scales;              // [N, X / group]
  long long N, x_stride, r_stride;
  int X, group;
};
cudaError_t launch_add_norm(const Dims& L, const AddNorm& t, cudaStream_t s);

// ---- a cache in pages and 8 bits
struct PagedAppend {
  const void* rows;            // [B, T, D], strides in elements
  long long stride_b, stride_t;
  uint8_t* codes;              // [n_pages, P, D]
  float* scales;               // [n_pages, P]
  const int32_t *table, *pos, *n_new;
  const float *weight, *inv_freq;
  int32_t* err;
  float eps;
  int n_pages, P, pages, B, T, D, R, norm;
};
// ---- paged_append.cu
cudaError_t launch_append_pages(const Dims& L, const PagedAppend& t, cudaStream_t s);

// n / d for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (floor(m n / 2^32) + n) / 2^l (T. Granlund and P. L. Montgomery, Division by Invariant Integers).
struct FastDiv {
  uint32_t m;
  int l;
};
inline FastDiv fast_div(uint32_t d) {
  int l = 0;
  while ((1ull << l) < d) ++l;
  return FastDiv{(uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}
struct PagedArgs {
  const uint8_t* codes;        // [n_pages, P, D]
  const float* scales;         // [n_pages, P]
  const void* q;               // [B, T, H, D], rotated
  void* out;                   // [B, T, H, D]
  const float *sink, *inv_freq;  // either may be null
  const int32_t *pos, *n_new, *token_table, *row_table, *n_rows, *sel, *n_sel;
  FastDiv by_page, by_T, by_ratio;  // division by P, T, ratio
  int n_pages, P, token_pages, row_pages;  // the pool's pages, rows a page, and the tables' widths
  int B, T, H, D, R, W, first, ratio, topk;
  float scale2;                // softmax scale * log2(e)
  // workspace
  int2* parts;                 // [B T] block of a query's first part, and their count
  float* part;                 // [2 blocks][D / cols][H][cols] parts of split queries, relative to their maximum
  float2* ml;                  // [2 blocks][H] their maxima (in powers of two) and sums
  float2* turns;               // [blocks][R / 2] cos, sin of the output's rotation, by the block of the first part
  int cols;                    // dims that a part holds side by side
  int tile, shift, min_tiles;  // keys a tile; log2 of the rows that lie in one page; the shortest piece of a query, in tiles
  int merge;                   // whether a merge follows (0: min_tiles is so large that no query is split)
  int32_t* err;
};
// Blocks (one an SM) that a call is spread over at most.
constexpr int kPagedBlocks = 152;
// ---- paged_attend.cu: the portable kernel, and the merge of split queries
void carve_paged(Carver& c, const Dims& L, int Q, PagedArgs* a);
cudaError_t launch_attend_pages(const Dims& L, PagedArgs a, cudaStream_t s);
// ---- tc_paged_attend.cu (tensor cores; bf16, H = 64, D = 512, R = 64, pages of whole 8-row groups)
bool tc_paged_supported(const Dims& L, int P);
cudaError_t launch_tc_paged(const PagedArgs& a, cudaStream_t s);

}  // namespace csa
