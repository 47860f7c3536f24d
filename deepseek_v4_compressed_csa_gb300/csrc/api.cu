// C-ABI entry points: argument validation (fail closed, before any launch),
// workspace carving, dispatch to the kernel translation units.
#include <math.h>

#include "kernels.h"

#include <atomic>
#include <initializer_list>

using namespace csa;

static std::atomic<unsigned long long> g_launches{0};
void csa::count_launches(int n) { g_launches.fetch_add((unsigned long long)n, std::memory_order_relaxed); }

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dev_tensor(const void* p) { return p != nullptr && aligned16(p); }
bool dev_i32(const void* p) { return p != nullptr && aligned4(p); }

csa_status make_dims(const csa_layer* l, Dims* d) {
  if (!l) return CSA_ERR_ARG;
  if (l->dtype != CSA_F32 && l->dtype != CSA_BF16) return CSA_ERR_ARG;
  if (l->H < 1 || l->D < 8 || l->D % 8 || l->D > 1024) return CSA_ERR_ARG;
  if (l->R < 2 || l->R > l->D || l->R % 8 || (l->D - l->R) % 8) return CSA_ERR_ARG;
  if (l->W < 1 || l->ratio < 1 || l->X < 8 || l->X % 8) return CSA_ERR_ARG;
  if (l->ratio == 4) {
    if (l->Hi < 1 || l->Di < 8 || l->Di % 8 || l->R > l->Di || (l->Di - l->R) % 2) return CSA_ERR_ARG;
    if (l->topk < 1 || l->topk > 4096) return CSA_ERR_ARG;
  }
  if (!(l->rms_eps >= 0.f) || !(l->scale >= 0.f)) return CSA_ERR_ARG;
  if (l->rollback < 0 || l->rollback > (1 << 20)) return CSA_ERR_ARG;
  if (l->index_fp8 != 0 && l->index_fp8 != 1) return CSA_ERR_ARG;
  // (the index pool is told apart from the attention pool by its row length)
  if (l->index_fp8 && (l->ratio != 4 || l->dtype != CSA_BF16 || l->Hi != 64 || l->Di != 128 || l->D == l->Di ||
                       l->R > 64 || l->R % 8))
    return CSA_ERR_UNSUPPORTED;
  d->dtype = l->dtype;
  d->H = l->H; d->D = l->D; d->R = l->R; d->W = l->W; d->ratio = l->ratio;
  d->Hi = l->Hi; d->Di = l->Di; d->topk = l->topk; d->X = l->X;
  d->scale = l->scale > 0.f ? l->scale : (float)(1.0 / sqrt((double)l->D));
  d->eps = l->rms_eps;
  d->lanes = (l->ratio == 4) ? 2 : 1;
  d->rollback = l->rollback;
  d->Wr = l->W + l->rollback;
  d->F = csa_frontier_slots(l->ratio) + l->rollback;
  d->ikey_fp8 = l->index_fp8;
  return CSA_OK;
}

csa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

size_t ws_compress(const Dims& L, int d, int B, int T) {
  Carver c(nullptr);
  carve_compress(c, L, d, B, T);
  return c.off;
}
size_t ws_compress_pair(const Dims& L, int B, int T) {
  Carver c(nullptr);
  carve_compress(c, L, L.D, B, T);
  carve_compress(c, L, L.Di, B, T);
  return c.off;
}
size_t ws_index(const Dims& L, int B, int cap) {
  Carver c(nullptr);
  carve_index(c, L, B, cap);
  return c.off;
}
size_t ws_decode(const Dims& L, int B, int cap) {
  Carver c(nullptr);
  carve_attend(c, L, B, attend_splits(L, false, !L.has_indexer(), cap), 0);
  return c.off;
}
void carve_prefill(Carver& c, const Dims& L, int T, int cap, IndexWs* iw, int32_t** sel, int32_t** n_sel,
                   AttendWs* aw) {
  if (L.has_indexer()) {
    *iw = carve_index(c, L, T, cap);
    *sel = c.take<int32_t>((size_t)T * L.topk);
    *n_sel = c.take<int32_t>(T);
  }
  *aw = carve_attend(c, L, T, attend_splits(L, true, false, cap), T);
}
size_t ws_compress_varlen(const Dims& L, int B, int N) {
  size_t best = 0;
  for (int d : {L.D, L.Di}) {
    if (d == L.Di && !L.has_indexer()) continue;
    Carver c(nullptr);
    carve_compress_varlen(c, L, d, B, N);
    best = c.off > best ? c.off : best;
  }
  return best;
}
size_t ws_prefill(const Dims& L, int T, int cap) {
  Carver c(nullptr);
  IndexWs iw{};
  int32_t *s = nullptr, *n = nullptr;
  AttendWs aw{};
  carve_prefill(c, L, T, cap, &iw, &s, &n, &aw);
  return c.off;
}

// A batch of trees: at most 64 nodes each (a path is a 64-bit mask), and grids of B x T queries.
constexpr int kTreeCapMax = INT32_MAX - 256;  // columns, cap + T of them, are ints
bool tree_sizes_ok(int B, int T) {
  return B >= 1 && B <= 65535 && T >= 1 && T <= 64 && (long long)B * T <= (1 << 18);
}
size_t ws_compress_tree(const Dims& L, bool both, int B, int T) {
  Carver c(nullptr);
  carve_compress_tree(c, L, L.D, B, T);
  if (both) carve_compress_tree(c, L, L.Di, B, T);
  return c.off;
}
size_t ws_attend_tree(const Dims& L, int B, int T, int cap) {
  Carver c(nullptr);
  carve_attend_tree(c, L, B, T, cap);
  return c.off;
}

size_t ws_attend_pages(const Dims& L, int Q) {
  Carver c(nullptr);
  PagedArgs a{};
  carve_paged(c, L, Q, &a);
  return c.off;
}
// B x T queries or new tokens around a cache in pages
constexpr int kPagedQueries = 1 << 16;
constexpr long long kPagedRows = INT32_MAX - 256;  // rows of the pool (their numbers are ints)
constexpr long long kPagedTable = 1 << 30;         // rows that a sequence's table has room for
bool pages_ok(const csa_pages* p) {
  return p && dev_tensor(p->codes) && dev_i32(p->scales) && p->n_pages >= 1 && p->page_rows >= 1 &&
         (long long)p->n_pages * p->page_rows <= kPagedRows;
}
bool table_ok(const csa_pages* p, const int32_t* table, int pages) {
  return dev_i32(table) && pages >= 1 && (long long)pages * p->page_rows <= kPagedTable;
}
constexpr long long kSpan = 1LL << 56;  // values that rows a stride apart may span: no sum of theirs passes 64 bits
// [lo, hi) of a tensor of n rows of `row` bytes, `stride` bytes apart
struct Span {
  uintptr_t lo, hi;
  Span(const void* p, long long n, long long row, long long stride)
      : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + (uintptr_t)((n - 1) * stride + row)) {}
  Span(const void* p, long long bytes) : Span(p, 1, bytes, 0) {}
  bool meets(const Span& o) const { return lo && o.lo && lo < o.hi && o.lo < hi; }  // (a tensor that is not there meets none)
};
// Whether what a call writes lies apart from all that it reads, and from what else it writes.
template <int kOuts, int kIns>
bool apart(const Span (&outs)[kOuts], const Span (&ins)[kIns]) {
  for (int i = 0; i < kOuts; ++i) {
    for (const Span& in : ins)
      if (outs[i].meets(in)) return false;
    for (int k = 0; k < i; ++k)
      if (outs[i].meets(outs[k])) return false;
  }
  return true;
}

}  // namespace

extern "C" {

unsigned long long csa_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

int csa_frontier_slots(int ratio) { return ratio == 4 ? 2 * ratio : ratio; }

const char* csa_status_string(csa_status s) {
  switch (s) {
    case CSA_OK: return "CSA_OK";
    case CSA_ERR_ARG: return "CSA_ERR_ARG: invalid argument";
    case CSA_ERR_UNSUPPORTED: return "CSA_ERR_UNSUPPORTED: no kernel for these arguments";
    case CSA_ERR_CUDA: return "CSA_ERR_CUDA: kernel launch failed";
    case CSA_ERR_WORKSPACE: return "CSA_ERR_WORKSPACE: workspace too small";
  }
  return "unknown csa_status";
}

csa_status csa_workspace_size(const csa_layer* layer, int op, int B, int T, int cap, size_t* bytes) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!bytes || B < 1 || cap < 1) return CSA_ERR_ARG;
  switch (op) {
    case CSA_OP_COMPRESS:
      if (T < 1) return CSA_ERR_ARG;
      *bytes = ws_compress(L, L.D, B, T);
      if (L.has_indexer()) {
        const size_t bi = ws_compress(L, L.Di, B, T);
        if (bi > *bytes) *bytes = bi;
      }
      return CSA_OK;
    case CSA_OP_COMPRESS_PAIR:
      if (T < 1 || !L.has_indexer()) return CSA_ERR_ARG;
      *bytes = ws_compress_pair(L, B, T);
      return CSA_OK;
    case CSA_OP_INDEX_TOPK:
      *bytes = ws_index(L, B, cap);
      return CSA_OK;
    case CSA_OP_ATTEND_DECODE:
      *bytes = ws_decode(L, B, cap);
      return CSA_OK;
    case CSA_OP_ATTEND_PREFILL:
      if (T < 1 || T > 16384) return CSA_ERR_ARG;
      *bytes = ws_prefill(L, T, cap);
      return CSA_OK;
    case CSA_OP_COMPRESS_VARLEN:  // T: the batch's total tokens N
      if (T < 1 || T > (1 << 20)) return CSA_ERR_ARG;
      *bytes = ws_compress_varlen(L, B, T);
      return CSA_OK;
    case CSA_OP_ATTEND_PREFILL_VARLEN:  // T: the batch's total tokens N
      if (T < 1 || T > 16384) return CSA_ERR_ARG;
      *bytes = ws_prefill(L, T, cap);
      return CSA_OK;
    case CSA_OP_COMPRESS_TREE:
      if (!tree_sizes_ok(B, T)) return CSA_ERR_ARG;
      *bytes = ws_compress_tree(L, L.has_indexer(), B, T);
      return CSA_OK;
    case CSA_OP_ATTEND_TREE:
      if (!tree_sizes_ok(B, T)) return CSA_ERR_ARG;
      *bytes = ws_attend_tree(L, B, T, cap);
      return CSA_OK;
    case CSA_OP_INDEX_SCORES_TREE:
      if (!tree_sizes_ok(B, T)) return CSA_ERR_ARG;
      *bytes = tree_scores_ws(L, B, T);
      return CSA_OK;
    case CSA_OP_ATTEND_PAGES:
      if (T < 1 || (long long)B * T > kPagedQueries) return CSA_ERR_ARG;
      *bytes = ws_attend_pages(L, B * T);
      return CSA_OK;
  }
  return CSA_ERR_ARG;
}

// Argument checks shared by the one-pool and two-pool compress calls.
static bool compress_args_ok(const Dims& L, const csa_compressor* comp, int B, int T, int cap, const void* frontier,
                             const void* pool, const int32_t* n_rows) {
  if (!comp || B < 1 || T < 1 || cap < 1) return false;
  if (comp->d < L.R || comp->d % 8 || (comp->d != L.D && comp->d != L.Di)) return false;
  if (!dev_tensor(comp->wkv) || !dev_tensor(comp->wgate) || !dev_tensor(comp->ape) || !dev_tensor(comp->norm_w))
    return false;
  return dev_tensor(frontier) && dev_tensor(pool) && dev_i32(n_rows);
}

csa_status csa_compress_append(const csa_layer* layer, const csa_compressor* comp, const void* x, int B, int T,
                               const int32_t* pos, void* frontier, void* pool, int cap, int32_t* n_rows,
                               const float* inv_freq, void* ws, size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!compress_args_ok(L, comp, B, T, cap, frontier, pool, n_rows)) return CSA_ERR_ARG;
  if (!dev_tensor(x) || !dev_tensor(inv_freq) || !dev_i32(pos) || !dev_i32(err)) return CSA_ERR_ARG;
  const size_t need = ws_compress(L, comp->d, B, T);
  if (ws_bytes < need || (need && !dev_tensor(ws))) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  CompressWs w = carve_compress(c, L, comp->d, B, T);
  return cuda_status(launch_compress(L, *comp, x, B, T, pos, frontier, pool, cap, n_rows, inv_freq, w, err,
                                     static_cast<cudaStream_t>(stream)));
}

csa_status csa_compress_append_pair(const csa_layer* layer, const csa_compressor* comp_a,
                                    const csa_compressor* comp_i, const void* x, int B, int T, const int32_t* pos,
                                    void* frontier_a, void* pool_a, int cap_a, int32_t* n_rows_a, void* frontier_i,
                                    void* pool_i, int cap_i, int32_t* n_rows_i, const float* inv_freq, void* ws,
                                    size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!L.has_indexer()) return CSA_ERR_UNSUPPORTED;
  if (!compress_args_ok(L, comp_a, B, T, cap_a, frontier_a, pool_a, n_rows_a) ||
      !compress_args_ok(L, comp_i, B, T, cap_i, frontier_i, pool_i, n_rows_i))
    return CSA_ERR_ARG;
  if (comp_a->d != L.D || comp_i->d != L.Di) return CSA_ERR_ARG;
  if (!dev_tensor(x) || !dev_tensor(inv_freq) || !dev_i32(pos) || !dev_i32(err)) return CSA_ERR_ARG;
  const size_t need = ws_compress_pair(L, B, T);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  const CompressWs wa = carve_compress(c, L, L.D, B, T);
  const CompressWs wi = carve_compress(c, L, L.Di, B, T);
  return cuda_status(launch_compress_pair(L, *comp_a, *comp_i, x, B, T, pos, frontier_a, pool_a, cap_a, n_rows_a,
                                          frontier_i, pool_i, cap_i, n_rows_i, inv_freq, wa, wi, err,
                                          static_cast<cudaStream_t>(stream)));
}

csa_status csa_index_topk(const csa_layer* layer, const void* iq, const void* iw, int B, const void* ikeys, int cap,
                          const int32_t* n_rows, const int32_t* pos, const float* inv_freq, int32_t* sel,
                          int32_t* n_sel, void* ws, size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!L.has_indexer()) return CSA_ERR_UNSUPPORTED;
  if (B < 1 || cap < 1) return CSA_ERR_ARG;
  if (!dev_tensor(iq) || !dev_i32(iw) || !dev_tensor(ikeys) || !dev_tensor(inv_freq)) return CSA_ERR_ARG;
  if (!dev_i32(n_rows) || !dev_i32(pos) || !dev_i32(sel) || !dev_i32(n_sel) || !dev_i32(err)) return CSA_ERR_ARG;
  const size_t need = ws_index(L, B, cap);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  IndexWs w = carve_index(c, L, B, cap);
  return cuda_status(launch_index_topk(L, iq, iw, B, ikeys, cap, n_rows, pos, 0, inv_freq, sel, n_sel, w, err,
                                       static_cast<cudaStream_t>(stream)));
}

csa_status csa_index_topk_overlapped(const csa_layer* layer, const void* iq, const void* iw, int B, const void* ikeys,
                                     int cap, const int32_t* n_rows, const int32_t* pos, const float* inv_freq,
                                     int32_t* sel, int32_t* n_sel, void* ws, size_t ws_bytes, int32_t* err,
                                     void* stream, void* pool_ready) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!L.has_indexer() || L.ikey_fp8) return CSA_ERR_UNSUPPORTED;
  if (B < 1 || cap < 1) return CSA_ERR_ARG;
  if (!dev_tensor(iq) || !dev_i32(iw) || !dev_tensor(ikeys) || !dev_tensor(inv_freq)) return CSA_ERR_ARG;
  if (!dev_i32(n_rows) || !dev_i32(pos) || !dev_i32(sel) || !dev_i32(n_sel) || !dev_i32(err)) return CSA_ERR_ARG;
  const size_t need = ws_index(L, B, cap);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  IndexWs w = carve_index(c, L, B, cap);
  return cuda_status(launch_index_topk_overlapped(L, iq, iw, B, ikeys, cap, n_rows, pos, inv_freq, sel, n_sel, w,
                                                  err, static_cast<cudaStream_t>(stream),
                                                  static_cast<cudaEvent_t>(pool_ready)));
}

csa_status csa_attend_decode(const csa_layer* layer, const void* q, const void* kv_new, const float* sink, int B,
                             void* window, const void* pool, int cap, const int32_t* n_rows, const int32_t* sel,
                             const int32_t* n_sel, const int32_t* pos, const float* inv_freq, void* out, void* ws,
                             size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (B < 1 || cap < 1) return CSA_ERR_ARG;
  if (!dev_tensor(q) || !dev_tensor(kv_new) || !dev_i32(sink) || !dev_tensor(window) || !dev_tensor(pool) ||
      !dev_tensor(inv_freq) || !dev_tensor(out))
    return CSA_ERR_ARG;
  if (!dev_i32(n_rows) || !dev_i32(pos) || !dev_i32(err)) return CSA_ERR_ARG;
  if (sel && (!dev_i32(sel) || !dev_i32(n_sel))) return CSA_ERR_ARG;
  if (sel && !L.has_indexer()) return CSA_ERR_ARG;
  const size_t need = ws_decode(L, B, cap);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  AttendWs w = carve_attend(c, L, B, attend_splits(L, false, !L.has_indexer(), cap), 0);
  return cuda_status(launch_attend_decode(L, q, kv_new, sink, B, window, pool, cap, n_rows, sel, n_sel, pos,
                                          inv_freq, out, w, err, static_cast<cudaStream_t>(stream)));
}

csa_status csa_attend_prefill_chunk(const csa_layer* layer, const void* q, const void* kv_new, const void* iq,
                                    const void* iw, const float* sink, int T, int32_t pos0, void* window,
                                    const void* pool, const void* ikeys, int cap, const int32_t* n_rows,
                                    const float* inv_freq, void* out, int32_t* sel_out, void* ws, size_t ws_bytes,
                                    int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (T < 1 || T > 16384 || pos0 < 0 || cap < 1) return CSA_ERR_ARG;
  if (!dev_tensor(q) || !dev_tensor(kv_new) || !dev_i32(sink) || !dev_tensor(window) || !dev_tensor(pool) ||
      !dev_tensor(inv_freq) || !dev_tensor(out))
    return CSA_ERR_ARG;
  if (!dev_i32(n_rows) || !dev_i32(err)) return CSA_ERR_ARG;
  if (L.has_indexer() && (!dev_tensor(iq) || !dev_i32(iw) || !dev_tensor(ikeys))) return CSA_ERR_ARG;
  if (sel_out && !dev_i32(sel_out)) return CSA_ERR_ARG;
  const size_t need = ws_prefill(L, T, cap);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  IndexWs iws{};
  int32_t *sel = nullptr, *n_sel = nullptr;
  AttendWs aw{};
  carve_prefill(c, L, T, cap, &iws, &sel, &n_sel, &aw);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (L.has_indexer()) {
    if (sel_out) sel = sel_out;
    cudaError_t e = launch_index_topk(L, iq, iw, T, ikeys, cap, n_rows, nullptr, pos0, inv_freq, sel, n_sel, iws,
                                      err, s);
    if (e != cudaSuccess) return CSA_ERR_CUDA;
  } else if (sel_out && L.topk > 0) {
    cudaMemsetAsync(sel_out, 0xff, (size_t)T * L.topk * sizeof(int32_t), s);
  }
  return cuda_status(launch_attend_prefill(L, q, kv_new, sink, T, pos0, window, pool, cap, n_rows,
                                           L.has_indexer() ? sel : nullptr, n_sel, inv_freq, out, aw, err, s));
}

// Host-side checks of a packed variable-length batch's sizes (the row table itself is on the device).
static bool varlen_args_ok(int B, const int32_t* cu_seqlens, int N, int T_max) {
  // (B + 1 <= 4096 N: the index scan's group table fits the query area of its workspace)
  return B >= 1 && B <= (1 << 16) && N >= 1 && T_max >= 1 && T_max <= N && (long long)B + 1 <= 4096LL * N &&
         dev_i32(cu_seqlens);
}

csa_status csa_compress_append_varlen(const csa_layer* layer, const csa_compressor* comp, const void* x, int B,
                                      const int32_t* cu_seqlens, int N, int T_max, const int32_t* pos,
                                      void* frontier, void* pool, int cap, int32_t* n_rows, const float* inv_freq,
                                      void* ws, size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!varlen_args_ok(B, cu_seqlens, N, T_max) || N > (1 << 20)) return CSA_ERR_ARG;
  if (!compress_args_ok(L, comp, B, 1, cap, frontier, pool, n_rows)) return CSA_ERR_ARG;
  if (!dev_tensor(x) || !dev_i32(pos) || !dev_tensor(inv_freq) || !dev_i32(err)) return CSA_ERR_ARG;
  Carver c0(nullptr);
  carve_compress_varlen(c0, L, comp->d, B, N);
  if (ws_bytes < c0.off || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  const CompressWs w = carve_compress_varlen(c, L, comp->d, B, N);
  return cuda_status(launch_compress_varlen(L, *comp, x, B, cu_seqlens, N, T_max, pos, frontier, pool, cap, n_rows,
                                            inv_freq, w, err, static_cast<cudaStream_t>(stream)));
}

csa_status csa_attend_prefill_varlen(const csa_layer* layer, const void* q, const void* kv_new, const void* iq,
                                     const void* iw, const float* sink, int B, const int32_t* cu_seqlens, int N,
                                     int T_max, const int32_t* pos, void* window, const void* pool,
                                     const void* ikeys, int cap, const int32_t* n_rows, const float* inv_freq,
                                     void* out, int32_t* sel_out, void* ws, size_t ws_bytes, int32_t* err,
                                     void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!varlen_args_ok(B, cu_seqlens, N, T_max) || N > 16384 || cap < 1) return CSA_ERR_ARG;
  if (!tc_attend_supported(L) || (L.has_indexer() && !tc_index_supported(L))) return CSA_ERR_UNSUPPORTED;
  if (!dev_tensor(q) || !dev_tensor(kv_new) || !dev_i32(sink) || !dev_tensor(window) || !dev_tensor(pool) ||
      !dev_tensor(inv_freq) || !dev_tensor(out))
    return CSA_ERR_ARG;
  if (!dev_i32(pos) || !dev_i32(n_rows) || !dev_i32(err)) return CSA_ERR_ARG;
  if (L.has_indexer() && (!dev_tensor(iq) || !dev_i32(iw) || !dev_tensor(ikeys))) return CSA_ERR_ARG;
  if (sel_out && !dev_i32(sel_out)) return CSA_ERR_ARG;
  const size_t need = ws_prefill(L, N, cap);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  IndexWs iws{};
  int32_t *sel = nullptr, *n_sel = nullptr;
  AttendWs aw{};
  carve_prefill(c, L, N, cap, &iws, &sel, &n_sel, &aw);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (L.has_indexer()) {
    if (sel_out) sel = sel_out;
    cudaError_t e = launch_index_topk(L, iq, iw, N, ikeys, cap, n_rows, pos, B, inv_freq, sel, n_sel, iws, err, s,
                                      cu_seqlens);
    if (e != cudaSuccess) return CSA_ERR_CUDA;
  } else if (sel_out && L.topk > 0) {
    cudaMemsetAsync(sel_out, 0xff, (size_t)N * L.topk * sizeof(int32_t), s);
  }
  return cuda_status(launch_attend_prefill_varlen(L, q, kv_new, sink, B, cu_seqlens, N, T_max, window, pool, cap,
                                                  n_rows, L.has_indexer() ? sel : nullptr, n_sel, pos, inv_freq,
                                                  out, aw, err, s));
}

csa_status csa_index_topk_verify(const csa_layer* layer, const void* iq, const void* iw, int B, int T,
                                 const void* ikeys, int cap, const int32_t* n_rows, const int32_t* pos,
                                 const float* inv_freq, int32_t* sel, int32_t* n_sel, void* ws, size_t ws_bytes,
                                 int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!L.has_indexer()) return CSA_ERR_UNSUPPORTED;
  if (B < 1 || T < 1 || T > 64 || cap < 1 || (long long)B * T > (1 << 20)) return CSA_ERR_ARG;
  if (!dev_tensor(iq) || !dev_i32(iw) || !dev_tensor(ikeys) || !dev_tensor(inv_freq)) return CSA_ERR_ARG;
  if (!dev_i32(n_rows) || !dev_i32(pos) || !dev_i32(sel) || !dev_i32(n_sel) || !dev_i32(err)) return CSA_ERR_ARG;
  const size_t need = ws_index(L, B * T, cap);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  IndexWs w = carve_index(c, L, B * T, cap);
  // with device positions the index kernels take the queries per sequence in place of pos0
  return cuda_status(launch_index_topk(L, iq, iw, B * T, ikeys, cap, n_rows, pos, T, inv_freq, sel, n_sel, w, err,
                                       static_cast<cudaStream_t>(stream)));
}

csa_status csa_attend_verify(const csa_layer* layer, const void* q, const void* kv_new, const float* sink, int B, int T,
                             void* window, const void* pool, int cap, const int32_t* n_rows, const int32_t* sel,
                             const int32_t* n_sel, const int32_t* pos, const float* inv_freq, void* out, void* ws,
                             size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!L.has_indexer() || !tc_attend_decode_supported(L)) return CSA_ERR_UNSUPPORTED;
  if (B < 1 || T < 1 || T > 64 || cap < 1 || (long long)B * T > (1 << 20)) return CSA_ERR_ARG;
  if (T - 1 > L.rollback) return CSA_ERR_ARG;  // the block's later tokens would overwrite window rows still attended
  if (!dev_tensor(q) || !dev_tensor(kv_new) || !dev_i32(sink) || !dev_tensor(window) || !dev_tensor(pool) ||
      !dev_tensor(inv_freq) || !dev_tensor(out))
    return CSA_ERR_ARG;
  if (!dev_i32(n_rows) || !dev_i32(pos) || !dev_i32(err) || !dev_i32(sel) || !dev_i32(n_sel)) return CSA_ERR_ARG;
  const size_t need = ws_decode(L, B * T, cap);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  AttendWs w = carve_attend(c, L, B * T, attend_splits(L, false, false, cap), 0);
  return cuda_status(launch_attend_verify(L, q, kv_new, sink, B, T, window, pool, cap, n_rows, sel, n_sel, pos,
                                          inv_freq, out, w, err, static_cast<cudaStream_t>(stream)));
}

csa_status csa_trim(const csa_layer* layer, int B, const int32_t* n_back, int32_t* pos, int32_t* n_rows_a,
                    int32_t* n_rows_i, int32_t* hw, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (B < 0) return CSA_ERR_ARG;
  if (B == 0) return CSA_OK;
  if (!dev_i32(n_back) || !dev_i32(pos) || !dev_i32(n_rows_a) || !dev_i32(hw) || !dev_i32(err)) return CSA_ERR_ARG;
  if (n_rows_i && !dev_i32(n_rows_i)) return CSA_ERR_ARG;
  if (L.has_indexer() && !n_rows_i) return CSA_ERR_ARG;
  return cuda_status(launch_trim(L, B, n_back, pos, n_rows_a, n_rows_i, hw, err, static_cast<cudaStream_t>(stream)));
}

csa_status csa_advance_positions(int32_t* pos, int B, int by, void* stream) {
  if (B < 0 || (B > 0 && !pos)) return CSA_ERR_ARG;
  if (B == 0) return CSA_OK;
  return cuda_status(launch_advance_positions(pos, B, by, static_cast<cudaStream_t>(stream)));
}

csa_status csa_index_rows_fp8(const csa_layer* layer, const void* src, long long n, void* dst, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!L.ikey_fp8) return CSA_ERR_UNSUPPORTED;
  if (n < 0 || n > (1LL << 34)) return CSA_ERR_ARG;
  if (n == 0) return CSA_OK;
  if (!dev_tensor(src) || !dev_tensor(dst)) return CSA_ERR_ARG;
  return cuda_status(launch_index_rows_fp8(src, n, dst, static_cast<cudaStream_t>(stream)));
}

csa_status csa_norm_rope(const csa_layer* layer, const csa_rows* rows, int n, int B, int T, const int32_t* parent,
                         const int32_t* pos, const float* inv_freq, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!rows || n < 1 || n > 4 || B < 1 || T < 1 || (long long)B * T > (1 << 24) || !dev_i32(err)) return CSA_ERR_ARG;
  if (parent && (!dev_i32(parent) || T > 64)) return CSA_ERR_ARG;
  if (inv_freq && (!dev_tensor(inv_freq) || !dev_i32(pos))) return CSA_ERR_ARG;
  for (int k = 0; k < n; ++k) {
    const csa_rows& r = rows[k];
    if (!dev_tensor(r.x) || !dev_tensor(r.out) || (r.weight && !dev_tensor(r.weight))) return CSA_ERR_ARG;
    if (r.heads < 1 || r.heads > 4096 || r.dim < 8 || r.dim > 1024 || r.dim % 8 || r.dim < L.R || (r.dim - L.R) % 8 ||
        (r.norm != 0 && r.norm != 1))
      return CSA_ERR_ARG;
    const long long dense = (long long)r.heads * r.dim;
    if (r.x_stride != 0 && (r.x_stride < dense || r.x_stride % 8)) return CSA_ERR_ARG;
    if (r.x == r.out && r.x_stride > dense) return CSA_ERR_ARG;
  }
  return cuda_status(launch_norm_rope(L, rows, n, B, T, parent, pos, inv_freq, err,
                                      static_cast<cudaStream_t>(stream)));
}

csa_status csa_compress_tree(const csa_layer* layer, const csa_compressor* comp_a, const csa_compressor* comp_i,
                             const void* x, int B, int T, const int32_t* parent, const int32_t* pos,
                             const void* frontier_a, void* proj_a, void* rows_a, const void* frontier_i, void* proj_i,
                             void* rows_i, const float* inv_freq, void* ws, size_t ws_bytes, int32_t* err,
                             void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!tree_sizes_ok(B, T)) return CSA_ERR_ARG;
  if (comp_i && !L.has_indexer()) return CSA_ERR_UNSUPPORTED;
  if (!compress_args_ok(L, comp_a, B, T, 1, frontier_a, proj_a, pos) || comp_a->d != L.D || !dev_tensor(rows_a))
    return CSA_ERR_ARG;
  if (comp_i && (!compress_args_ok(L, comp_i, B, T, 1, frontier_i, proj_i, pos) || comp_i->d != L.Di ||
                 !dev_tensor(rows_i)))
    return CSA_ERR_ARG;
  if (!dev_tensor(x) || !dev_i32(parent) || !dev_tensor(inv_freq) || !dev_i32(err)) return CSA_ERR_ARG;
  const size_t need = ws_compress_tree(L, comp_i != nullptr, B, T);
  if (ws_bytes < need || (need && !dev_tensor(ws))) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  TreeCompress pools[2] = {};
  pools[0] = TreeCompress{comp_a, frontier_a, proj_a, rows_a, carve_compress_tree(c, L, L.D, B, T)};
  if (comp_i) pools[1] = TreeCompress{comp_i, frontier_i, proj_i, rows_i, carve_compress_tree(c, L, L.Di, B, T)};
  return cuda_status(launch_compress_tree(L, pools, comp_i ? 2 : 1, x, B, T, parent, pos, inv_freq, err,
                                          static_cast<cudaStream_t>(stream)));
}

csa_status csa_index_scores_tree(const csa_layer* layer, const void* iq, const void* iw, int B, int T,
                                 const int32_t* parent, const void* ikeys, int cap, const void* rows_i,
                                 const int32_t* n_rows, const int32_t* pos, float* scores, void* ws, size_t ws_bytes,
                                 int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!L.has_indexer()) return CSA_ERR_UNSUPPORTED;
  if (!tree_sizes_ok(B, T) || cap < 1 || cap > kTreeCapMax) return CSA_ERR_ARG;
  if (!dev_tensor(iq) || !dev_tensor(iw) || !dev_tensor(ikeys) || !dev_tensor(rows_i) || !dev_i32(scores))
    return CSA_ERR_ARG;
  if (!dev_i32(parent) || !dev_i32(n_rows) || !dev_i32(pos) || !dev_i32(err)) return CSA_ERR_ARG;
  const size_t need = tree_scores_ws(L, B, T);
  if (ws_bytes < need || (need && !dev_tensor(ws))) return CSA_ERR_WORKSPACE;
  return cuda_status(launch_index_scores_tree(L, iq, iw, B, T, parent, ikeys, cap, rows_i, n_rows, pos, scores, ws, err,
                                              static_cast<cudaStream_t>(stream)));
}

csa_status csa_attend_tree(const csa_layer* layer, const void* q, const void* kv, const float* sink, int B, int T,
                           const int32_t* parent, const void* window, const void* pool, int cap, const void* rows_a,
                           const float* scores, const int32_t* n_rows, const int32_t* pos, const float* inv_freq,
                           void* out, int32_t* sel_out, void* ws, size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!tree_sizes_ok(B, T) || cap < 1 || (long long)cap + T + L.W > kTreeCapMax) return CSA_ERR_ARG;  // (a node's keys)
  if (!dev_tensor(q) || !dev_tensor(kv) || !dev_i32(sink) || !dev_tensor(window) || !dev_tensor(pool) ||
      !dev_tensor(rows_a) || !dev_tensor(inv_freq) || !dev_tensor(out))
    return CSA_ERR_ARG;
  if (!dev_i32(parent) || !dev_i32(n_rows) || !dev_i32(pos) || !dev_i32(err)) return CSA_ERR_ARG;
  if (scores && (!L.has_indexer() || !dev_i32(scores))) return CSA_ERR_ARG;
  if (sel_out && (!scores || !dev_i32(sel_out))) return CSA_ERR_ARG;
  const size_t need = ws_attend_tree(L, B, T, cap);
  if (ws_bytes < need || (need && !dev_tensor(ws))) return CSA_ERR_WORKSPACE;
  Carver c(ws);
  TreeAttend t{q, kv, window, pool, rows_a, scores, sink, inv_freq, parent, n_rows, pos, out, sel_out, B, T, cap,
               carve_attend_tree(c, L, B, T, cap)};
  return cuda_status(launch_attend_tree(L, t, err, static_cast<cudaStream_t>(stream)));
}

csa_status csa_commit_tree(const csa_layer* layer, int B, int T, const int32_t* parent, const int32_t* leaf,
                           const int32_t* pos, int32_t* pos_out, const void* kv, void* window, const void* proj_a,
                           void* frontier_a, const void* rows_a, void* pool_a, int cap_a, const int32_t* n_rows_a,
                           int32_t* n_rows_a_out, const void* proj_i, void* frontier_i, const void* rows_i,
                           void* pool_i, int cap_i, const int32_t* n_rows_i, int32_t* n_rows_i_out, int32_t* err,
                           void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (!tree_sizes_ok(B, T) || cap_a < 1) return CSA_ERR_ARG;
  if (!dev_i32(parent) || !dev_i32(leaf) || !dev_i32(pos) || !dev_i32(pos_out) || !dev_i32(err)) return CSA_ERR_ARG;
  if (!dev_tensor(kv) || !dev_tensor(window) || !dev_tensor(proj_a) || !dev_tensor(frontier_a) ||
      !dev_tensor(rows_a) || !dev_tensor(pool_a) || !dev_i32(n_rows_a) || !dev_i32(n_rows_a_out))
    return CSA_ERR_ARG;
  if (pool_i) {
    if (!L.has_indexer()) return CSA_ERR_UNSUPPORTED;
    if (!dev_tensor(proj_i) || !dev_tensor(frontier_i) || !dev_tensor(rows_i) || !dev_tensor(pool_i) || cap_i < 1 ||
        !dev_i32(n_rows_i) || !dev_i32(n_rows_i_out))
      return CSA_ERR_ARG;
  }
  TreeCommit t{};
  t.parent = parent; t.leaf = leaf; t.pos = pos; t.pos_out = pos_out; t.kv = kv; t.window = window;
  t.proj[0] = proj_a; t.rows[0] = rows_a; t.frontier[0] = frontier_a; t.pool[0] = pool_a;
  t.n_rows[0] = n_rows_a; t.n_rows_out[0] = n_rows_a_out; t.cap[0] = cap_a;
  t.proj[1] = proj_i; t.rows[1] = rows_i; t.frontier[1] = frontier_i; t.pool[1] = pool_i;
  t.n_rows[1] = n_rows_i; t.n_rows_out[1] = n_rows_i_out; t.cap[1] = cap_i;
  t.npool = pool_i ? 2 : 1; t.B = B; t.T = T;
  return cuda_status(launch_commit_tree(L, t, err, static_cast<cudaStream_t>(stream)));
}

csa_status csa_add_norm(const csa_layer* layer, const void* x, long long x_stride, const void* residual,
                        long long residual_stride, const float* weight, long long N, int X, void* out,
                        void* residual_out, void* codes, float* scales, int group, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (N < 0 || N > INT32_MAX || X < 8 || X % 8 || X > 16384) return CSA_ERR_ARG;
  if (N == 0) return CSA_OK;  // (its tensors may have no address)
  if ((codes == nullptr) != (scales == nullptr) || (!out && !residual_out && !codes)) return CSA_ERR_ARG;
  if (codes && group != X && (group < 8 || group > 256 || (group & (group - 1)) || X % group)) return CSA_ERR_ARG;
  if (!dev_tensor(x) || (residual && !dev_tensor(residual)) || (weight && !dev_tensor(weight))) return CSA_ERR_ARG;
  if ((out && !dev_tensor(out)) || (residual_out && !dev_tensor(residual_out)) || (codes && !dev_tensor(codes)) ||
      (scales && !dev_i32(scales)))
    return CSA_ERR_ARG;
  for (long long stride : {x_stride, residual_stride})
    if (stride != 0 && (stride < X || stride % 8 || stride > (1LL << 31) || stride > kSpan / N)) return CSA_ERR_ARG;
  AddNorm t{x, residual, weight, out, residual_out, static_cast<uint8_t*>(codes), scales, N,
            x_stride ? x_stride : X, residual_stride ? residual_stride : X, X, codes ? group : X};
  // a thread writes what it has read itself: an output may be a dense input, and nothing else that is read or written
  const long long es = (long long)esize(L.dtype), row = X * es, n = N;
  const Span in[2] = {Span(x, n, row, t.x_stride * es), Span(residual ? residual : x, n, row, (residual ? t.r_stride : t.x_stride) * es)};
  const long long in_stride[2] = {t.x_stride, residual ? t.r_stride : t.x_stride};
  const void* outs[4] = {out, residual_out, codes, scales};
  const long long bytes[4] = {row, row, X, (long long)(X / t.group) * 4};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    const Span o(outs[i], n, bytes[i], bytes[i]);
    for (int k = 0; k < 2; ++k)
      if (o.meets(in[k]) && !(i < 2 && o.lo == in[k].lo && in_stride[k] == X)) return CSA_ERR_ARG;
    if (weight && o.meets(Span(weight, 1, X * 4LL, 0))) return CSA_ERR_ARG;
    for (int k = 0; k < i; ++k)
      if (outs[k] && o.meets(Span(outs[k], n, bytes[k], bytes[k]))) return CSA_ERR_ARG;
  }
  return cuda_status(launch_add_norm(L, t, static_cast<cudaStream_t>(stream)));
}

csa_status csa_append_pages(const csa_layer* layer, const csa_pages* pages, const void* rows, long long stride_b,
                            long long stride_t, int B, int T, const int32_t* table, int width, const int32_t* pos,
                            const int32_t* n_new, const float* weight, int norm, const float* inv_freq, int32_t* err,
                            void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (B < 1 || T < 1 || (long long)B * T > (1 << 24) || (norm != 0 && norm != 1)) return CSA_ERR_ARG;
  if (!pages_ok(pages) || !table_ok(pages, table, width) || !dev_tensor(rows) || !dev_i32(pos) || !dev_i32(err))
    return CSA_ERR_ARG;
  if ((n_new && !dev_i32(n_new)) || (weight && !dev_tensor(weight)) || (inv_freq && !dev_tensor(inv_freq)))
    return CSA_ERR_ARG;
  if (stride_t != 0 && (stride_t < L.D || stride_t % 8 || stride_t > (1LL << 31))) return CSA_ERR_ARG;
  const long long st_t = stride_t ? stride_t : L.D, st_b = stride_b ? stride_b : T * st_t;
  if (st_b % 8 || st_b < 0 || st_b > (1LL << 40) || st_b > kSpan / B) return CSA_ERR_ARG;
  const long long es = (long long)esize(L.dtype), n_rows = (long long)pages->n_pages * pages->page_rows;
  const Span outs[] = {Span(pages->codes, n_rows * L.D), Span(pages->scales, n_rows * 4), Span(err, 4)};
  const Span ins[] = {Span(rows, ((B - 1) * st_b + (T - 1) * st_t + L.D) * es), Span(table, (long long)B * width * 4),
                      Span(pos, B * 4LL), Span(n_new, B * 4LL), Span(weight, L.D * 4LL), Span(inv_freq, L.R * 2LL)};
  if (!apart(outs, ins)) return CSA_ERR_ARG;
  PagedAppend t{rows, st_b, st_t, static_cast<uint8_t*>(pages->codes), pages->scales, table, pos, n_new, weight,
                inv_freq, err, L.eps, pages->n_pages, pages->page_rows, width, B, T, L.D, L.R, norm};
  return cuda_status(launch_append_pages(L, t, static_cast<cudaStream_t>(stream)));
}

csa_status csa_attend_pages(const csa_layer* layer, const csa_pages* pages, const void* q, int B, int T,
                            const float* sink, const int32_t* pos, const int32_t* n_new, const int32_t* token_table,
                            int token_width, int first, const int32_t* row_table, int row_width, const int32_t* n_rows,
                            const int32_t* sel, const int32_t* n_sel, const float* inv_freq, void* out, void* ws,
                            size_t ws_bytes, int32_t* err, void* stream) {
  Dims L;
  csa_status st = make_dims(layer, &L);
  if (st != CSA_OK) return st;
  if (B < 1 || T < 1 || (long long)B * T > kPagedQueries || first < 0) return CSA_ERR_ARG;
  if (!pages_ok(pages) || !dev_tensor(q) || !dev_tensor(out) || !dev_i32(pos) || !dev_i32(err)) return CSA_ERR_ARG;
  if (!token_table && !row_table) return CSA_ERR_ARG;
  if (token_table && !table_ok(pages, token_table, token_width)) return CSA_ERR_ARG;
  if (row_table && (!table_ok(pages, row_table, row_width) || !dev_i32(n_rows))) return CSA_ERR_ARG;
  if (sel && (!row_table || !L.has_indexer() || !dev_i32(sel) || !dev_i32(n_sel))) return CSA_ERR_ARG;
  if ((sink && !dev_i32(sink)) || (n_new && !dev_i32(n_new)) || (inv_freq && !dev_tensor(inv_freq)))
    return CSA_ERR_ARG;
  const long long n = (long long)B * T;
  // a query's keys and the tiles of a call are counted in ints; the smallest hold 32 keys, and each of a query's three
  // sections ends one
  const long long P = pages->page_rows;
  const long long most = (row_table ? (sel ? (long long)L.topk : row_width * P) : 0) + (token_table ? token_width * P : 0);
  if (most > INT32_MAX - 256 || n * (most / 32 + 4) > INT32_MAX) return CSA_ERR_ARG;
  const size_t need = ws_attend_pages(L, (int)n);
  if (ws_bytes < need || !dev_tensor(ws)) return CSA_ERR_WORKSPACE;
  const long long q_bytes = n * L.H * L.D * (long long)esize(L.dtype), n_slots = pages->n_pages * P;
  const Span outs[] = {Span(out, q_bytes), Span(ws, (long long)need), Span(err, 4)};
  const Span ins[] = {Span(pages->codes, n_slots * L.D), Span(pages->scales, n_slots * 4), Span(q, q_bytes), Span(sink, L.H * 4LL),
                      Span(pos, B * 4LL), Span(n_new, B * 4LL), Span(token_table, (long long)B * token_width * 4),
                      Span(row_table, (long long)B * row_width * 4), Span(row_table ? n_rows : nullptr, B * 4LL),
                      Span(sel, n * L.topk * 4), Span(sel ? n_sel : nullptr, n * 4), Span(inv_freq, L.R * 2LL)};
  if (!apart(outs, ins)) return CSA_ERR_ARG;
  PagedArgs a{};
  Carver c(ws);
  carve_paged(c, L, (int)n, &a);
  a.codes = static_cast<const uint8_t*>(pages->codes);
  a.scales = pages->scales;
  a.q = q; a.out = out; a.sink = sink; a.inv_freq = inv_freq;
  a.pos = pos; a.n_new = n_new; a.token_table = token_table; a.row_table = row_table; a.n_rows = n_rows;
  a.sel = sel; a.n_sel = n_sel;
  a.by_page = fast_div((uint32_t)pages->page_rows);
  a.by_T = fast_div((uint32_t)T);
  a.by_ratio = fast_div((uint32_t)L.ratio);
  a.n_pages = pages->n_pages; a.P = pages->page_rows; a.token_pages = token_width; a.row_pages = row_width;
  a.B = B; a.T = T; a.H = L.H; a.D = L.D; a.R = L.R; a.W = L.W; a.first = first; a.ratio = L.ratio; a.topk = L.topk;
  a.scale2 = L.scale * 1.4426950408889634f;
  a.err = err;
  return cuda_status(launch_attend_pages(L, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
