/*
 * csa.h — C ABI of one layer of DeepSeek-V4 Compressed Sparse Attention (CSA)
 * on a single GB300 (sm_103a).
 *
 * The layer (DeepSeek-V4-Flash shapes) has four parts, each a call here:
 *   csa_compress_append      gated-pooling compressor: projects tokens, pools
 *                            ratio-4 overlapping or ratio-128 windows, RMSNorm,
 *                            RoPE at the window start, appends rows to a pool.
 *   csa_index_topk           indexer: ReLU-weighted multi-head scores of the
 *                            query against the index-key pool, exact top-k.
 *   csa_attend_decode        MQA-shaped attention of H heads over one shared
 *                            latent (K = V): selected pool rows + sliding
 *                            window, sink logits, split-K partial softmax and
 *                            merge, inverse RoPE on the output.
 *   csa_attend_prefill_chunk the same for a chunk of T queries of one
 *                            sequence, each with its own causal top-k.
 *   (*_varlen: a packed batch of chunks of different lengths; *_verify: verify
 *   blocks of T tokens per sequence; csa_trim: rewind for speculative decoding;
 *   csa_norm_rope: per-head norm and rotation of what they take; *_tree: a tree
 *   of drafted tokens per sequence; csa_add_norm: the hidden states' norm, in
 *   the model dtype and 8 bits; *_pages: a cache in pages and 8 bits.)
 *
 * Definitions follow the pages the method is described on:
 *   [MTPLX#216]  "DeepSeek-V4-Flash: native deepseek_v4 AR backend"
 *   [mlx-lm#1189] "feat: add DeepSeek-V4 (Pro/Flash) model support"
 *   [v41-mlx]    "deepseek-v41-mlx" README
 *
 * Conventions for every call
 *   - Every tensor argument is a DEVICE pointer owned by the caller, dense,
 *     row-major, 16-byte aligned.  The library never allocates or frees device
 *     memory and keeps no state between calls.  Scratch memory comes from the
 *     caller through (ws, ws_bytes); csa_workspace_size() gives the size.
 *   - Storage dtype (layer->dtype): CSA_BF16 or CSA_F32 for activations,
 *     weights, pools, windows and outputs ("model dtype").  APE, norm weights,
 *     sink logits and the RoPE table are always fp32.  Arithmetic is fp32.
 *   - Any host thread may call, several at once; calls in flight together need
 *     workspaces and outputs of their own (the static scratch: see that call).
 *   - All work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream).  No call synchronises or reads device memory
 *     on the host, so calls can be captured in a CUDA graph.
 *   - Kernels are launched with programmatic dependent launch: each lets its
 *     successor in the stream start early and waits for its predecessor before
 *     reading anything that predecessor chain writes.  Before that wait a
 *     kernel may read its call's step inputs (queries, new tokens, weights,
 *     positions) and the window ring, so these must be complete when the call
 *     is enqueued behind work that does not trigger early (any ordinary kernel
 *     or copy; csa_advance_positions for pos).
 *     Of the *_tree calls' inputs these are x, the weights and pos; whatever else
 *     they read (parent, kv, rings, pools, draft buffers) may come from any call
 *     before them.
 *   - Errors found on the host are returned synchronously, before anything is
 *     enqueued (fail closed: nothing is modified).  Errors that depend on
 *     device-resident values (positions, row counts, indices) are OR-ed into
 *     the caller's device error word `err` (CSA_DEV_* bits) and the offending
 *     sequence / row is skipped; no call traps or asserts on the device.
 *   - RoPE: rope dims are the LAST R dims of a row, rotated as interleaved
 *     pairs (D-R+2i, D-R+2i+1) by theta_i = (float)p * inv_freq[i] (one fp32
 *     multiply).  inv_freq is a device fp32 table of R/2 entries, so the
 *     caller chooses plain or YaRN-scaled frequencies ([mlx-lm#1189], OmarB97's
 *     RoPE fixes: the rotary setting depends on the layer kind, and compress
 *     layers use base 160000).
 */
#ifndef CSA_H
#define CSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CSA_OK = 0,
  CSA_ERR_ARG = 1,         /* null / misaligned pointer, inconsistent or out-of-range sizes */
  CSA_ERR_UNSUPPORTED = 2, /* valid arguments with no kernel for them (see each call) */
  CSA_ERR_CUDA = 3,        /* a kernel launch failed (cudaGetLastError after enqueue) */
  CSA_ERR_WORKSPACE = 4    /* ws_bytes smaller than csa_workspace_size() */
} csa_status;

enum { CSA_F32 = 0, CSA_BF16 = 1 };

/* bits of the device error word */
enum {
  CSA_DEV_CAPACITY = 1, /* a compress call would emit a row at index >= cap: sequence skipped */
  CSA_DEV_STATE = 2,    /* n_rows[b] != floor(pos[b] / ratio) or pos[b] < 0: sequence skipped */
  CSA_DEV_RANGE = 4,    /* a selected row index outside [0, n_rows[b]): that row is skipped */
  CSA_DEV_ROLLBACK = 8  /* csa_trim beyond the rollback margin (or below 0): sequence left unchanged */
};

/* operation ids for csa_workspace_size */
enum {
  CSA_OP_COMPRESS = 0,
  CSA_OP_INDEX_TOPK = 1,
  CSA_OP_ATTEND_DECODE = 2,
  CSA_OP_ATTEND_PREFILL = 3,
  CSA_OP_COMPRESS_PAIR = 4, /* csa_compress_append_pair (ratio-4 layers) */
  CSA_OP_COMPRESS_VARLEN = 5,       /* csa_compress_append_varlen: B sequences, T = N packed tokens */
  CSA_OP_ATTEND_PREFILL_VARLEN = 6, /* csa_attend_prefill_varlen: B sequences, T = N packed tokens */
  CSA_OP_COMPRESS_TREE = 7,         /* csa_compress_tree: B trees of T nodes */
  CSA_OP_ATTEND_TREE = 8,           /* csa_attend_tree: B trees of T nodes */
  CSA_OP_INDEX_SCORES_TREE = 9,     /* csa_index_scores_tree: B trees of T nodes */
  CSA_OP_ATTEND_PAGES = 10          /* csa_attend_pages: B sequences of T queries (cap ignored) */
};

/* One CSA layer.
 *   H query heads over one latent of D dims (K = V), rope on the last R dims;
 *   W-token sliding window; compress `ratio` (4: overlapping windows of 8
 *   tokens through two lanes, with the indexer; any other ratio r: one lane,
 *   non-overlapping windows of r tokens, no indexer); indexer Hi heads of Di
 *   dims keeping `topk` rows; hidden size X.
 *   scale: attention logit scale (the pages' kernels use D^-1/2; 0 selects it).
 *   rms_eps: RMSNorm epsilon of the compressed rows.
 *   rollback: tokens csa_trim may rewind (0: none).  The window ring then holds
 *     W + rollback slots (token t in slot t mod (W + rollback)) and each frontier
 *     ring csa_frontier_slots(ratio) + rollback slots (its journal of projected
 *     rows); a query still attends only its last W tokens.  Every call of a layer
 *     takes buffers of those sizes.
 *   index_fp8: 0 (index keys in the model dtype) or 1 (fp8 index rows of
 *     CSA_FP8_ROW_BYTES: the index pool, written by the compress calls and read
 *     by every index call (csa_index_topk, _verify, csa_attend_prefill_chunk,
 *     _varlen), is then a [B, cap, 144] byte tensor (a prefill chunk's ikeys
 *     [cap, 144]); ratio 4, bf16, Hi = 64, Di = 128 (D != 128), R <= 64 only,
 *     else CSA_ERR_UNSUPPORTED; csa_index_topk_overlapped returns
 *     CSA_ERR_UNSUPPORTED with it). */
typedef struct {
  int dtype;
  int H, D, R, W, ratio, Hi, Di, topk, X;
  float scale;
  float rms_eps;
  int rollback;
  int index_fp8;
} csa_layer;

/* Bytes of one index-key row when layer->index_fp8 = 1: the row (already in
 * the model dtype, as the bf16 format would store it) rotated by the
 * unnormalised 128-point Walsh-Hadamard transform (fp32 butterflies of span
 * 1, 2, .., 64), as 128 E4M3 codes of rotated / scale (nearest even,
 * saturating), then the fp32 scale = amax / 448 at byte 128, then padding.
 * The index queries are rotated and quantised per head the same way and a
 * score is the bf16 definition on the decoded values, divided by 128
 * ([mlx-lm#1189], the indexer thread: a Hadamard rotation and a low-precision
 * activation simulation in the indexer, the rotation cancelling in the dot
 * product; the format itself is this library's choice). */
#define CSA_FP8_ROW_BYTES 144

/* One compressor (the attention pool's, d = D, or the index pool's, d = Di).
 * L = 2 lanes when ratio == 4, else 1.
 *   wkv, wgate [L*d, X] model dtype (out-features x in-features);
 *   ape  [ratio, L*d] fp32: absolute position embedding added to the gates;
 *   norm_w [d] fp32: RMSNorm weight.
 * Lane 0 (first d outputs) pools the previous window, lane 1 the current one.
 * For the Flash ratio-4 attention pool that makes ape [4, 1024] and wkv, wgate
 * [1024, 4096] ([mlx-lm#1189], Thump604's fixes, on the overlap compressor's
 * weight shapes). */
typedef struct {
  const void* wkv;
  const void* wgate;
  const float* ape;
  const float* norm_w;
  int d;
} csa_compressor;

/* Frontier ring length in tokens without a rollback journal: 2*ratio when
 * ratio == 4, else ratio (a layer with rollback r adds r slots). */
int csa_frontier_slots(int ratio);

/* Bytes of scratch memory `op` needs for batch B (T: tokens per sequence for
 * CSA_OP_COMPRESS, chunk length for CSA_OP_ATTEND_PREFILL, else ignored) and
 * pool capacity `cap` rows.  Returns CSA_ERR_ARG on bad dimensions. */
csa_status csa_workspace_size(const csa_layer* layer, int op, int B, int T, int cap, size_t* bytes);

/* csa_compress_append — append T tokens per sequence to one compressed pool.
 *
 * Definition ([MTPLX#216] "What V4 adds": learned gated pooling over
 * overlapping ratio-4 or non-overlapping ratio-128 windows, maintained
 * incrementally by prefill and decode alike; [mlx-lm#1189] OmarB97's RoPE
 * fixes: a pool row is rotated when emitted; stepnoy "Fix" 3: the chunk tail is carried
 * and the absolute position accumulates; [MTPLX#216] "Decode path": the row is
 * pooled in fp32 and cast back before the norm):
 *   for token p = pos[b] + i:  kv_p = Wkv x_p,  g_p = Wgate x_p  (model dtype)
 *   when p = (j+1)*ratio - 1 completes window j:
 *     entries: ratio 4 -> tokens of window j-1 via lane 0 (absent for j = 0)
 *              and tokens of window j via lane 1; otherwise window j's tokens;
 *     per channel c: u_c = sum_e softmax_e(g_e,c + ape[t_e mod ratio][c]) kv_e,c
 *     row j = RoPE(RMSNorm(u), j*ratio), rounded to the model dtype at each step,
 *     written to pool[b][j]; n_rows[b] = j + 1.
 * Arguments
 *   x        [B, T, X]             model dtype, tokens at pos[b] .. pos[b]+T-1
 *   pos      [B] int32 (device)    position of x[b][0]; the library never writes it
 *   frontier [B, F, 2*L*d]         model dtype, F = csa_frontier_slots(ratio) + layer->rollback:
 *                                  ring of the projected (kv | gate) rows of the last F tokens,
 *                                  slot t mod F; read for tokens before pos[b], rewritten for the
 *                                  last tokens
 *   pool     [B, cap, d]           model dtype, rows [0, n_rows[b]) valid
 *   n_rows   [B] int32 (device)    in/out; must equal floor(pos[b] / ratio) on entry
 *   inv_freq [R/2] fp32
 *   err      int32 (device)        error word (CSA_DEV_STATE, CSA_DEV_CAPACITY); a sequence
 *                                  that would fail is left entirely unchanged
 * Call it once for the attention pool and, on ratio-4 layers, once for the
 * index pool, with the same pos and the same n_rows values. */
csa_status csa_compress_append(const csa_layer* layer, const csa_compressor* comp, const void* x, int B, int T,
                               const int32_t* pos, void* frontier, void* pool, int cap, int32_t* n_rows,
                               const float* inv_freq, void* ws, size_t ws_bytes, int32_t* err, void* stream);

/* csa_compress_append_pair — both compressed pools of a ratio-4 layer (the
 * attention pool, comp_a with d = D, and the index pool, comp_i with d = Di) for
 * the same T tokens per sequence: the arguments, errors and definition of
 * csa_compress_append for the attention pool and then for the index pool, with
 * each pool's own frontier, pool, cap and n_rows, and one shared x, pos,
 * inv_freq and error word.  Results are those two calls' (identical for T > 1;
 * for one token the projections' fp32 sums may be split differently along the
 * hidden axis, within the projection's own rounding).  The pages compress both pools from the same hidden
 * states at the same positions ([MTPLX#216] "What V4 adds": the indexer keeps
 * its own compressed keys beside the attention pool).  Workspace:
 * CSA_OP_COMPRESS_PAIR.  With one token per sequence (decode) the two
 * projections run as one kernel and the two pooling steps as one, so that
 * neither call waits behind the other; longer chunks run the two calls in turn.
 * CSA_ERR_UNSUPPORTED on layers without an indexer (ratio != 4). */
csa_status csa_compress_append_pair(const csa_layer* layer, const csa_compressor* comp_a,
                                    const csa_compressor* comp_i, const void* x, int B, int T, const int32_t* pos,
                                    void* frontier_a, void* pool_a, int cap_a, int32_t* n_rows_a, void* frontier_i,
                                    void* pool_i, int cap_i, int32_t* n_rows_i, const float* inv_freq, void* ws,
                                    size_t ws_bytes, int32_t* err, void* stream);

/* csa_index_topk — the indexer for one decode query per sequence.
 *
 * Definition ([mlx-lm#1189] stepnoy's patch point 3 and aidiffuser's indexer:
 * raw head weights with the scale folded in, no sigmoid, ReLU on the logits,
 * sum over heads; the index pool accumulates in the cache so its row space is
 * the attention pool's; OmarB97: row j is visible to position p iff
 * (j+1)*ratio <= p+1):
 *   n_vis = min(n_rows[b], floor((pos[b]+1)/ratio))
 *   q_h   = RoPE(iq[b][h], pos[b])  (model dtype)
 *   s_j   = sum_h iw[b][h] * Di^-1/2 * Hi^-1/2 * max(q_h . ikeys[b][j], 0),  j < n_vis
 *   if n_vis <= topk: sel = 0 .. n_vis-1; else the topk largest s_j, ties to
 *   the lower j.  sel is written in ascending row order, padded with -1.
 * Arguments
 *   iq [B, Hi, Di], iw [B, Hi]   model dtype
 *   ikeys [B, cap, Di]           model dtype index-key pool
 *   n_rows, pos [B] int32 (device)
 *   sel [B, topk] int32, n_sel [B] int32 (device outputs)
 * Requires ratio == 4 (the layers that carry an indexer) and topk <= 4096. */
csa_status csa_index_topk(const csa_layer* layer, const void* iq, const void* iw, int B, const void* ikeys, int cap,
                          const int32_t* n_rows, const int32_t* pos, const float* inv_freq, int32_t* sel,
                          int32_t* n_sel, void* ws, size_t ws_bytes, int32_t* err, void* stream);

/* csa_index_topk_overlapped — csa_index_topk split around the index pool's
 * compress call for the same token, so that the scan of the cached index keys
 * (the bulk of the call) runs while that compress call runs on another stream.
 * The pages define the same selection as csa_index_topk and have no such split:
 * it is a scheduling form of that call, with identical outputs up to the
 * floating-point order of the two rows scored in its second stage.
 *   stage 1 (enqueued on `stream` at once): s_j for rows j < floor(pos[b]/ratio),
 *     the rows complete before the token; reads neither n_rows nor any index-key
 *     row the concurrent compress call may write;
 *   then `stream` waits for `pool_ready` (a cudaEvent_t recorded after
 *     csa_compress_append for the index pool and this token; NULL: no wait);
 *   stage 2: s_j for row floor(pos[b]/ratio) and row n_rows[b]-1 (the rows that
 *     call may have written), then the selection exactly as csa_index_topk.
 * Arguments, workspace (CSA_OP_INDEX_TOPK) and errors as csa_index_topk; the
 * caller orders the compress call after any earlier use of the index pool, and
 * must not start another call that writes ikeys or n_rows for these sequences
 * before this one completes.  Shapes the tensor-core scan does not cover, or
 * cap > 16384, run the whole call after the event.
 * One stream, no event: enqueued right after csa_compress_append(_pair) for the
 * same token on the same stream, with pool_ready NULL, stage 1 runs beside that
 * call's kernels: it does not wait for the kernels before it (it reads only the
 * rows complete before the token and the step's inputs, and writes only its
 * workspace) and waits for them at its end, and the compress call's projection
 * kernel lets its successors start only once all earlier work in the stream
 * is complete.  Enqueued behind anything else, stage 1's inputs must be complete
 * and its workspace free when it is enqueued behind work that does not trigger
 * early. */
csa_status csa_index_topk_overlapped(const csa_layer* layer, const void* iq, const void* iw, int B, const void* ikeys,
                                     int cap, const int32_t* n_rows, const int32_t* pos, const float* inv_freq,
                                     int32_t* sel, int32_t* n_sel, void* ws, size_t ws_bytes, int32_t* err,
                                     void* stream, void* pool_ready);

/* csa_attend_decode — one decode query per sequence.
 *
 * Definition ([MTPLX#216] "What V4 adds": 64 query heads over one 512-dim
 * latent with per-head sink logits and a 128-token sliding window; [v41-mlx]:
 * the inverse rope on the attention output, sinks in the softmax denominator
 * only; [mlx-lm#1189] stepnoy: decode gathers its own top-k rows so the softmax
 * is not diluted over the whole pool):
 *   window[b][p mod W] = RoPE(kv_new[b], p)            p = pos[b]
 *   keys  = pool[b][sel[b][0 .. n_sel[b])]  (sel == NULL: rows 0 .. n_vis-1)
 *           ++ window tokens t in [max(0, p-W+1), p]
 *   l_ht  = scale * RoPE(q[b][h], p) . key_t
 *   o_h   = sum_t e^{l_ht} key_t / (e^{sink[h]} + sum_t e^{l_ht})
 *   out[b][h] = RoPE^-1(o_h, p)   (model dtype before and after the rotation)
 * computed as split-K partial softmaxes (m, l, acc) merged in a second pass.
 * Arguments
 *   q [B, H, D], kv_new [B, D]   model dtype
 *   sink [H] fp32
 *   window [B, Wr, D]            model dtype ring, Wr = W + layer->rollback, slot t mod Wr
 *                                (written at slot p mod Wr)
 *   pool [B, cap, D]             model dtype
 *   n_rows, n_sel, pos [B] int32 (device); sel [B, topk] int32 or NULL
 *   out [B, H, D]                model dtype
 * A selected index outside [0, n_rows[b]) raises CSA_DEV_RANGE and is skipped. */
csa_status csa_attend_decode(const csa_layer* layer, const void* q, const void* kv_new, const float* sink, int B,
                             void* window, const void* pool, int cap, const int32_t* n_rows, const int32_t* sel,
                             const int32_t* n_sel, const int32_t* pos, const float* inv_freq, void* out, void* ws,
                             size_t ws_bytes, int32_t* err, void* stream);

/* csa_attend_prefill_chunk — T queries of one sequence at positions pos0 .. pos0+T-1.
 *
 * The compressors must already have consumed the chunk (n_rows counts the rows
 * emitted up to its end).  Each query p attends the pool rows visible to it,
 * reduced by its OWN top-k when the layer has an indexer and more than topk
 * rows are visible ([mlx-lm#1189] stepnoy's patch point 3: per-query top-k
 * AND-ed with the visibility mask; aidiffuser: build the membership from the
 * index list rather than a dense compare), plus its window tokens: ring
 * entries for tokens before pos0, the chunk's own kv_new roped at their
 * positions otherwise.  After the chunk the window ring holds its last
 * W + rollback tokens.  Same formulas as csa_attend_decode / csa_index_topk per query.
 * Arguments
 *   q [T, H, D], kv_new [T, D], iq [T, Hi, Di], iw [T, Hi]   model dtype (iq, iw,
 *                                  ikeys may be NULL when ratio != 4)
 *   sink [H] fp32; pos0 host int; window [W + rollback, D]; pool [cap, D]; ikeys [cap, Di]
 *   n_rows int32 (device, one value)
 *   out [T, H, D]; sel_out [T, topk] int32 or NULL (the selected rows, -1 padded)
 * Requires 1 <= T <= 16384 and ratio == 4 or no indexer use. */
csa_status csa_attend_prefill_chunk(const csa_layer* layer, const void* q, const void* kv_new, const void* iq,
                                    const void* iw, const float* sink, int T, int32_t pos0, void* window,
                                    const void* pool, const void* ikeys, int cap, const int32_t* n_rows,
                                    const float* inv_freq, void* out, int32_t* sel_out, void* ws, size_t ws_bytes,
                                    int32_t* err, void* stream);

/* csa_compress_append_varlen, csa_attend_prefill_varlen — a packed batch of
 * prefill chunks of different lengths (ragged batched prefill): sequence b's
 * chunk is rows cu_seqlens[b] .. cu_seqlens[b+1]-1 of every packed tensor, at
 * positions pos[b] .. pos[b] + T_b - 1 (T_b = cu_seqlens[b+1] - cu_seqlens[b]).
 *
 * Definition: for every sequence, exactly csa_compress_append on its chunk (each
 * pool), then csa_attend_prefill_chunk on it with pos0 = pos[b] ([MTPLX#216]
 * "Verification": decode == prefill across chunked prefill and batching).  The
 * sequences share the launches: one projection over the N packed tokens, and
 * per-query scoring, top-k and attention over all of them.
 * Arguments
 *   x [N, X]; q [N, H, D]; kv_new [N, D]; iq [N, Hi, Di]; iw [N, Hi]   model dtype,
 *     packed (iq, iw, ikeys may be NULL when ratio != 4)
 *   cu_seqlens int32 [B + 1] (device): 0 = cu[0] <= cu[1] <= ... <= cu[B] = N
 *     (an empty chunk is allowed); T_max (host) >= every T_b sizes the grids
 *   pos int32 [B] (device): each chunk's first position; not advanced here
 *   frontier, pool, n_rows, window, ikeys: per sequence as for csa_compress_append
 *     and csa_attend_decode ([B, ...] with pool capacity cap)
 *   out [N, H, D]; sel_out [N, topk] int32 or NULL
 * Workspace: csa_workspace_size(.., CSA_OP_COMPRESS_VARLEN, B, N, cap, ..) and
 *   (.., CSA_OP_ATTEND_PREFILL_VARLEN, B, N, cap, ..).
 * Errors: as the single-chunk calls; N <= 2^20 for the compress call and
 *   N <= 16384 for the attention call (CSA_ERR_ARG beyond).  A row-table entry
 *   with cu[b] < 0, cu[b+1] < cu[b] or cu[b+1] > N is flagged CSA_DEV_STATE by
 *   the compress call, which leaves that sequence unchanged; every packed row
 *   index the attention call derives from the table is clamped into [0, N).
 *   The attention call needs the tensor-core shapes (bf16, H = 64, D = 512,
 *   R = 64; Hi = 64, Di = 128 with an indexer): CSA_ERR_UNSUPPORTED otherwise. */
csa_status csa_compress_append_varlen(const csa_layer* layer, const csa_compressor* comp, const void* x, int B,
                                      const int32_t* cu_seqlens, int N, int T_max, const int32_t* pos,
                                      void* frontier, void* pool, int cap, int32_t* n_rows, const float* inv_freq,
                                      void* ws, size_t ws_bytes, int32_t* err, void* stream);
csa_status csa_attend_prefill_varlen(const csa_layer* layer, const void* q, const void* kv_new, const void* iq,
                                     const void* iw, const float* sink, int B, const int32_t* cu_seqlens, int N,
                                     int T_max, const int32_t* pos, void* window, const void* pool,
                                     const void* ikeys, int cap, const int32_t* n_rows, const float* inv_freq,
                                     void* out, int32_t* sel_out, void* ws, size_t ws_bytes, int32_t* err,
                                     void* stream);

/* csa_index_topk_verify, csa_attend_verify — a verify block: T consecutive tokens
 * per sequence (a speculative step's last accepted token and its T-1 drafts),
 * each query with its own causal top-k and attention, B sequences at once.
 *
 * Definition ([MTPLX#216], "Benchmark notes" and the MTP post: verification runs
 * a K+1-wide query block per sequence, the KV projected inside a K+1-wide GEMM;
 * the per-query semantics are those of a prefill chunk, [mlx-lm#1189] stepnoy's
 * patch point 3): call csa_compress_append (or _pair) with the block's T tokens
 * first; then, for query i of sequence b at p = pos[b] + i, the selection and the
 * output are csa_index_topk's and csa_attend_decode's at position p, with the
 * rows visible at p (those emitted by tokens <= p) and the window tokens
 * [p-W+1, p], the block's own earlier tokens included.  csa_attend_verify first
 * writes all T tokens, roped, to their ring slots (pos[b] + i) mod (W + rollback),
 * so the layer needs rollback >= T - 1 (else CSA_ERR_ARG): the block's later
 * tokens must not overwrite window rows its earlier queries attend.  Neither call
 * advances pos; after verification the caller advances it by T (csa_advance_positions)
 * and rewinds the rejected drafts with csa_trim.
 * Arguments as csa_index_topk / csa_attend_decode with one more axis of T queries
 * per sequence: iq [B, T, Hi, Di], iw [B, T, Hi], q [B, T, H, D], kv_new [B, T, D],
 * sel [B, T, topk], n_sel [B, T], out [B, T, H, D]; pos [B] is the position of each
 * block's first token; 1 <= T <= 64.  Workspaces: csa_workspace_size(..,
 * CSA_OP_INDEX_TOPK, B * T, 1, cap, ..) and (.., CSA_OP_ATTEND_DECODE, B * T, ..).
 * Tensor-core shapes (bf16, 64 x 512 latent, 64 x 128 indexer) with an indexer
 * (ratio 4); other layers get CSA_ERR_UNSUPPORTED. */
csa_status csa_index_topk_verify(const csa_layer* layer, const void* iq, const void* iw, int B, int T,
                                 const void* ikeys, int cap, const int32_t* n_rows, const int32_t* pos,
                                 const float* inv_freq, int32_t* sel, int32_t* n_sel, void* ws, size_t ws_bytes,
                                 int32_t* err, void* stream);
csa_status csa_attend_verify(const csa_layer* layer, const void* q, const void* kv_new, const float* sink, int B, int T,
                             void* window, const void* pool, int cap, const int32_t* n_rows, const int32_t* sel,
                             const int32_t* n_sel, const int32_t* pos, const float* inv_freq, void* out, void* ws,
                             size_t ws_bytes, int32_t* err, void* stream);

/* csa_trim — rewind sequences by n_back[b] tokens, exactly (speculative decoding:
 * the rejected draft tokens are taken back).
 *
 * Definition ([MTPLX#216], the MTP / speculative-lane post: the cache trim rewinds
 * every lane exactly; emitted compressed rows are truncated, since a row depends
 * only on its one completed window; the compressor frontiers are rebuilt from a
 * bounded journal of their own projected rows; the sliding window keeps
 * rollback_capacity extra rows, since an evicted row cannot be recovered; asked
 * to go further, trim refuses instead of clamping).  Here the journal and the
 * extra window rows are the layer's rollback slots (csa_layer.rollback), so a
 * trim moves no data: with p = pos[b] and p' = p - n_back[b],
 *   hw[b]       = max(hw[b], p)          (the highest position the sequence reached)
 *   refuse      if n_back[b] < 0, p' < 0, p' < hw[b] - rollback, or n_rows[b] != p / ratio
 *   pos[b]      = p'
 *   n_rows[b]   = p' / ratio  (for n_rows_a and, when given, n_rows_i)
 * After it, decoding tokens from p' gives bit for bit what the sequence would
 * have given had the rewound tokens never been decoded: the frontier ring still
 * holds the projections of the ratio-window tokens before p', the window ring
 * the W tokens before p', and pool rows past the new n_rows are rewritten when
 * their windows complete again.
 * Arguments (device, int32 [B]): n_back; pos, n_rows_a (attention pool) and
 * n_rows_i (index pool; NULL for layers without an indexer) in/out; hw in/out,
 * caller-owned, set to the sequence's position when it starts (0 for a new one).
 * A refused sequence is left entirely unchanged and CSA_DEV_ROLLBACK (or
 * CSA_DEV_STATE) is OR-ed into err.  One small kernel on `stream`. */
csa_status csa_trim(const csa_layer* layer, int B, const int32_t* n_back, int32_t* pos, int32_t* n_rows_a,
                    int32_t* n_rows_i, int32_t* hw, int32_t* err, void* stream);

/* csa_norm_rope — the rows that attention and the indexer take, prepared in one
 * pass: per token and head, an RMS norm and the rotation.
 *
 * Definition (heads normalised one by one, the latent with its weight, then RoPE
 * in fp32: [MTPLX#216] "What V4 adds"; OmarB97's RoPE fixes in [mlx-lm#1189]):
 *   y = x * (mean(x^2) + rms_eps)^-1/2 * weight   (norm != 0; weight NULL: ones)
 *   out = RoPE(y, p), p = pos[b] + depth           (inv_freq NULL: no rotation)
 * in fp32, rounded to the model dtype once.  depth is the node's depth in its
 * sequence's tree when `parent` is given (see csa_compress_tree; T <= 64) and
 * the token's index i otherwise, so one call serves a decode step (T = 1), a
 * chunk, a verify block and a tree.  With inv_freq NULL the rows are only
 * normalised: what csa_attend_decode, _prefill_chunk, _verify take, which rotate
 * by themselves.  csa_index_scores_tree and csa_attend_tree take rotated rows.
 * Arguments
 *   rows      n <= 4 descriptors (host array), each one tensor of B x T tokens:
 *     x       `heads` rows of `dim` values per token, token (b, i) at
 *             x + (b T + i) x_stride (elements; 0: heads * dim, dense; else a
 *             multiple of 8 and at least heads * dim)
 *     out     [B, T, heads, dim] dense; may be x itself when x is dense, and must
 *             not overlap any tensor of the call otherwise
 *     weight  [dim] fp32 or NULL; norm: 0 or 1; dim a multiple of 8, R <= dim <=
 *             1024, (dim - R) a multiple of 8
 *   parent    [B, T] int32 or NULL; an unused slot's rows are left as they were
 *   pos [B]   (may be NULL without a rotation), inv_freq [R/2] fp32
 * Errors: CSA_ERR_ARG for sizes out of range (B, T, B*T <= 2^24, heads <= 4096,
 * T <= 64 with a parent array); CSA_DEV_STATE for pos[b] < 0, a position past
 * 2^31 - 1 or an inconsistent parent array (those tokens are skipped). */
typedef struct {
  const void* x;
  void* out;
  const float* weight;
  int heads, dim, norm;
  long long x_stride;
} csa_rows;
csa_status csa_norm_rope(const csa_layer* layer, const csa_rows* rows, int n, int B, int T, const int32_t* parent,
                         const int32_t* pos, const float* inv_freq, int32_t* err, void* stream);

/* csa_compress_tree, csa_index_scores_tree, csa_attend_tree, csa_commit_tree — a
 * speculative step that verifies a TREE of drafted tokens per sequence.
 *
 * The tree of sequence b is parent[b][0 .. T): parent -1 follows the last
 * committed token, 0 <= parent < i follows that node, and a value below -1 marks
 * an unused slot (sequences of a batch may have trees of different sizes; T <= 64,
 * B <= 65535, B*T <= 2^18).  Node i is a token at position p = pos[b] + depth(i), depth 0 for a child
 * of the last committed token.
 *
 * Definition: every node's row, scores and output are what sequential decoding
 * of its path (its ancestors from the root, then itself) would give
 * ([MTPLX#216] "Verification": the same results whether tokens arrive one by one
 * or in a block).  The cache is read only until csa_commit_tree; what the nodes
 * add is kept in draft buffers of the caller:
 *   kv     [B, T, D]       latent rows, normalised and rotated (csa_norm_rope)
 *   proj_a [B, T, 2*L*D]   projected kv | gate rows (csa_compress_tree)
 *   rows_a [B, T, D]       the compressed row that node i completes, (p + 1) mod
 *                          ratio == 0; the other nodes' entries are not touched
 *   proj_i, rows_i         the same for the index pool (rows of Di values, or of
 *                          CSA_FP8_ROW_BYTES with index_fp8)
 * An unused slot's entries and outputs are left as they were.  A parent that is
 * not below its node, or a used node under an unused one, raises CSA_DEV_STATE
 * and the nodes it concerns are skipped; so does a sequence with pos[b] < 0 or
 * above 2^31 - 65, or n_rows[b] != floor(pos[b] / ratio).  With two calls in flight on different
 * streams, workspaces and draft buffers must differ.
 *
 * csa_compress_tree: x [B, T, X] model dtype; the entries of a window before
 * pos[b] come from the frontier rings, the others from the path's nodes; the
 * stages and their roundings are csa_compress_append's.  The projections' fp32
 * sums may be split differently along the hidden axis there and here (and here by
 * B*T and the device): a projection may round to the neighbouring value, and the
 * row that it enters may differ by as much; otherwise a committed row is the row
 * csa_compress_append would have written.  One call's results do not change from
 * run to run.  comp_i and its buffers are NULL for the attention pool alone.
 * Workspace: CSA_OP_COMPRESS_TREE (cap ignored). */
csa_status csa_compress_tree(const csa_layer* layer, const csa_compressor* comp_a, const csa_compressor* comp_i,
                             const void* x, int B, int T, const int32_t* parent, const int32_t* pos,
                             const void* frontier_a, void* proj_a, void* rows_a, const void* frontier_i, void* proj_i,
                             void* rows_i, const float* inv_freq, void* ws, size_t ws_bytes, int32_t* err,
                             void* stream);

/* csa_index_scores_tree: the nodes' index scores, csa_index_topk's formula on
 * rotated queries iq [B, T, Hi, Di] (csa_norm_rope without a norm), iw [B, T, Hi]:
 *   scores [B, T, cap + T] fp32 (cap <= 2^31 - 257);
 *   columns c < n_rows[b]: committed row c;
 *   columns n_rows[b] + a, a < T: the row of node a for the nodes a of i's path
 *   that complete one, -infinity for the others; later columns are not touched.
 * ikeys [B, cap, Di], rows_i [B, T, Di]; with index_fp8 both are fp8 rows, and the
 * queries are brought into the same form (rotation, scale, codes) as in
 * csa_index_topk.  Requires ratio == 4.
 * Workspace: CSA_OP_INDEX_SCORES_TREE (cap ignored; 0 bytes, and ws may be NULL,
 * without index_fp8). */
csa_status csa_index_scores_tree(const csa_layer* layer, const void* iq, const void* iw, int B, int T,
                                 const int32_t* parent, const void* ikeys, int cap, const void* rows_i,
                                 const int32_t* n_rows, const int32_t* pos, float* scores, void* ws, size_t ws_bytes,
                                 int32_t* err, void* stream);

/* csa_attend_tree: selection and attention of every node (cap + T + W <= 2^31 - 257).
 *   visible columns: c < n_rows[b], and n_rows[b] + a for the completing nodes a
 *   of the path; the topk largest scores among them (ties to the lower column),
 *   all of them when there are no more or when scores is NULL (layers without an
 *   indexer, or every row wanted);
 *   keys = those rows (pool, or rows_a) ++ window tokens t in [p - W + 1, p]
 *   (window ring before pos[b], kv of the path's nodes from there);
 *   o = softmax with the sink as in csa_attend_decode, on rotated q;
 *   out = RoPE^-1(o, p), in fp32, rounded to the model dtype once.
 *   q [B, T, H, D], sink [H] fp32, scores [B, T, cap + T] or NULL,
 *   out [B, T, H, D], sel_out [B, T, topk] int32 or NULL: the selected columns,
 *   ascending, -1 padded (only with scores).
 * Workspace: CSA_OP_ATTEND_TREE. */
csa_status csa_attend_tree(const csa_layer* layer, const void* q, const void* kv, const float* sink, int B, int T,
                           const int32_t* parent, const void* window, const void* pool, int cap, const void* rows_a,
                           const float* scores, const int32_t* n_rows, const int32_t* pos, const float* inv_freq,
                           void* out, int32_t* sel_out, void* ws, size_t ws_bytes, int32_t* err, void* stream);

/* csa_commit_tree: leaf[b] (-1: nothing) is the last accepted node of sequence b;
 * its path becomes committed tokens: their kv rows enter the window ring, their
 * projections the frontier rings, the rows that they complete the pools, and
 * pos_out[b] = pos[b] + (path length), n_rows_out[b] = floor(pos_out[b] / ratio).
 * pos_out, n_rows_a_out, n_rows_i_out may be pos, n_rows_a, n_rows_i themselves.
 * A sequence whose leaf is no node, whose state is inconsistent (CSA_DEV_STATE) or
 * whose pool is too small (CSA_DEV_CAPACITY) is left unchanged (the outputs are
 * the inputs).  The index pool's arguments are NULL for the attention pool alone.
 * After it csa_trim rewinds as after decoding. */
csa_status csa_commit_tree(const csa_layer* layer, int B, int T, const int32_t* parent, const int32_t* leaf,
                           const int32_t* pos, int32_t* pos_out, const void* kv, void* window, const void* proj_a,
                           void* frontier_a, const void* rows_a, void* pool_a, int cap_a, const int32_t* n_rows_a,
                           int32_t* n_rows_a_out, const void* proj_i, void* frontier_i, const void* rows_i,
                           void* pool_i, int cap_i, const int32_t* n_rows_i, int32_t* n_rows_i_out, int32_t* err,
                           void* stream);

/* csa_add_norm — the hidden states that a layer takes: the residual's addition,
 * the RMS norm, and the norm once more in 8 bits, in one pass.
 *
 * Definition (per row of X values, in fp32):
 *   h = x + residual                                  (residual NULL: h = x)
 *   y = h * (mean(h^2) + rms_eps)^-1/2 * weight       (weight NULL: ones)
 *   residual_out = h, out = y, each rounded to the model dtype once;
 *   per group of `group` values of y: scale = max |y| / 448,
 *   codes = E4M3(y / scale) (nearest even, saturating; the quotient is a product
 *   with the scale's reciprocal, within two roundings), zeros where the scale is 0.
 * The norm is that of the fp32 sum, not of the rounded one.  A NaN makes its
 * group's scale NaN; codes and scales stand for code * scale.
 * Arguments
 *   x, residual     N rows of X model-dtype values, x_stride / residual_stride
 *                   elements apart (0: dense; else a multiple of 8, at least X)
 *   weight [X] fp32 or NULL
 *   out, residual_out [N, X] model dtype, dense; either may be NULL
 *   codes [N, X] bytes and scales [N, X / group] fp32, both or neither (group is
 *                   then ignored)
 *   group           8, 16, 32, 64, 128 or 256, dividing X; or X
 * An output may be x or residual itself where that is dense; apart from that no
 * output may overlap an input or another output (CSA_ERR_ARG, as are no output
 * at all, X not a multiple of 8 or above 16384, N < 0 or above 2^31 - 1).  N == 0
 * enqueues nothing.  One kernel on `stream`; it reads nothing before its
 * predecessors in the stream have completed, and the next kernel starts once it
 * has written, so its outputs may be any call's inputs. */
csa_status csa_add_norm(const csa_layer* layer, const void* x, long long x_stride, const void* residual,
                        long long residual_stride, const float* weight, long long N, int X, void* out,
                        void* residual_out, void* codes, float* scales, int group, void* stream);

/* csa_append_pages, csa_attend_pages — a layer's cache in pages and 8 bits.
 *
 * The pool of pages (csa_pages, caller-owned device memory) holds rows of D
 * values: codes [n_pages, page_rows, D] E4M3 and scales [n_pages, page_rows]
 * fp32, a row standing for scale * code.  table [B, width] int32 names, for
 * sequence b, the page of its logical rows [k page_rows, (k + 1) page_rows) in
 * table[b][k].  Pages of one pool may belong to tables of different kinds: a
 * token table (logical row t is token t's latent row) and a table of compressed
 * rows.  A page that nothing reads or writes any more (tokens behind the window)
 * may be handed out again, its entry be anything.
 * pos [B] int32: the position of each sequence's first query or new row of the
 * call; n_new [B] int32 or NULL (T each): how many of its T are there, 0 .. T.
 * What lies behind them is neither read for a result nor written.
 * At most 2^31 - 257 rows in a pool, 2^30 in a table; a table's entry outside
 * [0, n_pages) that a call meets raises CSA_DEV_RANGE, a row behind the table's
 * width CSA_DEV_CAPACITY, and the row is left out; pos[b] < 0 or above
 * 2^31 - 1 - T or n_new[b] outside [0, T] raises CSA_DEV_STATE and skips the sequence.
 * What a call writes (the pool or the output, workspace, error word) may overlap
 * neither what it reads nor what else it writes, pages of the pool that it does not
 * meet included (CSA_ERR_ARG).
 * Both calls read nothing before their predecessors in the stream have completed,
 * and the next kernel starts once they have written.
 *
 * csa_append_pages: rows [B, T, D] model dtype become the logical rows
 * pos[b] + i, i < n_new[b], of table's sequences.  Per row, in fp32:
 *   y = x * (mean(x^2) + rms_eps)^-1/2 * weight   (norm != 0; weight NULL: ones)
 *   y = RoPE(y, pos[b] + i)                       (inv_freq NULL: no rotation)
 *   scale = max |y| / 448, codes = E4M3(y / scale) (nearest even, saturating;
 *   zeros where the scale is 0, a NaN scale for a row with a NaN)
 * stride_b, stride_t: elements between sequences and tokens (0: dense; else
 * multiples of 8, tokens at least D apart).  B * T <= 2^24.  Two rows of one call
 * in one place (tables that share a page being written) leave a mixture of both. */
typedef struct {
  void* codes;
  float* scales;
  int n_pages, page_rows;
} csa_pages;
csa_status csa_append_pages(const csa_layer* layer, const csa_pages* pages, const void* rows, long long stride_b,
                            long long stride_t, int B, int T, const int32_t* table, int width, const int32_t* pos,
                            const int32_t* n_new, const float* weight, int norm, const float* inv_freq, int32_t* err,
                            void* stream);

/* csa_attend_pages: query i < n_new[b] of sequence b, at p = pos[b] + i, attends
 *   compressed rows: row_table's rows sel[b][i][0 .. n_sel[b][i]) (each index as
 *     often as it is listed; one outside [0, n_rows[b]) raises CSA_DEV_RANGE and
 *     is left out), or without sel all rows j < n_rows[b] with
 *     (j + 1) * ratio <= p + 1; none with row_table NULL;
 *   tokens: token_table's rows t in [p - W + 1, p] (layer->W) and t in
 *     [0, first), t >= 0, each once; none with token_table NULL;
 *   l_hk = scale * q[b][i][h] . key_k,  o_h = sum_k e^{l_hk} key_k / (e^{sink_h} + sum_k e^{l_hk})
 *   out[b][i][h] = RoPE^-1(o_h, p) in fp32, rounded to the model dtype once.
 * The cache holds the queries' own rows already (csa_append_pages).  q is rotated
 * (csa_norm_rope).  A query without any key gives zeros.
 *   q, out [B, T, H, D] model dtype, apart from one another; sink [H] fp32 or NULL (no sink);
 *   sel [B, T, topk], n_sel [B, T] int32 (ratio 4, with row_table); inv_freq NULL:
 *   no rotation of the output.
 * On the tensor cores (bf16, H = 64, D = 512, R = 64, page_rows a multiple of 8)
 * the queries enter the products as two E4M3 parts (the 8 bits of a bf16 value,
 * those 2^-13 below the head's largest fewer), the probabilities times the keys'
 * scales in fp16 and from that as an E5M2 and an E4M3 part, sums in fp32.  Such a
 * weight is off by at most 2^-8 of itself (and fp16's 2^-11), where that is more by
 * 2^-15 of the head's largest weight, at most 1/8 of itself; below 2^-20 of the
 * largest by 2^-22 of that.  Where small weights that are alike would all be rounded
 * to one side, and that comes to 2^-9 of the weights, they are rounded by turns: one
 * may then be off by 1/4 (or 2^-14 of the largest), many together by 2^-8.
 * The portable kernel takes any other layer, all in fp32, and is far slower: the
 * Flash shapes in pages of 13 rows take 79 us a selection and 900 us 128 of them,
 * in pages of 16 rows 15 and 25; 16 heads over the 512-dim latent take 92 us where
 * 64 take 22 (one query of 32K rows).  A call's result
 * depends on how its keys are cut into tiles (by B, T and all lengths), not on the
 * run: the same call gives the same bits.
 * B * T <= 2^16, and CSA_ERR_ARG where a sequence's tables have room for 2^31 - 256 keys, or B * T such for 2^36.
 * Workspace: CSA_OP_ATTEND_PAGES (parts of queries for 152 blocks: 40 MB for the
 * Flash shapes, whatever B and T), not shared by two calls in flight. */
csa_status csa_attend_pages(const csa_layer* layer, const csa_pages* pages, const void* q, int B, int T,
                            const float* sink, const int32_t* pos, const int32_t* n_new, const int32_t* token_table,
                            int token_width, int first, const int32_t* row_table, int row_width, const int32_t* n_rows,
                            const int32_t* sel, const int32_t* n_sel, const float* inv_freq, void* out, void* ws,
                            size_t ws_bytes, int32_t* err, void* stream);

/* csa_index_topk_static — csa_index_topk without a caller-supplied workspace.
 *
 * No counterpart in the paper: this is a calling convention, not a step of the
 * method.  Some callers cannot allocate device memory at the point where they
 * run the indexer: code running inside a region whose allocator is frozen (a
 * serving engine that reserves all device memory up front and hands out no
 * scratch, or a runtime that forbids cudaMalloc and its implicit device-wide
 * synchronisation on a latency-critical decode path), or a plain C caller with
 * no allocator of its own.  This entry point takes its scratch memory from a
 * file-scope device array of csa_static_scratch_bytes() bytes (4 MiB) inside
 * the library; it allocates and frees nothing.
 *   - Arguments, results and errors are those of csa_index_topk, without ws.
 *   - Returns CSA_ERR_WORKSPACE when the call needs more scratch than the array
 *     holds (csa_workspace_size(..., CSA_OP_INDEX_TOPK, B, 1, cap) bytes; about
 *     B * (Hi*Di*4 + cap*4) — e.g. 32 sequences with 8400-row pools fit).
 *   - The first call on each device looks up the array's device address (with
 *     that device current) and keeps it together with the id of the device's
 *     CUDA context; make that first call before any stream capture.  A call in
 *     a context other than the one the address was found in (the device was
 *     reset and its context created again) looks it up again, since the array
 *     may then sit elsewhere: that call too should come before any capture.
 *   - Every call on a device shares the one array: calls whose kernels overlap
 *     on the GPU (different streams without ordering) race on it.  Calls in one
 *     stream are ordered and safe.  Nothing in the array needs to start at zero;
 *     it keeps the last call's contents.
 *   - Every GPU that loads the library holds the array until the process exits. */
size_t csa_static_scratch_bytes(void);
csa_status csa_index_topk_static(const csa_layer* layer, const void* iq, const void* iw, int B, const void* ikeys,
                                 int cap, const int32_t* n_rows, const int32_t* pos, const float* inv_freq,
                                 int32_t* sel, int32_t* n_sel, int32_t* err, void* stream);

/* Advance the positions of B sequences by `by` tokens: pos[b] += by, in one kernel
 * on `stream` (a device array of B int32, caller-owned).  A decode loop calls it
 * after the step's last library call (csa_attend_decode), since every call of a
 * step reads pos; it is not part of the method ("Decode path": the position of
 * the next token), only the loop's bookkeeping, launched like the library's
 * other kernels so that it may start while the step's last kernel finishes.
 * Unlike them it lets the next kernel start only once it has written pos, so
 * the next step's calls may read pos before their programmatic wait.
 * Errors: CSA_ERR_ARG for a null pos, B < 0; CSA_ERR_CUDA if the launch fails.
 * B == 0 enqueues nothing. */
csa_status csa_advance_positions(int32_t* pos, int B, int by, void* stream);

/* csa_index_rows_fp8 — index-key rows in the model dtype to fp8 index rows.
 *
 * src: n rows of Di = 128 bf16 values (an index pool written with index_fp8 = 0,
 * or rows from elsewhere; device, 16-byte aligned, caller-owned, read only);
 * dst: n rows of CSA_FP8_ROW_BYTES bytes (device, 16-byte aligned, caller-owned,
 * written).  Each row becomes exactly the row csa_compress_append would store
 * for it in a layer with index_fp8 = 1 (rotation, scale, E4M3 codes, zero
 * padding; see CSA_FP8_ROW_BYTES), so a cache built in the model dtype can be
 * carried over to the fp8 format.  Not a step of the method: a format
 * conversion.  The layer must have index_fp8 = 1 (else CSA_ERR_UNSUPPORTED).
 * Errors: CSA_ERR_ARG for n < 0 or n > 2^34, a null or misaligned pointer;
 * CSA_ERR_CUDA if the launch fails.  n == 0 enqueues nothing.  One kernel on
 * `stream`; src and dst must not overlap. */
csa_status csa_index_rows_fp8(const csa_layer* layer, const void* src, long long n, void* dst, void* stream);

/* Number of kernels this library has enqueued in this process (all calls,
 * all devices).  Diagnostic only: lets a caller count the launches of a region. */
unsigned long long csa_kernel_launches(void);

/* Human-readable name of a status code. */
const char* csa_status_string(csa_status s);

#ifdef __cplusplus
}
#endif
#endif /* CSA_H */
