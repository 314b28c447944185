/*
 * dspark_target.h -- C ABI of the target's side of a decode cycle on MI355X (gfx950): the
 * paged cache that the scheduled rows are written to and read from, and the target's logits
 * in the form that dspark_verify reads.
 *
 *   dspark_schedule -> ell
 *   dspark_cache_plan          rows, pages and cache slots of this step, from ell on the device
 *   per layer: dspark_cache_append, dspark_tree_attention
 *   dspark_target_logits[_tree] penalties, biases, grammar masks; packed rows -> verify's layout
 *   dspark_verify_rows -> n_acc (-1 for requests that the plan gave no rows)
 *   dspark_cache_commit        accepted path moved, lengths advanced, finished requests' pages back
 *
 * The conventions are those of dspark.h: device pointers unless said otherwise, caller-owned
 * memory, all work enqueued on `stream`, negative returns for calls refused on the host,
 * faults in device data OR-ed into *dev_status (nullable) with every access kept in bounds.
 * No call synchronises or allocates; all may be captured in a graph.  Results do not depend
 * on the order in which workgroups run.  Workspaces are 16-byte aligned, need no preparation
 * and hold nothing between calls; calls that overlap need one each.
 *
 * Rows.  A step runs `rows` packed rows at most: request q owns rows row_off[q] ..
 * row_off[q+1]-1 (row_off [R+1], on the device); row i of a request is node i of its block:
 * node 0 the anchor (the last emitted token), nodes 1.. the drafted tokens.  Rows at and
 * behind row_off[R] belong to nobody and are never read or written.
 *
 * Cache.  Tokens live in pages of page_size tokens (a power of two, 8 .. 1024).  k_cache and
 * v_cache hold n_pages pages of Hkv heads of page_size rows of D elements (D contiguous);
 * page, head and token strides are in elements, so [page][head][token][D] and
 * [page][token][head][D] both serve.  Token t of request q is row t % page_size of page
 * table[q][t / page_size]; table is [R][max_pages] int32.  ctx[q] tokens of request q are
 * committed; the block's node i is token ctx[q] + i.  n_pages * page_size < 2^31 and
 * max_pages * page_size <= 2^30.  R <= 2^20 (dspark_target_logits: 65535).
 */
#ifndef DSPARK_TARGET_H
#define DSPARK_TARGET_H

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* further bits OR-ed into *dev_status (beside DSPARK_FAULT_TOKEN and DSPARK_FAULT_LEN) */
enum {
  DSPARK_FAULT_PAGE = 8,   /* no free page left, or a page or slot id out of range */
  DSPARK_FAULT_TREE = 16,  /* a parent or a path that is not a tree's */
  DSPARK_FAULT_PARAM = 32  /* a penalty or a mask index out of range */
};

/* nodes of a tree of drafted tokens, the anchor included (an ancestor mask has 64 bits, and
 * the anchor needs none) */
enum { DSPARK_MAX_TREE_NODES = 65 };

/* ------------------------------------------------------------------------------------
 * Step plan: block tables and slot maps from lengths on the device.
 *   n_q    = lens[q] + extra: the rows request q brings (extra = 1: lens is the scheduler's
 *            ell and the anchor comes on top; extra = 0: lens counts tokens, as for a prompt)
 *   need_q = max(0, ceil((ctx[q] + n_q) / page_size) - held[q]) pages, none if n_q = 0
 * Requests are served in index order: q gets its rows iff n_0 + .. + n_q <= rows and
 * need_q = 0 or need_0 + .. + need_q <= *n_free (sums over the requests before it that fit
 * in `rows`).  One that is not served gets none (row_off[q+1] = row_off[q]) and keeps what
 * it holds; DSPARK_FAULT_LEN (rows) or DSPARK_FAULT_PAGE (pages) says so.  Its target logits are
 * nobody's, so verification has to leave it out: dspark_verify_rows takes row_off for that.
 *   pages  the k-th page handed out is free_pages[*n_free - 1 - k] (a stack); in place:
 *          table[q][held[q] ..], held[q] += need_q, *n_free -= all of them.  Nothing else of
 *          table is written, and a call repeated for the same step changes nothing.
 *   row i of q: req = q, position = ctx[q] + depth(i), slot = page * page_size + offset of
 *          token ctx[q] + i, anc = bits j-1 of the nodes j >= 1 among i and its ancestors
 * parent [R][width] int32 (NULL: chains, depth(i) = i): parent[q][i] in [0, i) is the node
 * above node i >= 1 (parent[q][0] is not read); then n_q <= min(width, 65) and anc is
 * written (required); anc is ignored for chains.
 * Refused requests (no rows): ctx < 0, lens + extra < 0, ctx + n beyond max_pages pages, held
 * outside [0, max_pages], a tree too large (DSPARK_FAULT_LEN).  A parent out of range counts
 * as i - 1 (DSPARK_FAULT_TREE); a page id below 0 or whose slots pass 2^31 gives slot -1
 * (DSPARK_FAULT_PAGE); *n_free outside [0, free_len] is clamped (DSPARK_FAULT_PAGE).
 * Outputs: row_off [R+1]; req, position, slot [rows] int32 (req and position nullable);
 * anc [rows] uint64.  Rows at and behind row_off[R] are left as they were.
 * Workspace: ws_bytes >= dspark_cache_plan_workspace_bytes(R, rows, width), width 0 for
 * chains; where that is 0 (small steps), ws may be NULL.
 * ------------------------------------------------------------------------------------ */
size_t dspark_cache_plan_workspace_bytes(int R, int rows, int width);

int dspark_cache_plan(int R, int rows, int page_size, int max_pages, int free_len, int extra,
                      const int32_t *lens, const int32_t *ctx, int32_t *held, int32_t *table,
                      const int32_t *free_pages, int32_t *n_free, const int32_t *parent,
                      int width, int32_t *row_off, int32_t *req, int32_t *position,
                      int32_t *slot, uint64_t *anc, int32_t *dev_status, void *ws,
                      size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------------------
 * Cache append: row i's keys and values (Hkv heads of D contiguous elements, rows k_row and
 * v_row elements apart) into cache slot slot[i].
 * slot [rows] int32; slot -1 skips the row, any other value outside [0, n_pages *
 * page_size) skips it and sets DSPARK_FAULT_PAGE.  n_rows (device, nullable): only the first
 * *n_rows rows exist (pass row_off + R); no value of it reads past `rows`.  Slots of one
 * call are distinct; of rows with the same slot either's elements may remain.  k and v lie
 * outside the memory from the caches' first to their last element.
 * D % 8 == 0, D <= 1024; strides multiples of 16 bytes, pointers 16-byte aligned.
 * ------------------------------------------------------------------------------------ */
int dspark_cache_append(int rows, int Hkv, int D, dspark_dtype dt, int page_size, int n_pages,
                        const void *k, const void *v, int64_t k_row, int64_t v_row,
                        const int32_t *slot, const int32_t *n_rows, void *k_cache,
                        void *v_cache, int64_t page_stride, int64_t head_stride,
                        int64_t tok_stride, int32_t *dev_status, hipStream_t stream);

/* ------------------------------------------------------------------------------------
 * Attention of a step's rows over the paged cache (their own keys and values appended).
 * Query head a of Hq reads cache head a / (Hq / Hkv).  Row i of request q sees
 *   every token t < ctx[q], the anchor (t = ctx[q]), and node j >= 1 of its block (t =
 *   ctx[q] + j) iff j <= i (anc NULL: a chain, or a piece of a prompt of any length) or bit
 *   j-1 of anc[row] is set (a tree; j < n_q <= 65).
 *   o[row][a]   = sum_t softmax_t(scale * q[row][a] . K[t]) V[t],   scale > 0, scale log2(e) finite
 *   lse[row][a] = ln sum_t exp(scale * q . K[t])        (nullable, float)
 * Scores, maxima, sums and o are held in float; with bf16 operands the weights exp(s - max)
 * are rounded to bf16 for the product with V.  What lies in the cache at tokens that a row
 * does not see (stale, infinite or NaN) does not reach it.
 * q [rows][Hq][D] with rows q_row elements apart; o [rows][Hq][D] dense, apart from q.
 * D in {64, 128}; Hq a multiple of Hkv; rows * Hq <= 2^31 - 1024; dt as the cache's; strides
 * multiples of 16 bytes, pointers 16-byte aligned.  ctx + n beyond max_pages pages, ctx < 0 or
 * row_off out of order are clamped (DSPARK_FAULT_LEN); a page id outside [0, n_pages) reads page 0
 * (DSPARK_FAULT_PAGE); with anc, nodes past 64 are seen by nobody but through ctx
 * (DSPARK_FAULT_TREE).
 * Workspace: ws_bytes >= dspark_tree_attention_workspace_bytes(...) (0: sizes out of range).
 * ------------------------------------------------------------------------------------ */
size_t dspark_tree_attention_workspace_bytes(int R, int rows, int Hq, int Hkv, int D,
                                             dspark_dtype dt);

int dspark_tree_attention(int R, int rows, int Hq, int Hkv, int D, dspark_dtype dt,
                          int page_size, int max_pages, int n_pages, const void *q,
                          int64_t q_row, const void *k_cache, const void *v_cache,
                          int64_t page_stride, int64_t head_stride, int64_t tok_stride,
                          const int32_t *table, const int32_t *ctx, const int32_t *row_off,
                          const uint64_t *anc, float scale, void *o, float *lse,
                          int32_t *dev_status, void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------------------
 * Target logits: the rows of a step, with the request's penalties, biases and grammar masks,
 * in the layout dspark_verify reads.  Row j = 0..ell[q] of request q is the target's
 * distribution after the anchor and x_1 .. x_j; for every id v, in float and rounded once,
 *   l = logits[row][v]
 *   seen (v in hist[q][0 .. hist_len[q]) or among x_1 .. x_j): l = l > 0 ? l / rep : l * rep
 *   c = times v occurs in hist[q][prompt_len[q] .. hist_len[q]) and x_1 .. x_j
 *   l = l - freq * c - (c > 0 ? pres : 0) + bias of v
 *   v not allowed by the row's mask: l = -inf (whatever l was)
 *   out[q][j][v] = l;  rows j > ell[q] are left as they were
 * hist holds the request's tokens, prompt first, the anchor included.
 * Inputs: logits: row row_off[q] + j, rows `row_stride` elements apart (row_off NULL: row
 *   q * (gamma + 1) + j), `rows` rows in all; row_off [R+1]: request q has no row at or
 *   behind row_off[q+1]; ell [R]; x [R][gamma] int32;
 *   hist [R][hist_stride] int32, hist_len, prompt_len [R] (hist NULL: only drafted tokens
 *   count; prompt_len NULL: 0); rep, pres, freq [R] float (each nullable: 1, 0, 0);
 *   bias_id [R][nbias] int32 (-1: unused) and bias [R][nbias] float: of several entries for
 *   one id the last counts; mask [n_mask][mask_stride] uint32 (bit v % 32 of word v / 32
 *   set: allowed; mask_stride >= ceil(V / 32)), mask_idx [R][gamma+1] int32: the row's mask,
 *   -1 none (mask_idx NULL: mask q * (gamma + 1) + j).
 * out may be logits itself where row_off is NULL and row_stride is V, and overlaps it in no
 * other way.
 * A row whose mask allows nothing is all -inf (dspark_verify rejects the token drafted there,
 * emits -1 where it had to draw from that row, and sets DSPARK_FAULT_EMPTY).
 * Faults: ell outside [0, gamma] (DSPARK_FAULT_LEN, clamped); a row that is
 *   not the request's or outside [0, rows) (DSPARK_FAULT_LEN, its out row is left as it was:
 *   what becomes of requests that the plan gave no rows); hist_len outside [0, hist_stride],
 *   prompt_len outside [0, hist_len] (DSPARK_FAULT_LEN, clamped); a token or bias id outside
 *   [0, V) (DSPARK_FAULT_TOKEN, ignored); rep not finite or below FLT_MIN, pres or freq not finite
 *   (DSPARK_FAULT_PARAM: 1, 0, 0); a mask index outside [-1, n_mask) (DSPARK_FAULT_PARAM:
 *   no mask).
 * V % 8 == 0, V <= 2^30; logits (NULL where rows is 0), out and row_stride 16-byte aligned.
 * ------------------------------------------------------------------------------------ */
int dspark_target_logits(int R, int gamma, int V, dspark_dtype dt, const void *logits,
                         int64_t row_stride, int rows, const int32_t *row_off,
                         const int32_t *ell, const int32_t *x, const int32_t *hist,
                         int hist_stride, const int32_t *hist_len, const int32_t *prompt_len,
                         const float *rep, const float *pres, const float *freq,
                         const int32_t *bias_id, const float *bias, int nbias,
                         const uint32_t *mask, int n_mask, int mask_stride,
                         const int32_t *mask_idx, void *out, int32_t *dev_status,
                         hipStream_t stream);

/* The same for trees of drafted tokens, whose rows do not follow one another: row j of request q
 * is node j, x[q][j-1] its token, and anc [rows] uint64 (a plan's; row row_off[q] + j as logits
 * are; NULL: a chain, exactly dspark_target_logits) the nodes on the way to it.  Wherever
 * x_1 .. x_j stands above, it is the tokens x_i of the row's mask (bits i - 1) instead.  Bits of
 * nodes past gamma are ignored. */
int dspark_target_logits_tree(int R, int gamma, int V, dspark_dtype dt, const void *logits,
                              int64_t row_stride, int rows, const int32_t *row_off,
                              const int32_t *ell, const int32_t *x, const uint64_t *anc,
                              const int32_t *hist, int hist_stride, const int32_t *hist_len,
                              const int32_t *prompt_len, const float *rep, const float *pres,
                              const float *freq, const int32_t *bias_id, const float *bias,
                              int nbias, const uint32_t *mask, int n_mask, int mask_stride,
                              const int32_t *mask_idx, void *out, int32_t *dev_status,
                              hipStream_t stream);

/* ------------------------------------------------------------------------------------
 * dspark_verify (dspark.h) behind a step plan, which may give a request no rows.  row_off [R+1]
 * int32: the plan's (NULL: exactly dspark_verify).  A request with row_off[q+1] = row_off[q] was
 * not in the step: its target rows are not read, n_acc = -1 (which dspark_cache_commit takes to
 * leave it as it is), y all -1, c_star all NaN, and x_next[q] = x0[q], its anchor (x0 [R] int32,
 * needed with x_next; may be x_next itself).  One with fewer rows than ell + 1 counts as
 * scheduled for rows - 1 positions, with fewer than 0 as not in the step (both
 * DSPARK_FAULT_LEN).  Workspace: dspark_verify_workspace_bytes(R, gamma, V, r).
 * ------------------------------------------------------------------------------------ */
int dspark_verify_rows(int R, int gamma, int V, int r, dspark_dtype dt, const void *target,
                       const void *U, const void *W2t, const void *bias_rows,
                       dspark_dtype bias_dt, const int32_t *x, const float *lse,
                       const float *logit_x, const int32_t *ell, const int32_t *row_off,
                       const int32_t *x0, uint64_t seed, uint64_t cycle, int32_t *n_acc,
                       int32_t *y, float *c_star, int32_t *x_next, int32_t *dev_status, void *ws,
                       size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------------------
 * Commit after verification.
 *   path [R][gamma] int32 (NULL: chains, nothing moves): the accepted nodes of a tree in
 *     order, ascending; for i = 1..n_acc[q], in every one of `layers` caches (layer_stride
 *     elements apart), token ctx[q] + i takes the keys and values that token
 *     ctx[q] + path[q][i-1] had before the call
 *   ctx_out[q] = ctx[q] + n_acc[q] + 1 (the anchor and the accepted nodes; n_acc = -1, as
 *     dspark_verify_rows gives it: the request had no rows); ctx_out may be ctx, and overlaps no
 *     other argument, nor ctx in any other way
 *   done [R] int32 (nullable): a request with done != 0 gives its pages back:
 *     free_pages[*n_free ..] takes table[q][0 .. held[q]) in request order, *n_free grows,
 *     held[q] = ctx_out[q] = 0 (its tokens are not moved).  Every page held is given back, so
 *     no two requests hold the same one then
 * n_acc outside [-1, gamma] (gamma checked with a path only) or past the pages held is
 * clamped (DSPARK_FAULT_LEN); held outside [0, max_pages] counts as the nearer end
 * (DSPARK_FAULT_LEN); a path that does not ascend from 1 or passes the pages held, or n_acc
 * entries of it, is moved no further (DSPARK_FAULT_TREE); a page id outside [0, n_pages)
 * moves nothing (DSPARK_FAULT_PAGE); pages past free_len are dropped (DSPARK_FAULT_PAGE).
 * gamma <= 64.  D % 8 == 0, D <= 1024; the cache arguments are read only with a path.
 * Workspace: ws_bytes >= dspark_cache_commit_workspace_bytes(R, max_pages, moves_in_place),
 * the last nonzero with a path and ctx_out == ctx; where that is 0, ws may be NULL.
 * ------------------------------------------------------------------------------------ */
size_t dspark_cache_commit_workspace_bytes(int R, int max_pages, int moves_in_place);

int dspark_cache_commit(int R, int gamma, int page_size, int max_pages, int free_len,
                        const int32_t *n_acc, const int32_t *path, const int32_t *done,
                        const int32_t *ctx, int32_t *ctx_out, int32_t *held,
                        const int32_t *table, int32_t *free_pages, int32_t *n_free, int layers,
                        int Hkv, int D, dspark_dtype dt, int n_pages, void *k_cache,
                        void *v_cache, int64_t layer_stride, int64_t page_stride,
                        int64_t head_stride, int64_t tok_stride, int32_t *dev_status, void *ws,
                        size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif
