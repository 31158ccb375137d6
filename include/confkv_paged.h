/*
 * confkv_paged.h -- C ABI of the paged-cache and beam-search operators.
 *
 * A paged cache keeps K and V of many sequences in pools of fixed-size pages;
 * a sequence's tokens lie in the pages that its row of a page table names, in
 * order.  The pools and the tables are the caller's.  The operators are the
 * steps of a decode loop around them: prompt chunks, single tokens and trees
 * of drafted tokens are appended (rotated by their positions on the way) and
 * attended in the same way, an accepted path is taken over with
 * confkv_paged_commit, tokens are weighed by the attention that they get and
 * evicted by it with confkv_paged_weigh and confkv_paged_evict, and beams are
 * selected from the logits with confkv_beam_select and reordered with
 * confkv_paged_fork.
 *
 * Conventions (those of confkv.h hold here too):
 *   - Tensor arguments are DEVICE pointers on the cache's GPU, owned by the
 *     caller, row-major in the stated layout, and only touched by work
 *     enqueued on `stream` during the call.  No output lies in an input or in
 *     the batch's tensors unless a function allows it.  Element types are fp16 or bf16
 *     bit patterns (CONFKV_FP16 / CONFKV_BF16) unless stated otherwise.
 *   - Calls return CONFKV_OK or a negative CONFKV_ERR_* code; argument errors
 *     are found on the host before any work is enqueued.  What only the GPU
 *     can see (a page number outside the pool, a length past the page table,
 *     a path that is none) is skipped there without any access out of range
 *     (what attend gives for such rows is said there) and latched as
 *     CONFKV_FLAG_* bits, which confkv_paged_status returns.
 *   - No call allocates device memory or, but for status, synchronises the
 *     host, so all but create, free and status can be captured in CUDA graphs.
 *   - A cache handle holds the attention's scratch, memory of the caller: the
 *     GPU work of successive confkv_paged_attend calls on one handle must be
 *     ordered (one stream, or streams ordered by events; the same for graphs
 *     that were captured from it).  Handles are cheap; concurrent streams take
 *     one each, with a scratch of its own, over the same pools.
 */
#ifndef CONFKV_PAGED_H_
#define CONFKV_PAGED_H_

#include <stddef.h>
#include <stdint.h>

#include "confkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CONFKV_FP16 0
#define CONFKV_BF16 1
#define CONFKV_FP32 2      /* logits of confkv_beam_select only */

/* further device-side flags (bit mask, beside CONFKV_FLAG_* of confkv.h) */
#define CONFKV_FLAG_BAD_PAGE 8     /* a page number outside the pool */
#define CONFKV_FLAG_BAD_INDEX 16   /* a negative length, a path or parent that is none */

typedef struct confkv_paged confkv_paged;

/*
 * confkv_paged_scratch -- bytes of device scratch that a handle on `device`
 * (negative: the current one) needs for this head_dim, 256-byte aligned; 0 for
 * a head_dim that is refused or where the device cannot be read.  The caller
 * zeroes its first CONFKV_PAGED_ZEROED bytes before the handle's first call;
 * every call leaves them ready for the next.
 */
#define CONFKV_PAGED_ZEROED 16384
size_t confkv_paged_scratch(int head_dim, int device);

/*
 * confkv_paged_create -- a handle on caller-owned pools
 *   k_pages, v_pages: [layers][num_pages][kv_heads][page_size][head_dim],
 *   contiguous, 128-byte aligned.
 *   heads % kv_heads == 0, heads / kv_heads <= 16, head_dim 64 or 128,
 *   page_size 16, 32, 64, 128 or 256, dtype CONFKV_FP16 or CONFKV_BF16;
 *   layers * num_pages * kv_heads * page_size < 2^31.
 *   device: CUDA device of the pools (negative: the current one).
 *   scratch: confkv_paged_scratch bytes there, not shared with other handles.
 * *out receives the handle (NULL on failure): CONFKV_ERR_INVALID_ARG,
 * CONFKV_ERR_CAPACITY (scratch too small), CONFKV_ERR_OOM (host memory) or
 * CONFKV_ERR_CUDA.
 */
int confkv_paged_create(int layers, int heads, int kv_heads, int head_dim, int num_pages,
                        int page_size, int dtype, int device, void* k_pages, void* v_pages,
                        void* scratch, size_t scratch_bytes, confkv_paged** out);

/* Releases the handle (NULL is a no-op); pools and scratch stay the caller's,
 * who keeps them until the handle's work is done. */
void confkv_paged_free(confkv_paged* kv);

/* Message of the last error of this handle (never NULL). */
const char* confkv_paged_last_error(const confkv_paged* kv);

/*
 * confkv_paged_status -- synchronise the device, return the CONFKV_FLAG_*
 * bits latched since the last call in *flags (may be NULL) and clear them:
 * CONFKV_ERR_DEVICE where any was set, else CONFKV_OK.  CONFKV_FLAG_TIMEOUT
 * (a wait inside an attend call gave up after 2 s) makes that call's output
 * void; the handle is usable again after this call.
 */
int confkv_paged_status(confkv_paged* kv, int32_t* flags);

/*
 * The ragged batch that append and attend work on: rows q_start[b] ..
 * q_start[b+1] - 1 of the row tensors are sequence b's new tokens (none where
 * the two are equal); new token i of sequence b lies at place ctx_len[b] + i
 * of its sequence.  Rows before q_start[0] and from q_start[batch] on belong
 * to no sequence: nothing is computed for them and their outputs are left as
 * they were.
 */
typedef struct confkv_paged_batch {
  int32_t batch;               /* sequences B, 1 .. 65536 */
  int32_t max_blocks;          /* entries of a page-table row (a bound on the
                                  lengths: attend shares few rows' work among
                                  CTAs by it, so a row no wider than needed
                                  makes short calls faster) */
  const int32_t* page_table;   /* [B][max_blocks]; entries past a sequence's
                                  last page are not read */
  const int32_t* ctx_len;      /* [B] tokens cached before the new ones (0 allowed) */
  const int32_t* q_start;      /* [B + 1], not decreasing */
  const uint32_t* mask;        /* attend: [rows][mask_words] or NULL.  Bit j
                                  of row i: row i sees new token j of its own
                                  sequence (set its own bit too).  NULL: new
                                  token i sees new tokens 0 .. i.  Cached
                                  tokens are seen by every row. */
  int32_t mask_words;          /* words per row; new tokens from 32 * mask_words
                                  on are seen by no row */
} confkv_paged_batch;

/*
 * confkv_paged_append -- stores the new rows' K and V in layer `layer`'s
 * pages, K rotated by its position on the way, and rotates Q.
 *   k, v: [rows][kv_heads][head_dim], rows k_stride / v_stride elements apart
 *   q:    [rows][heads][head_dim] and q_out of that shape (both or neither;
 *         q_out may be q itself), rows q_stride / q_out_stride elements apart
 *   positions: [rows] the rows' positions in their text, or NULL: a row's place
 *         in its sequence (a tree's drafted tokens lie in other places than
 *         their depth).
 *   inv_freq: fp32 [rotary_dim / 2], or NULL (rotary_dim 0): nothing is
 *         rotated.  Channel pair i of the first rotary_dim channels turns by
 *         positions * inv_freq[i]: (a, b) -> (a cos - b sin, b cos + a sin),
 *         with a, b = channels i and i + rotary_dim / 2, or 2 i and 2 i + 1
 *         where interleaved is 1.  rotary_dim % 16 == 0, <= head_dim.
 * Pointers 16-byte aligned, strides multiples of 8.  The angle is reduced in
 * 64-bit fixed point, so far positions lose nothing; the rotation is fp32,
 * rounded once.  A row finds its sequence by reading q_start: work in rows x batch
 * / 32 words, which shows from some thousands of sequences on.
 */
int confkv_paged_append(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows,
                        const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                        const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                        const int32_t* positions, const float* inv_freq, int rotary_dim,
                        int interleaved, void* stream);

/*
 * confkv_paged_append_normed -- the same with each head of q and k normed before
 * it is rotated, y_c = x_c w_c / sqrt(sum_c x_c^2 / head_dim + eps), and with
 * several positions per row (an image's patch has a time, a height and a width).
 * Norm, rotation and what lies between are fp32; q_out and K are rounded once.
 */
typedef struct confkv_paged_norm {
  const void* q_norm;          /* [head_dim] weights of q's heads, or NULL: not normed */
  const void* k_norm;          /* [head_dim] weights of k's heads, or NULL */
  int32_t norm_dtype;          /* of both: CONFKV_FP32 or the cache's type */
  float eps;                   /* 1e-12 or more */
  const int32_t* axis;         /* [rotary_dim / 2] or NULL.  With it positions is
                                  [rows][axes], and channel pair i turns by
                                  positions[row][axis[i]] * inv_freq[i]; a pair
                                  whose axis is none is not turned
                                  (CONFKV_FLAG_BAD_INDEX). */
  int32_t axes;                /* 1 .. 8 */
} confkv_paged_norm;
int confkv_paged_append_normed(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                               const int32_t* positions, const float* inv_freq, int rotary_dim,
                               int interleaved, const confkv_paged_norm* norm, void* stream);

/*
 * confkv_paged_attend -- attention of the new rows over their sequences'
 * cached tokens and the new tokens that the batch's mask lets them see (whose
 * K and V append has stored): out = softmax(scale q k) v.
 *   q:   [rows][heads][head_dim], rows q_stride elements apart
 *   out: [rows][heads][head_dim] contiguous, of the cache's type
 *   lse: fp32 [rows][heads] ln sum exp(scale q k), or NULL
 *   scale: 0 means 1 / sqrt(head_dim); else positive
 * A row that sees nothing (no cached token and an empty mask) gives 0 and
 * lse -inf; one whose query or a key that it sees is NaN gives NaN in both.
 * What masked places and places past a sequence's end hold (NaN,
 * infinities) does not matter.  A sequence that is longer than its page table
 * ends where the table does (CONFKV_FLAG_CAPACITY); a row that sees a token of a
 * page outside the pool gives NaN in both (CONFKV_FLAG_BAD_PAGE).  Results do not
 * depend on what else is in the batch's other calls, and are the same on every
 * run.
 * Scores, their maxima and sums, and the outputs' sums are 32-bit; the weights
 * exp(score - max) are rounded once to the cache's type before they meet v, the
 * outputs once (relative errors 2^-11 each for fp16, 2^-8 for bf16).
 * One kernel takes the whole batch, chosen by its average of new rows: prompts'
 * chunks beside many single tokens can take up to 1.6 times what a call for each
 * takes.
 */
int confkv_paged_attend(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows,
                        const void* q, int64_t q_stride, void* out, float* lse, float scale,
                        void* stream);

/*
 * confkv_paged_attend_shared -- the same where groups of neighbouring sequences
 * share a prefix (the beams of a prompt, requests behind one instruction), which is
 * read once for a group.  Sequences group_start[g] .. group_start[g + 1] - 1 are
 * group g; their first prefix_len[g] cached tokens are the same in each and are
 * taken from the pages of the first one (whose table the others' need not
 * repeat; the prefix's last, less than 128 tokens each sequence reads from its own
 * pages, so those must be there).  Sequences in no group are taken as attend takes
 * them.  Any page_size and prefix length (0 too).
 * A sequence with fewer cached tokens than the whole steps of 128 of its group's
 * prefix is left out: its rows stay as they were (CONFKV_FLAG_BAD_INDEX); that flag
 * too for starts that fall or leave 0 .. batch and for negative lengths.
 * Every row's result is joined from two parts, in fp32, the prefix's first: within
 * attend's precision, but not the same bits.  Two launches in a row: faster than attend on
 * the same tables where the prefixes' K and V, counted for every sequence, are more than
 * L2 holds (some 130 MB) and rows are few; slower below that.
 */
typedef struct confkv_paged_prefix {
  int32_t groups;              /* 1 .. batch */
  const int32_t* group_start;  /* [groups + 1] sequences, not decreasing */
  const int32_t* prefix_len;   /* [groups] */
  void* partial;               /* scratch, 16-byte aligned, written and read by
                                  each call: calls that share it must be ordered */
  size_t partial_bytes;        /* confkv_paged_partial of the rows or more */
} confkv_paged_prefix;
size_t confkv_paged_partial(int rows, int heads, int head_dim);    /* 0 for sizes that are refused */
int confkv_paged_attend_shared(confkv_paged* kv, const confkv_paged_batch* batch,
                               const confkv_paged_prefix* prefix, int layer, int rows, const void* q,
                               int64_t q_stride, void* out, float* lse, float scale, void* stream);

/*
 * confkv_paged_weigh -- adds the new rows' attention weights to the accumulated
 * weight of each token that they see: for KV head h of sequence b
 *   mass_out[b][h][t] = decay mass[b][h][t] + gain sum exp(scale q k_t - lse)
 * over b's new rows and h's query heads, for every cached token t; new tokens
 * (places ctx_len[b] on) start from 0.  Rows see what they see in attend (causal,
 * or by the batch's mask); k is read from layer `layer`'s pages.
 *   q, lse: what attend was given and gave (a row with lse -inf adds nothing)
 *   mass, mass_out: fp32 [batch][kv_heads][cap] (mass_out may be mass itself)
 *   pos: int32 [batch][kv_heads][cap] or NULL: receives the new tokens' positions
 *        (`positions` [rows], or NULL: their places)
 *   scale: 0 means 1 / sqrt(head_dim)
 * gain 1, decay 1 add the weights up; gain (1 - decay) / (heads / kv_heads) makes
 * the running mean over the group's heads (confkv_step's is over all heads, and it ranks
 * by more than that).  Sums are fp32, in one order.  Nothing is written for sequences without new rows and
 * for places from ctx_len + new tokens on: a mass_out of its own holds what it held there
 * (a cache that goes on from step to step is weighed in place).  Places from cap on are
 * dropped (CONFKV_FLAG_CAPACITY).  Every sequence's k is read through its own table from its
 * first token on, behind a shared prefix too: a page outside the pool, which
 * attend_shared would not look at, makes its tokens' masses NaN (CONFKV_FLAG_BAD_PAGE).
 * commit and fork move no masses.  A drafted tree is weighed behind commit, by the
 * accepted path's rows of q and lse alone (its rows see one another in order, so
 * without the mask; ctx_len as it was before): weighed before, its drafts' masses would
 * stay at the drafts' places and rejected ones' weight on the cached tokens.  Behind fork
 * the caller gathers mass and pos by parent as it does its own states.  A NaN in a row that sees a token or in the token's k makes its
 * mass NaN.
 */
int confkv_paged_weigh(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows, const void* q,
                       int64_t q_stride, const float* lse, const float* mass, float* mass_out, int32_t* pos,
                       int cap, const int32_t* positions, float decay, float gain, float scale, void* stream);

/*
 * confkv_paged_evict -- every KV head of every sequence and layer keeps N =
 * min(length[b], keep[b]) of its cached tokens: its places below first[b] (a
 * prefix that others share, the first tokens of a text) before the tokens of the
 * `protect` newest positions (above the head's largest position - protect) before
 * those of the larger mass; equal ones by the lower place, NaN last.  The kept tokens
 * from place N on take the places of evicted ones below N, the r-th of them the
 * r-th such place, with K, V, mass and position; the other kept ones stay.
 *   length, keep, new_len: int32 [batch], or with per_layer 1 [layers][batch];
 *         new_len = N, not length itself.  keep can be confkv_confidence_noalloc's
 *         budget.
 *   mass, mass_out: fp32 [layers][batch][kv_heads][cap], pos, pos_out: int32
 *         likewise; the outputs are both the inputs themselves, or neither, and then
 *         places from N on are not written.  cap <= 524288.
 *   first: int32 [batch] or NULL (0)
 * Heads and layers keep different tokens: a place means another token in each.
 * The pages of places that change (those of places first[b] .. N - 1) belong to one
 * sequence each: where sequences share a prefix's pages, first[b] is the tokens in
 * them or more (which pages are shared is not looked at).  A sequence with a negative length, budget or first, or longer than
 * its table or cap, stays as it is, with its length (a flag; outputs of their own
 * receive its places, up to cap); a token whose page or whose new place's page is
 * outside the pool is not moved (CONFKV_FLAG_BAD_PAGE).
 */
int confkv_paged_evict(confkv_paged* kv, int batch, int max_blocks, const int32_t* page_table,
                       const int32_t* length, int per_layer, const float* mass, const int32_t* pos, int cap,
                       const int32_t* keep, const int32_t* first, int protect, float* mass_out,
                       int32_t* pos_out, int32_t* new_len, void* stream);

/*
 * confkv_paged_commit -- keeps an accepted path of drafted tokens: in every
 * layer, drafted token path[b][j] of sequence b (place ctx_len[b] + path[b][j])
 * moves to place ctx_len[b] + j, for j < path_len[b]; new_len[b] = ctx_len[b]
 * + path_len[b].
 *   path: [B][path_cap], rising (path[b][0] < path[b][1] < ...), path_cap
 *   <= 1024; path_len: [B]; new_len: [B], not ctx_len itself.
 * A sequence whose path is no such path stays as it is, with new_len = ctx_len
 * and a flag.  The pages of the drafted tokens belong to one sequence each.  Masses and
 * positions of confkv_paged_weigh do not move: weigh the accepted rows afterwards.
 */
int confkv_paged_commit(confkv_paged* kv, int batch, int max_blocks, const int32_t* page_table,
                        const int32_t* ctx_len, const int32_t* path, int path_cap,
                        const int32_t* path_len, int32_t* new_len, void* stream);

/*
 * confkv_paged_fork -- reorders beams: row r of `rows` = batch x beams takes
 * over the sequence of row p = (r / beams) * beams + parent[r].
 *   table_out[r]: p's full pages, shared, and, where its length is no multiple
 *   of page_size, tail_pages[r] as the last entry; entries behind are left as
 *   they were.  The filled slots of p's last page are copied to tail_pages[r]
 *   in every layer.  len_out[r] = len_in[p].
 *   parent: [rows] in 0 .. beams - 1; -1 (a selection without a candidate)
 *   takes row r's own.
 * tail_pages are pages that no row of this call reads (free, or of an earlier
 * step), all different, except that tail_pages[r] may be p's own last page if
 * no other row takes it.  table_out and len_out are not table_in and len_in.
 * Masses and positions of confkv_paged_weigh are gathered by the caller.
 */
int confkv_paged_fork(confkv_paged* kv, int rows, int beams, int max_blocks, const int32_t* parent,
                      const int32_t* table_in, const int32_t* len_in, const int32_t* tail_pages,
                      int32_t* table_out, int32_t* len_out, void* stream);

/*
 * confkv_beam_workspace -- bytes of device scratch for confkv_beam_select (0
 * for sizes that it refuses).  The caller zeroes it once; every call leaves
 * it ready for the next, whatever sizes both have.  Calls that share it must be
 * ordered, and it must be large enough for each.
 */
size_t confkv_beam_workspace(int batch, int beams, int vocab, int keep, int dtype);

/*
 * confkv_beam_select -- the `keep` best continuations of each sequence:
 * candidate (w, v) has the score scores[b][w] + logits[b][w][v] - ln sum_u
 * exp logits[b][w][u].
 *   logits: [batch][beams][vocab] of `dtype` (CONFKV_FP16, BF16, FP32), rows
 *           row_stride elements apart
 *   scores: fp32 [batch][beams]; -inf: a beam without candidates
 *   finished: uint8 [batch][beams] or NULL; a finished beam has one candidate,
 *           pad_token, at the beam's own score (its logits are not read)
 *   score_out fp32, parent_out, token_out int32 [batch][keep], best first,
 *           equal scores by the lower (w, v); where fewer candidates have a
 *           finite score the rest are (-inf, -1, -1).  Sums are 32-bit within a
 *           thread and exact beyond: ln sum exp is good to 4e-8 as measured (2^-18
 *           at worst for 2^18 tokens), and candidates of different beams that are
 *           nearer may change places.
 *   flags_out: int32 [batch][beams] or NULL: CONFKV_FLAG_NONFINITE where a row
 *           with a NaN or +inf logit, without a finite one, or with a NaN or
 *           +inf score was left out, else 0.
 *   device: CUDA device of the tensors and the workspace (negative: the
 *   current one).
 * beams <= 32, keep <= 64, 2 <= vocab <= 2^24, batch x beams <= 65535,
 * pad_token in 0 .. vocab - 1.
 */
int confkv_beam_select(const void* logits, int dtype, int64_t row_stride, int batch, int beams,
                       int vocab, int keep, const float* scores, const uint8_t* finished,
                       int pad_token, float* score_out, int32_t* parent_out, int32_t* token_out,
                       int32_t* flags_out, void* workspace, size_t workspace_bytes, int device,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONFKV_PAGED_H_ */
