/*
 * moe_serve.h - C ABI of the serving operators around the expert layer on
 * MI355X (gfx950): attention over a paged key-value cache (one new token per
 * sequence, with or without prefixes that sequences share, or whole prompts), the
 * cache's own upkeep (append, with or without rotary positions, extend, fork,
 * free, compact), products with 4-bit weights, and the sampling of tokens.
 *
 * The cache.  Keys and values sit in pages of `page` consecutive positions:
 *   data     [layers][2][pages][kv_heads][page][head_dim]; index 0 of the
 *            second axis holds keys, 1 values; bf16, fp16 or e4m3
 *   tables   i32 [seqs][cols]  the page of positions [i page, (i + 1) page) of
 *            a sequence; -1 where there is none
 *   lengths  i32 [seqs]        positions of a sequence, the new ones among them
 *   refs     i32 [pages]       sequences that hold a page; 0: the page is free
 *   k_scale, v_scale  f32 [kv_heads]: an e4m3 code stands for code * scale
 *            (NULL: 1); not used with the 16-bit types
 *   flags    u32 [1]           sticky, see MOE_KV_FLAG_*
 * All of it is device memory that the caller owns; nothing is allocated, and
 * lengths and tables are read on the device only.
 *
 * Attention.  For a query row at position p of a sequence of n positions,
 *   out = sum_t softmax_t(scale q . k_t) v_t
 * over the visible t: t <= p, t < n and, with window > 0, t > p - window or
 * t < sinks.  Query head i reads key-value head i / (q_heads / kv_heads).
 * lse is the natural logarithm of the sum of exponentials.  A row that sees
 * nothing gives zeros and -inf.  Keys and values that a row does not see have
 * no part in it, whatever they hold (NaN and infinities among them).  An
 * infinite value that it sees makes its output that infinity, however small the
 * weight; NaN, or infinities of both signs, make it NaN.
 *
 * Precision.  Products of 16-bit values are exact in f32; scores, the running
 * maximum and sum and the outputs are held in f32; the output is rounded once.
 * The weights exp(s - max) enter the second product as a pair of 16-bit values
 * (decode) or as one 16-bit value (prompt: of the size of the output's own
 * rounding; together they are off by 0.0022 in bf16, where decode is by 0.0016).
 *
 * Contents out of range (a page number outside the pool, a length beyond the
 * table, a sequence number outside the cache) are never followed: positions
 * without a page, and those beyond cols * page, are not seen and not written (new
 * tokens stay at the positions that the length gives them; fork and extend cut
 * it), and unknown sequences are skipped.
 *
 * Calls only enqueue work on `stream`, which belongs to the current device,
 * and may be captured into a HIP graph.  Every call returns a moe_status.
 */
#ifndef MOE_SERVE_H
#define MOE_SERVE_H

#include "moe_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_E4M3 = 2, MOE_F32 = 3 /* logits only */ };

/* Sticky flags of a cache. */
enum {
    MOE_KV_FLAG_NO_PAGES = 1, /* fork or extend found too few free pages */
    MOE_KV_FLAG_NO_COLS = 2   /* extend: a sequence would outgrow its table row */
};

/* Supported: head_dim 64, 96, 128, 192 or 256; page a power of two from 16 to
 * 1024; seqs * cols * (page / 16) below 2^31; data 16-byte aligned. */
typedef struct {
    void *data;
    int32_t *tables, *lengths, *refs;
    const float *k_scale, *v_scale;
    uint32_t *flags;
    int32_t dtype; /* MOE_BF16, MOE_FP16 or MOE_E4M3 */
    int32_t layers, pages, kv_heads, page, head_dim, seqs, cols;
} moe_kv_cache;

moe_status moe_kv_validate(const moe_kv_cache *kv);

/* Writes k and v (dtype MOE_BF16 or MOE_FP16; the cache's own, or any of the
 * two into an e4m3 cache) of `tokens` new tokens into the pages of one layer.
 * Rows of a token are kv_heads * head_dim long, the heads head_stride elements
 * apart, tokens token_stride apart (both multiples of 8).  cu NULL: token i is
 * the last position of sequence i (a sequence of length 0 gets nothing).
 * Else cu is i32 [batch + 1] and tokens cu[b] .. cu[b + 1] - 1 are the last
 * positions of sequence b.  Into e4m3: code = e4m3(clamp(x / scale, -448,
 * 448)), to nearest even; NaN stays NaN.
 * A sequence that extend could not lengthen has no new positions: its tokens
 * would be written over its last ones, which in a full page may be those of the
 * sequences that share it.  The second form takes what extend granted, i32
 * [seqs] by sequence (NULL: as the first), and writes nothing for a sequence
 * that has more tokens in the call than it was granted positions. */
moe_status moe_kv_append(const moe_kv_cache *kv, int32_t layer, const void *k, const void *v,
                         int32_t dtype, int64_t token_stride, int64_t head_stride, int32_t tokens,
                         const int32_t *cu, int32_t batch, moe_stream_t stream);
moe_status moe_kv_append_granted(const moe_kv_cache *kv, int32_t layer, const void *k,
                                 const void *v, int32_t dtype, int64_t token_stride,
                                 int64_t head_stride, int32_t tokens, const int32_t *cu,
                                 int32_t batch, const int32_t *granted, moe_stream_t stream);

/* Rotary positions: of a head, dimensions first .. first + rot - 1 (both multiples of
 * 16) are turned, in pairs (2j, 2j + 1) of them (interleaved) or (j, j + rot / 2).
 * Pair j of a token at position p becomes, with t = turns[j] p turns,
 *   amplitude (x0 cos t - x1 sin t), amplitude (x1 cos t + x0 sin t).
 * turns: device memory, f64 [rot / 2], the pair's frequency over 2 pi, finite. */
typedef struct {
    const double *turns;
    int32_t first, rot, interleaved;
    float amplitude;
} moe_rotary;

/* As moe_kv_append_granted, with the keys, and the queries q beside them, turned by
 * the tokens' positions in their sequences: q [tokens][q_heads][head_dim] with
 * strides like k's, q_out the same without gaps (q itself where that has none; it
 * overlaps nothing else).  Positions times frequencies are formed in 64 bits, the rest
 * in f32, and what is turned is rounded once (an e4m3 key straight to its code).
 * Keys and values that append leaves out are left out here too; the queries of their
 * tokens are turned all the same.  Queries of a sequence without positions (length
 * 0) come back as they are, rows outside [cu[0], cu[batch]) are not written. */
moe_status moe_kv_append_rotated(const moe_kv_cache *kv, int32_t layer, const moe_rotary *rotary,
                                 const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                 int32_t q_heads, const void *k, const void *v, int32_t dtype,
                                 int64_t token_stride, int64_t head_stride, int32_t tokens,
                                 const int32_t *cu, int32_t batch, const int32_t *granted,
                                 void *q_out, moe_stream_t stream);

/* Gives back the pages of n distinct sequences: each of their pages loses one
 * reference, their rows become -1 and their lengths 0. */
moe_status moe_kv_free(const moe_kv_cache *kv, const int32_t *seqs, int32_t n, moe_stream_t stream);

/* Bytes of scratch that fork and extend (n sequences) and compact (n = 0) need. */
size_t moe_kv_scratch_size(const moe_kv_cache *kv, int32_t n);

/* Makes sequence children[i] a copy of parents[i], for n pairs; children are
 * distinct, hold nothing and are nobody's parent in the same call.  Full pages
 * are shared (one reference more); a last page that is not full is copied, in
 * every layer, into the lowest free page (in the order of the pairs); entries
 * that are not pages are taken over as they are.  Where no page is free the
 * child ends at its last full page, and the cache's flag MOE_KV_FLAG_NO_PAGES
 * is set. */
moe_status moe_kv_fork(const moe_kv_cache *kv, const int32_t *parents, const int32_t *children,
                       int32_t n, void *scratch, moe_stream_t stream);

/* Lengthens n distinct sequences by counts[i] >= 0 positions and gives them
 * the pages for it (the lowest free ones, in the order of the list; NULL seqs:
 * sequences 0 .. n - 1).  A sequence that pages or columns do not suffice for
 * keeps its length and takes no page, so that those after it may still get
 * theirs, and a flag is set.  The last page must not be shared.  The second form
 * also writes the positions that each of the sequences was given, counts[i] or
 * none, to granted[its number] (i32 [seqs], NULL: as the first; the others'
 * entries stay as they are). */
moe_status moe_kv_extend(const moe_kv_cache *kv, const int32_t *seqs, const int32_t *counts,
                         int32_t n, void *scratch, moe_stream_t stream);
moe_status moe_kv_extend_granted(const moe_kv_cache *kv, const int32_t *seqs,
                                 const int32_t *counts, int32_t n, int32_t *granted,
                                 void *scratch, moe_stream_t stream);

/* Moves the pages in use together: with m pages in use, the i-th free page
 * below m receives the i-th used page from m on, in every layer.  new_tables
 * [seqs][cols] and new_refs [pages] receive the tables and references that
 * then hold; they may be the cache's own. */
moe_status moe_kv_compact(const moe_kv_cache *kv, int32_t *new_tables, int32_t *new_refs,
                          void *scratch, moe_stream_t stream);

typedef struct {
    int32_t q_heads;  /* a multiple of kv_heads */
    int32_t batch;    /* most sequences of a call, at most the cache's */
    int32_t longest;  /* positions of the longest sequence a plan is made for;
                         longer ones are right, too, only split less finely */
    int32_t window;   /* 0: none */
    int32_t sinks;    /* first positions that stay visible beside a window */
    float scale;      /* of the scores, e.g. head_dim^-1/2 */
} moe_attn_config;

moe_status moe_attn_validate(const moe_kv_cache *kv, const moe_attn_config *cfg);

/* Bytes of workspace and of counters (both 16-byte aligned) of a decode call,
 * or of prompt calls with up to `tokens` new tokens (tokens = 0: decode).  Counters
 * are zero before the first call that uses them, and every call leaves them
 * zero; the workspace carries nothing from call to call.  Calls that may run
 * at the same time need their own of both; a call may be of several launches, so
 * threads that share them on one stream make their calls one after the other. */
moe_status moe_attn_workspace(const moe_kv_cache *kv, const moe_attn_config *cfg, int32_t tokens,
                              size_t *workspace, size_t *counters);

/* One new token for each of the sequences 0 .. batch - 1, whose keys and
 * values are in the cache already: q [batch][q_heads][head_dim] with strides,
 * out the same without gaps, lse f32 [batch][q_heads].  dtype of q and out:
 * that of a 16-bit cache, either beside an e4m3 cache. */
moe_status moe_attn_decode(const moe_kv_cache *kv, const moe_attn_config *cfg, int32_t layer,
                           const void *q, int32_t dtype, int64_t token_stride, int64_t head_stride,
                           int32_t batch, void *out, float *lse, void *workspace, uint32_t *counters,
                           moe_stream_t stream);

/* The new tokens of several sequences: rows cu[b] .. cu[b + 1] - 1 of q are
 * the last positions of sequence b, b < batch; cu does not decrease.  Rows
 * outside [cu[0], cu[batch]) are not written. */
moe_status moe_attn_prompt(const moe_kv_cache *kv, const moe_attn_config *cfg, int32_t layer,
                           const void *q, int32_t dtype, int64_t token_stride, int64_t head_stride,
                           int32_t tokens, const int32_t *cu, int32_t batch, void *out, float *lse,
                           void *workspace, uint32_t *counters, moe_stream_t stream);

/* Decode where groups of sequences share a prefix: its keys and values are read once
 * for a group instead of once for each sequence.  A plan says which: group g has
 * the members members[cu[g]] .. members[cu[g + 1] - 1], each of the sequences 0 ..
 * batch - 1 in one group at most, and positions 0 .. prefix[g] - 1 of all of them hold
 * the same keys and values (as after fork; the pages of the member that is longest
 * there are read, the first one of equal ones).  Lengths and tables are read when the
 * call runs, so a plan holds while the members share their prefix: they may grow, pages
 * may move, and a member may be freed (it then sees nothing), but not become another
 * sequence.
 * least: bytes of keys and values of one layer that reading prefixes once for each group has
 * to spare, counting of a prefix what a member sees at most (with a window its positions and
 * the sinks); with less, sequences are decoded one by one (below 0: 40 MB, about where
 * that was measured to take no longer; 0: prefixes are always read apart).
 * Host only: cu [groups + 1], members and prefix are host memory.  data NULL: only the
 * sizes; else it receives plan->ints integers, which the caller copies to the device and
 * puts the address of into plan->data. */
typedef struct {
    const int32_t *data;  /* device memory, 16-byte aligned */
    int64_t ints;         /* its size */
    int32_t batch, q_heads, kv_heads, head_dim;
    int32_t units;        /* workgroups that read prefixes */
    int32_t tiles;        /* rows of a group, 128 at a time */
    int32_t slots;        /* partial results per kv head */
    int32_t parts;        /* most of a prefix */
    int32_t members;
    int32_t window, sinks;
    int32_t tail;         /* most positions that a sequence has by itself */
} moe_attn_shared;
moe_status moe_attn_share(const moe_kv_cache *kv, const moe_attn_config *cfg, int32_t batch,
                          int32_t groups, const int32_t *cu, const int32_t *members,
                          const int32_t *prefix, int64_t least, moe_attn_shared *plan,
                          int32_t *data);
/* As moe_attn_workspace, of moe_attn_decode_shared. */
moe_status moe_attn_shared_workspace(const moe_kv_cache *kv, const moe_attn_config *cfg,
                                     const moe_attn_shared *plan, size_t *workspace,
                                     size_t *counters);
/* As moe_attn_decode, of plan->batch sequences; kv and cfg are those the plan was made for
 * (a cfg for shorter sequences, fewer of them or other heads or windows is refused). */
moe_status moe_attn_decode_shared(const moe_kv_cache *kv, const moe_attn_config *cfg,
                                  const moe_attn_shared *plan, int32_t layer, const void *q,
                                  int32_t dtype, int64_t token_stride, int64_t head_stride,
                                  void *out, float *lse, void *workspace, uint32_t *counters,
                                  moe_stream_t stream);

/* Draws a token from each row of logits x.  With weights w_i = exp((x_i - max) / T)
 * and tokens ordered by logit, the largest first, equal ones by index, a row keeps
 *   the first top_k tokens (0, or at least the vocabulary: all);
 *   of those the ones before which the weights' sum is below top_p times that of
 *   all of them (1 or more: all), but always the first;
 *   of those the ones with w_i >= min_p (0: all; more than 1 counts as 1);
 * and draws the first token in order of index at which the sum of kept weights
 * exceeds u times their sum.  logprob: the logarithm of the probability that it is
 * drawn, w_i over that sum.  T = 0 (below 2^-100, or NaN) takes the first largest logit,
 * logprob 0.  Logits of -inf and NaN are never drawn; a row of nothing else gives -1
 * and -inf.  With a logit of +inf only those have weight, 1 each.  u below 0 or NaN
 * counts as 0, which draws the first kept token, however small its weight; from 1 on the
 * last one is drawn.  Weights and their sums are in 64 bits (a weight that is zero there is
 * never drawn), and of tokens next to a border of top_p integers of 2^-44 of the largest
 * of them, whose sums have no order.
 * Each filter is a device array by row, or NULL: the value for all rows beside it. */
typedef struct {
    const float *temperature, *top_p, *min_p;
    const int32_t *top_k;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
} moe_sampling;

/* Bytes of workspace and of counters (both 16-byte aligned; see moe_attn_workspace) of
 * calls with up to `rows` rows. */
moe_status moe_sample_workspace(int32_t rows, int32_t vocab, size_t *workspace, size_t *counters);

/* x [rows][vocab] (dtype MOE_BF16, MOE_FP16 or MOE_F32) with rows row_stride elements
 * apart, at the type's own alignment; u f32 [rows]; token i32 [rows]; logprob f32 [rows].
 * vocab up to 2^19. */
moe_status moe_sample(const void *x, int32_t dtype, int64_t row_stride, int32_t rows, int32_t vocab,
                      const float *u, const moe_sampling *filters, int32_t *token, float *logprob,
                      void *workspace, uint32_t *counters, moe_stream_t stream);

/* y = x W^T with W[n][j] = (code[n][j] - zero[n][j / group]) * scale[n][j / group]:
 * codes u8 [n][k / 2] (column 2j in the low half of byte j), scales [n][k /
 * group] in x's type, zeros u8 [n][k / group] below 16, or NULL for 8; x
 * [tokens][k] of finite values (in bf16 of magnitudes up to 2^112: sums of (code +
 * 128) x over a group have to be finite, too) with rows x_stride apart (a multiple
 * of 8, at most 2^25), y [tokens][n].  group 32, 64 or 128; k a multiple of group; n
 * any; x and codes 16-byte aligned.  Integers times x are summed exactly as products in f32, the
 * scale is applied to each group's sum in f32, and y is rounded once. */
moe_status moe_w4_linear(const void *x, int64_t x_stride, int32_t dtype, const uint8_t *codes,
                         const void *scales, const uint8_t *zeros, int32_t tokens, int32_t k,
                         int32_t n, int32_t group, void *y, moe_stream_t stream);

/* The HIP error behind the calling thread's last MOE_ERR_HIP. */
int32_t moe_serve_last_hip_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_SERVE_H */
