/*
 * spec_serve.h -- C ABI of the operators around the verification step: what a serving loop
 * runs between the drafts and spec_verify_* (see spec_verify.h for the verification itself
 * and for the conventions on pointers, strides, int32 arrays, streams, workspaces and error
 * codes, which hold here too).
 *
 *   spec_logit_adjust   penalties, biases and grammar masks on the verified rows' logits
 *   spec_kv_append      the new tokens' keys and values into a paged cache held in 4 bits
 *   spec_kv_attention   the new tokens' attention (chain or tree) over that cache
 *   spec_kv8_append, spec_kv8_read, spec_kv8_attention
 *                       the same over a paged cache held in 8 bits, and its tokens back in 16 bits
 *
 * Arrays may be read and written by the kernels in any order: outputs must not overlap
 * inputs except where an entry says so.
 */
#ifndef SPEC_SERVE_H
#define SPEC_SERVE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of keys, values, queries and attention outputs. */
typedef enum { SV_KV_BF16 = 1, SV_KV_FP16 = 2 } sv_kv_dtype;

#define SV_MAX_BIAS 4096    /* entries of a sequence's bias list */
#define SV_MAX_HISTORY (1 << 30)

/*
 * Adjusts the logits that the verification entries take.
 *
 *   logits   [B][rows][V]  fp32 or bf16; strides as in spec_verify.h.
 *   out      [B][rows][V]  the same type, strides of its own (not 0 where there is more than one
 *            row or sequence).  May be `logits` itself with the same strides: then only the
 *            16-byte groups that change are written.
 *   history  [B][history_stride]  each sequence's tokens so far, lengths[b] of them valid, the
 *            first prompt_lengths[b] of them the prompt (both clamped to the row; NULL
 *            prompt_lengths: none).  NULL: no history.  Tokens outside [0, V) count nowhere.
 *   draft_tokens, parent   what the rows' contexts hold beyond the history:
 *            parent NULL   a chain, draft_tokens [B][rows - 1]: row i follows draft i - 1, its
 *                          context holds drafts 0 .. i - 1 (NULL: no drafts are counted);
 *            parent [rows] a tree (parent[0] = -1, 0 <= parent[v] < v; one tree for the batch),
 *                          draft_tokens [B][rows]: row v's context holds the nodes on the path
 *                          from the root's child to v.  The root is the history's last token
 *                          and is not counted again.  A parent outside [0, v) ends the path.
 *   repetition, frequency, presence   [B] fp32, NULL: off (1, 0, 0).  repetition > 0.
 *   bias_tokens, bias_values  [B][nbias], nbias <= SV_MAX_BIAS.  Entries with a token outside
 *            [0, V) are unused; of several entries for one token the last counts.
 *   allowed  [B][rows][ceil(V / 32)] words, bit t % 32 of word t / 32 set: token t is allowed.
 *            NULL: all are.
 * For the token t of row i, with l its logit, n its occurrences in the output part of the row's
 * context (history behind the prompt, and drafts) and s whether it occurs in the context at all:
 *   l := s ? (l > 0 ? l / repetition : l * repetition) : l
 *   l := l - frequency * n - presence * (n > 0)
 *   l := l + bias(t)
 *   l := allowed(t) ? l : -inf      (whatever l was, NaN and +inf too)
 * in fp32, rounded once to the output's type.  A row whose mask leaves nothing is all -inf; the
 * verification entries report such a sequence as bad data.
 */
sv_status spec_logit_adjust(const void *logits, int64_t batch_stride, int64_t row_stride, void *out,
                            int64_t out_batch_stride, int64_t out_row_stride, sv_dtype dtype, int B, int rows,
                            int V, const int32_t *history, int64_t history_stride, const int32_t *lengths,
                            const int32_t *prompt_lengths, const int32_t *draft_tokens, const int32_t *parent,
                            const float *repetition, const float *frequency, const float *presence,
                            const int32_t *bias_tokens, const float *bias_values, int nbias,
                            const int32_t *allowed, void *stream);

/*
 * The paged cache held in 4 bits.
 *
 *   cache       [num_pages][kv_heads][spec_kv_page_bytes(page_size, head_dim)] bytes, 16-byte
 *               aligned.  head_dim 64, 128 or 256; page_size a multiple of 16 up to 1024.  A
 *               page and head holds, for its page_size tokens: the keys' codes
 *               (page_size * head_dim / 2 bytes), the values' codes (as many), then two fp16
 *               words (scale, zero) per token for the keys, and for the values.  Nothing in it
 *               needs initialising: only slots below a sequence's length are ever used.
 *   page_table  [B][table_width]  token j of sequence b is in page page_table[b][j / page_size],
 *               slot j % page_size.  Entries past a sequence's length are not used.  A page
 *               outside [0, num_pages) is never touched: appended tokens are dropped, and its
 *               tokens are masked in the attention.  A table spans at most 2^31 - 128 tokens
 *               (2^31 - 1 for the append).
 *   start       [B]  tokens of each sequence in the cache before this step; its new tokens are
 *               start .. start + new_lens[b] - 1 (NULL new_lens: all T).  start is clamped to
 *               [0, table_width * page_size], new_lens to [0, T]; tokens past the table's end
 *               are dropped.
 * One head's vector x of a token (the rotated key, or the value) is held as
 *   zero = fp16(min x), scale = max(fp16((max x - min x) / 15), 2^-24), both at most 65504,
 *   code_d = round((x_d - zero) / scale) clamped to 0 .. 15, standing for zero + scale code_d,
 * rounding to nearest even, of the exact values (fp16(y): y rounded to fp32, then to fp16; the kernel
 * settles what 32 bits leave in doubt in 64).  A zero of -0 is held as +0.  A vector with a NaN or an infinity is held as NaN throughout.
 *
 * Rotation (cos, sin NULL: none): cos and sin are [table_len][pairs] fp32, pairs <= head_dim / 2;
 * pair i is dimensions (i, i + pairs), or (2 i, 2 i + 1) if interleaved; it becomes
 * (a cos - b sin, b cos + a sin) with the angles of the token's position: positions[b][t], or
 * start[b] + t if positions is NULL, clamped to the table.  Dimensions from 2 pairs on stay.
 */
size_t spec_kv_page_bytes(int page_size, int head_dim);

/*
 * Appends T new tokens per sequence.
 *   k, v       [B][T][kv_heads][head_dim] bf16 or fp16 (sv_kv_dtype), strides in elements for
 *              the first three axes, contiguous last axis.
 *   k_values, v_values   [B][T][kv_heads][head_dim] contiguous, of the inputs' type, NULL: not
 *              wanted: what the cache holds for the new tokens, as an attention over them in
 *              16 bits would read it; 0 for tokens from new_lens[b] on.  A token that is dropped
 *              (past the table, or its page out of range) gets what it would have been held as.
 * Two sequences must not append to the same slot.  No workspace.
 */
sv_status spec_kv_append(const void *k, int64_t k_batch_stride, int64_t k_token_stride, int64_t k_head_stride,
                         const void *v, int64_t v_batch_stride, int64_t v_token_stride, int64_t v_head_stride,
                         sv_kv_dtype dtype, int B, int T, int kv_heads, int head_dim, void *cache, int num_pages,
                         int page_size, const int32_t *page_table, int table_width, const int32_t *start,
                         const int32_t *new_lens, const float *cos, const float *sin, int table_len, int pairs,
                         int interleaved, const int32_t *positions, void *k_values, void *v_values, void *stream);

/*
 * Attention of the T new tokens over the cache, which holds them already.
 *   q, out     [B][T][heads][head_dim] bf16 or fp16, strides in elements for q's first three axes;
 *              out contiguous.  heads a multiple of kv_heads: head h reads kv head
 *              h / (heads / kv_heads).  q is rotated as spec_kv_append rotates keys.
 *   parent     NULL: a chain, token t sees the tokens before `start` and new tokens 0 .. t;
 *              [T], T <= SV_MAX_TREE_NODES: a tree (parent[0] = -1, 0 <= parent[v] < v, one for
 *              the batch), token t sees the tokens before `start`, its ancestors and itself.  A
 *              parent outside [0, v) ends the path.
 *   scale      finite; the scores are scale * (q . k).
 * out = softmax(scores over the tokens seen) . values; 0 for a token that sees none, and for
 * tokens from new_lens[b] on.
 * workspace  spec_kv_attention_workspace_size(...) bytes, 16-byte aligned, any contents.  Its first
 *            int32 is the call's status once the stream has completed: SV_OK, or SV_ERR_TIMEOUT if
 *            a bounded device wait (one second) gave up; `out` is then NaN throughout.
 */
size_t spec_kv_attention_workspace_size(int B, int T, int heads, int kv_heads, int head_dim);
sv_status spec_kv_attention(const void *q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
                            sv_kv_dtype dtype, int B, int T, int heads, int kv_heads, int head_dim,
                            const void *cache, int num_pages, int page_size, const int32_t *page_table,
                            int table_width, const int32_t *start, const int32_t *new_lens, const int32_t *parent,
                            float scale, const float *cos, const float *sin, int table_len, int pairs,
                            int interleaved, const int32_t *positions, void *out, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * The paged cache held in 8 bits: floats of 8 bits with a scale for each block of 16 slots and head.  Pages, page tables,
 * start, new_lens, head dimensions, page sizes, the rotation and what is out of range are as for the cache held in 4 bits.
 *
 *   cache       [num_pages][kv_heads][spec_kv8_page_bytes(page_size, head_dim)] bytes, 16-byte aligned.  A page and head
 *               holds, for its page_size slots: the keys' codes (page_size * head_dim bytes), the values' codes (as many), then
 *               16 bytes for each block of 16 slots.  Code d of slot t is in byte t / 8 * 8 head_dim + d / 16 * 128 + t % 8 * 16 +
 *               d % 16.  A block's bytes are a 32-bit word for its keys, one for its values, and 8 unused bytes; a word has
 *               the block's scale as a bfloat16 in its upper half, and in bit t % 16 of its lower half whether slot t's
 *               vector is held as NaN.  Nothing needs initialising: only what was appended is ever used.
 * A code is a float with a sign, 4 bits of exponent and 3 of mantissa (1 to 448, steps of 2^-9 below 2^-6).  A number x is
 * held as the code nearest to x / scale (ties to the even one, at most 448 in magnitude, zero as +0), of the exact rotated
 * key: what 32 bits leave in doubt is settled in 64.  A vector with a NaN or an infinity is held as NaN throughout.
 * A block's scale is a power of two, 2^-40 .. 2^40.  An append that writes slots of a block takes 2^(e - 8), with 2^e the least
 * power of two that is not below the largest magnitude that it writes there (NaN vectors left out).  If the block's first slots
 * hold tokens from before `start`, the scale is no less than it was, and where it grows their codes are
 * rounded to it (exact but for codes below 2^-6).  A block that begins with a new token takes no account of what it held.
 */
size_t spec_kv8_page_bytes(int page_size, int head_dim);

/*
 * Appends T new tokens per sequence.  Arguments as for spec_kv_append.  Tokens of k_values, v_values that are dropped
 * get what they would have been held as in a block without older tokens.  Two sequences must not append to the same block
 * of 16 slots (its scale is theirs together).  No workspace.
 */
sv_status spec_kv8_append(const void *k, int64_t k_batch_stride, int64_t k_token_stride, int64_t k_head_stride,
                          const void *v, int64_t v_batch_stride, int64_t v_token_stride, int64_t v_head_stride,
                          sv_kv_dtype dtype, int B, int T, int kv_heads, int head_dim, void *cache, int num_pages,
                          int page_size, const int32_t *page_table, int table_width, const int32_t *start,
                          const int32_t *new_lens, const float *cos, const float *sin, int table_len, int pairs,
                          int interleaved, const int32_t *positions, void *k_values, void *v_values, void *stream);

/*
 * Tokens of the cache in 16 bits.
 *   start, lens  [B]  row t of sequence b is its token start[b] + t (start clamped to [0, table_width * page_size]) for t <
 *                lens[b] (clamped to [0, T]; NULL: T).
 *   slots        NULL, or [B][T]: row t is token slots[b][t] instead.
 *   k, v         [B][T][kv_heads][head_dim] contiguous, 16-byte aligned, bf16 or fp16 (sv_kv_dtype): the keys as they are held,
 *                rotated; rounded to the type.  0 for rows from lens[b] on, tokens outside the table and pages out of range.
 */
sv_status spec_kv8_read(const void *cache, int num_pages, int page_size, int B, int T, int kv_heads, int head_dim,
                        const int32_t *page_table, int table_width, const int32_t *start, const int32_t *lens,
                        const int32_t *slots, sv_kv_dtype dtype, void *k, void *v, void *stream);

/*
 * Attention of the T new tokens over the cache, which holds them already.  Arguments, workspace and status as for
 * spec_kv_attention.  A row that sees a token whose key or value is held as NaN is NaN, and so is one whose query has a NaN or
 * an infinity.  The workspace grows with the batch: the queries are kept there in parts.
 * What is rounded on the way, beside sums in fp32: a query's number by 2^-12 of itself (not at all if it is bf16 and not rotated) and by 2^-17 of
 * its row's largest one; a token's weight (its probability times its value's scale) by 2^-8.6 of itself for bf16 results and by 2^-12
 * for fp16 ones, and by 2^-51 of the largest weight that the row has among 128 neighbouring tokens.  So a token of nearly all of the probability, or
 * a loud one in the same block, takes nothing from the others.  (More than 64 rows a kv head of 64 or 128 dimensions: 2^-17 of itself, and no more.)
 */
size_t spec_kv8_attention_workspace_size(int B, int T, int heads, int kv_heads, int head_dim);
sv_status spec_kv8_attention(const void *q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
                             sv_kv_dtype dtype, int B, int T, int heads, int kv_heads, int head_dim,
                             const void *cache, int num_pages, int page_size, const int32_t *page_table,
                             int table_width, const int32_t *start, const int32_t *new_lens, const int32_t *parent,
                             float scale, const float *cos, const float *sin, int table_len, int pairs,
                             int interleaved, const int32_t *positions, void *out, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Test hook (host only): the byte of code `dim` of slot `token` within a page and head.  -1 if an argument is out of range. */
int64_t spec_kv8_code_offset(int page_size, int head_dim, int values, int token, int dim);

/*
 * Test hook (host only): where code `dim` of slot `token` is within a page and head, in
 * half-bytes (2 * byte + 1 for a byte's upper half); of the values if `values`, else of the
 * keys.  -1 if an argument is out of range.
 */
int64_t spec_kv_code_offset(int page_size, int head_dim, int values, int token, int dim);

/*
 * Test hook of the bounds-checked build: from now on no thread block of spec_kv_attention or spec_kv8_attention gets the
 * unit-th piece of the cache (from 0) that it is to read, or any after it; -1: all do.  The waits for
 * them run out after a second each, the call ends with SV_ERR_TIMEOUT in its workspace, and its output
 * is NaN.  SV_ERR_UNSUPPORTED in the normal build.
 */
sv_status spec_kv_lose_unit(int unit);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_SERVE_H */
