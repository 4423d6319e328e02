/*
 * domino_verify.h — C ABI of the operators around the verification of a draft
 * block on MI355X (gfx950): the key-value cache of the target model, the
 * attention of a block's tokens over it, the rules applied to the target's
 * logits, and the decision which proposals stand.
 *
 * A rollout (domino_rollout.h) proposes up to 15 tokens for each request.  The
 * target model scores the block in one pass; these operators carry that pass
 * around the target's own matrix products:
 *   domino_rotation_run       norms of query and key heads, rotation by position
 *   domino_attention_append   keys and values of the new tokens into pages
 *   domino_attention_run      causal attention of the new tokens over the pages
 *   domino_attention_create_fp4, _read   the same over a cache held in 4 bits
 *   domino_verify_process     penalties, biases and grammar masks on logits
 *   domino_verify_run         the same rules fused with the acceptance of the
 *                             proposals and the choice of the token that follows
 *   domino_scores_run         log-probabilities of given tokens, entropies and the
 *                             likeliest ids of rows of logits
 *
 * Conventions are those of domino_rollout.h: a handle owns its workspace, on
 * the device that is current at create, and is not re-entrant (one run in
 * flight per handle); every run enqueues kernels on the caller's stream (NULL =
 * the default stream), checks host scalars and pointers only, allocates
 * nothing, does not synchronise and may be captured into a graph.  Lengths,
 * page tables and token ids live on the device and are never trusted as
 * addresses: what is out of range is not dereferenced, and each function says
 * what it yields then.
 */
#ifndef DOMINO_VERIFY_H
#define DOMINO_VERIFY_H

#include "domino_rollout.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ norm and rotation of heads */

typedef struct {
  int32_t q_heads;      /* 1..1024                                              */
  int32_t kv_heads;     /* 1..1024                                              */
  int32_t head_dim;     /* D: 64, 128 or 256                                    */
  int32_t rotary_dim;   /* R: elements that are rotated, a multiple of 16, <= D */
  int32_t dtype;        /* domino_dtype_t of heads and weights                  */
  int32_t interleaved;  /* 0: element i turns with i + R / 2; 1: 2i with 2i + 1 */
  float magnitude;      /* factor of cosines and sines, usually 1               */
} domino_rotation_config_t;

typedef struct domino_rotation domino_rotation_t;

/* Heads of one kind (device pointers): token i, head h at
 * in + i * token_stride + h * head_stride (elements), out alike; arrays are
 * 16-byte aligned and strides multiples of 16 bytes, out's at least head_dim
 * where there is more than one.  out may be in with the same strides; any other
 * overlap is undefined. */
typedef struct {
  const void* in;
  int64_t token_stride, head_stride;
  const void* weight;   /* [head_dim] or NULL: no norm                          */
  void* out;
  int64_t out_token_stride, out_head_stride;
} domino_heads_t;

/* Validates the configuration, checks that the current HIP device is gfx950
 * and keeps the frequencies inv_freq[rotary_dim / 2] (host memory, radians a
 * position, finite and within 1000 of 0).  Synchronises the device. */
domino_status_t domino_rotation_create(const domino_rotation_config_t* cfg, const double* inv_freq,
                                       domino_rotation_t** out);

/* For each token i and head, x its elements and p = positions[i]:
 *   y = x / sqrt(mean(x^2) + eps) * weight       (y = x without weights)
 *   a' = magnitude * (a cos(p f_j) - b sin(p f_j))
 *   b' = magnitude * (b cos(p f_j) + a sin(p f_j))   for the pairs (a, b) of y, j < R / 2
 * and elements from R on are y.  The weights of q and k are given together or
 * not at all.  All of it is fp32 and rounded once; the whole turns of an angle
 * are taken off before it is rounded to fp32, so that any position is as good as
 * the first at every frequency.  Tokens with a negative position are not written.
 * eps >= 0 and finite. */
domino_status_t domino_rotation_run(domino_rotation_t* h, const domino_heads_t* q, const domino_heads_t* k,
                                    const int32_t* positions, int32_t tokens, float eps, void* stream);

/* Frees the workspace.  NULL is a no-op. */
void domino_rotation_destroy(domino_rotation_t* h);

/* As domino_attention_last_error. */
const char* domino_rotation_last_error(const domino_rotation_t* h);

/* ------------------------------------------------------------ paged attention */

typedef struct {
  int32_t q_heads;      /* > 0, a multiple of kv_heads                          */
  int32_t kv_heads;     /* > 0                                                  */
  int32_t head_dim;     /* 64, 128 or 256                                       */
  int32_t page_size;    /* keys per page: a power of two, 16..4096              */
  int32_t max_requests; /* 1..1024                                              */
  int32_t dtype;        /* domino_dtype_t of queries, cache and output          */
} domino_attention_config_t;

typedef struct domino_attention domino_attention_t;

/* A batch's cache and lengths (device pointers, caller-owned).  Strides count
 * elements; element (page, head, row, i) of a cache lies at
 * page * page_stride + head * head_stride + row * row_stride + i, the same for
 * keys and values.  The three strides are multiples of 16 bytes, and a page
 * spans less than 2^31 bytes; offsets across pages are 64-bit.
 *
 * Request b has q_start[b + 1] - q_start[b] new tokens, rows q_start[b].. of
 * the token arrays, and kv_len[b] keys in its cache, the new tokens' own
 * included: new token t stands at position kv_len[b] - new + t, and position
 * p in row p % page_size of page page_table[b][p / page_size].
 *
 * A request is malformed if its rows are not within [0, tokens], it has more
 * than max_new new tokens, kv_len[b] is negative, or kv_len[b] exceeds max_kv,
 * what the table's width holds or 2^30.  A position before 0 (fewer keys than new
 * tokens) has no key; its token's attention is empty. */
typedef struct {
  void* k_cache;
  void* v_cache;
  int64_t page_stride, head_stride, row_stride;
  int32_t num_pages;          /* pages of each cache                            */
  const int32_t* page_table;  /* [requests, table_width], rows table_stride apart */
  int64_t table_stride;
  int32_t table_width;
  const int32_t* kv_len;      /* [requests]                                     */
  const int32_t* q_start;     /* [requests + 1]                                 */
  int32_t requests;           /* 1..max_requests                                */
  int32_t tokens;             /* rows of the token arrays (>= 0)                */
  int32_t max_new;            /* upper bound of a request's new tokens          */
  int32_t max_kv;             /* upper bound of kv_len                          */
} domino_cache_t;

/* Validates the configuration, checks that the current HIP device is gfx950
 * and allocates the workspace of the split attention (partial outputs of two
 * segments for each workgroup, at most 69 MB).  Synchronises the device. */
domino_status_t domino_attention_create(const domino_attention_config_t* cfg,
                                        domino_attention_t** out);

/* Writes keys and values of the new tokens into the cache: token row i, head h
 * of k lies at k + i * k_token_stride + h * k_head_stride (elements, multiples
 * of 16 bytes), v alike.  Tokens of a malformed request, at a negative
 * position, or whose page id is outside [0, num_pages) are not written.  Where
 * two tokens of a call meet in one row (a page id stands twice), pieces of either
 * remain. */
domino_status_t domino_attention_append(domino_attention_t* h, const domino_cache_t* cache,
                                        const void* k, int64_t k_token_stride,
                                        int64_t k_head_stride, const void* v,
                                        int64_t v_token_stride, int64_t v_head_stride,
                                        void* stream);

/* Attention of the new tokens.  With p the position of a token, key position
 * j is visible to it if j <= p and (window == 0 or j > p - window or
 * j < sinks).  Query head h reads key head h / (q_heads / kv_heads).
 *   s_j = scale * (q . k_j);  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m);
 *   lse = m + ln sum_j e^(s_j - m),  m = max_j s_j, j over the visible keys.
 * Scores, softmax statistics and sums are fp32; for bf16 the weights
 * e^(s_j - m) multiply v to 15 bits where max_new * q_heads / kv_heads is at
 * most 32, rounded to bf16 beyond that, and the result is rounded once.  Without a visible key, out is 0 and lse is -inf.  Keys and
 * values that no new token sees do not influence the result whatever they
 * hold, and pages that hold only such keys are not read.  Tokens of a
 * malformed request (its first max_new rows within [0, tokens)) get NaN, and
 * so do tokens that see a key of a page outside [0, num_pages); other tokens
 * of that request may.  window >= 0, sinks >= 0, scale finite and > 0.  q and out rows:
 * token i, head h at i * token_stride + h * head_stride (elements, multiples
 * of 16 bytes; out's at least head_dim where there is more than one); lse is
 * [tokens, q_heads] fp32 or NULL.  max_new and max_kv choose the kernels:
 * bounds near the truth are faster. */
domino_status_t domino_attention_run(domino_attention_t* h, const domino_cache_t* cache,
                                     const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                     int32_t window, int32_t sinks, float scale, void* out,
                                     int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                     void* stream);

/* ---- a cache held in 4 bits
 *
 * A handle of domino_attention_create_fp4 takes the calls of one of
 * domino_attention_create, with queries, new keys and values and outputs in
 * bf16 (dtype must be DOMINO_DTYPE_BF16) and a cache in which 32 elements of a
 * token and key head, a block, share a power of two 2^e.  Its byte holds e + 127,
 * 255 makes the block NaN; an element is 4 bits, the upper one a sign and the
 * lower three the number 0, 0.5, 1, 1.5, 2, 3, 4, 6 of that index.  In a page of a head lie
 *   page_size x head_dim / 2 bytes: elements, row after row, the lower element
 *     of two in the low bits of a byte;
 *   page_size x head_dim / 32 bytes: powers, row after row.
 * page_stride and head_stride of the cache count bytes and are multiples of 16,
 * row_stride must be head_dim / 2.
 *
 * Append gives a block the least e with max |x| <= 7 x 2^e, kept within
 * [-125, 125], and each element the nearest number, of two the one of even
 * index, at most 6; a block with an infinity or NaN becomes NaN.  Numbers up to
 * 6 x 2^e are off by at most half a step of the numbers around them, others by
 * at most 2^e (the largest bf16 numbers, from 7 x 2^125 on, become 6 x 2^125).  Run
 * computes its formula over the numbers that the cache stands for, which bf16
 * holds exactly; blocks of NaN and unseen keys have the effects stated there.
 * Powers of 2^-126 and less may count as zero, blocks of 2^126 and more as NaN.
 * In append and read a request's new tokens, by the bounds, times kv_heads and
 * head_dim stay below 2^33. */
domino_status_t domino_attention_create_fp4(const domino_attention_config_t* cfg,
                                            domino_attention_t** out);

/* Gives back what the cache of 4 bits stands for at the positions of the new
 * tokens: rows of k and v as in append, written in bf16 (at least head_dim
 * apart).  Tokens of a malformed request (its first max_new rows within
 * [0, tokens)), at a negative position, or whose page id is outside
 * [0, num_pages) get NaN. */
domino_status_t domino_attention_read(domino_attention_t* h, const domino_cache_t* cache, void* k,
                                      int64_t k_token_stride, int64_t k_head_stride, void* v,
                                      int64_t v_token_stride, int64_t v_head_stride, void* stream);

/* Frees the workspace.  NULL is a no-op. */
void domino_attention_destroy(domino_attention_t* h);

/* Message of the handle's last error, or of this thread's last failed create
 * when h is NULL.  Never NULL. */
const char* domino_attention_last_error(const domino_attention_t* h);

/* ------------------------------------------------------------ logits and acceptance */

typedef struct {
  int32_t vocab;        /* V > 0                                                */
  int32_t max_requests; /* 1..1024                                              */
  int32_t max_rows;     /* 1..64: rows of logits of a request (proposals + 1)   */
  int32_t dtype;        /* domino_dtype_t of the logits                         */
} domino_verify_config_t;

typedef struct domino_verify domino_verify_t;

/* Logits and the rules for them (device pointers; a NULL rule does not apply).
 * Row t of request b holds the logits that follow the request's text and its
 * first t proposals.  For id v:
 *   c    = occurrences of v in history[b][prompt_len .. history_len) and among
 *          the proposals draft[b][0 .. t)
 *   seen = c > 0, or v in history[b][0 .. prompt_len)
 *   x = seen ? (x > 0 ? x / repetition : x * repetition) : x
 *   x = x - frequency * c
 *   x = x - presence * [c > 0]
 *   x = x + bias(v)      (the last entry of an id in the request's list holds)
 *   x = -inf             where the mask's bit v % 32 of word v / 32 is 0
 * in this order, each operation rounded in fp32.  Ids outside [0, V) in a
 * history, draft or bias list are passed over; lengths are clipped to
 * [0, width].  The history and the proposals count only if at least one of
 * the three penalties is given. */
typedef struct {
  const void* logits;
  int64_t request_stride, row_stride; /* elements, >= 0 as every stride here    */
  int32_t requests, rows;
  const int32_t* draft;               /* [requests, rows - 1] proposals or NULL */
  int64_t draft_stride;
  const int32_t* draft_len;           /* [requests] proposals of each, or NULL: rows - 1 */
  const int32_t* history;             /* [requests, history_width] token ids    */
  int64_t history_stride;
  int32_t history_width;
  const int32_t* history_len;         /* [requests] or NULL: history_width      */
  const int32_t* prompt_len;          /* [requests] or NULL: 0                  */
  const float* repetition;            /* [requests], > 0                        */
  const float* frequency;             /* [requests]                             */
  const float* presence;              /* [requests]                             */
  const int32_t* bias_ids;            /* [requests, bias_width]                 */
  const float* bias_values;
  int64_t bias_stride;
  int32_t bias_width;
  const int32_t* bias_len;            /* [requests] or NULL: bias_width         */
  const uint32_t* mask;               /* [requests, rows, ceil(V / 32)], bit 1 = allowed */
  int64_t mask_request_stride, mask_row_stride; /* words; 0 shares a mask       */
} domino_logits_t;

/* Validates the configuration, checks that the current HIP device is gfx950
 * and allocates the workspace (row statistics of each part of the vocabulary).
 * Synchronises the device. */
domino_status_t domino_verify_create(const domino_verify_config_t* cfg, domino_verify_t** out);

/* Writes the processed logits, rounded once to the handle's dtype.  out may be
 * the logits themselves with the same strides; any other overlap is undefined. */
domino_status_t domino_verify_process(domino_verify_t* h, const domino_logits_t* logits, void* out,
                                      int64_t out_request_stride, int64_t out_row_stride,
                                      void* stream);

/* Accepts proposals from the processed logits (kept in fp32, never written).
 * A request with temperature T > 0 samples, with T <= 0 (or temperature NULL)
 * it is greedy.  With l = log softmax(x / T) (T = 1 if greedy) and
 * n = min(draft_len, rows - 1), proposal d of row t = 0, 1, .. n - 1 stands if
 *   greedy:   d is the lowest id of the largest x;
 *   sampling: accept_u[b][t] < e^l(d), or no other id has x > -inf.
 * At the first row whose proposal does not stand, or at row n, the token is
 *   the lowest id of the largest x - T ln(noise[b][v]) over the ids v with
 *   x > -inf, without d if a proposal was refused there
 * (greedy: of the largest x).  With noise drawn from the unit exponential and
 * accept_u uniform in [0, 1), tokens follow the target's distribution exactly,
 * since each proposal is the drafter's only candidate.  noise must be > 0.
 *   out_tokens   [requests, rows] int32: the proposals that stand, the token
 *                after them, then -1
 *   out_accepted [requests] int32: how many proposals stand
 *   out_logprob  [requests, rows] fp32 or NULL: l of each token, then 0
 * A row without an id of x > -inf yields token -1 and log-probability -inf.
 * NaN logits count as -inf and +inf as the largest fp32 number; T is clipped
 * to [1e-30, 1e30].  accept_u (if rows > 1) and noise must be given where
 * temperature is. */
domino_status_t domino_verify_run(domino_verify_t* h, const domino_logits_t* logits,
                                  const float* temperature, const float* accept_u,
                                  int64_t accept_stride, const float* noise, int64_t noise_stride,
                                  int32_t* out_tokens, int32_t* out_accepted, float* out_logprob,
                                  void* stream);

/* Frees the workspace.  NULL is a no-op. */
void domino_verify_destroy(domino_verify_t* h);

/* As domino_attention_last_error. */
const char* domino_verify_last_error(const domino_verify_t* h);

/* ------------------------------------------------------------ scores of tokens */

typedef struct {
  int32_t vocab;     /* V, 1..2^24                                             */
  int32_t max_rows;  /* 1..65535                                               */
  int32_t max_top;   /* 0..64: the most ids of a row that are asked for        */
  int32_t dtype;     /* domino_dtype_t of the logits                           */
} domino_scores_config_t;

typedef struct domino_scores domino_scores_t;

/* Validates the configuration, checks that the current HIP device is gfx950
 * and allocates the workspace (statistics of parts of rows and, with max_top,
 * V / 32 bytes a row).  Synchronises the device. */
domino_status_t domino_scores_create(const domino_scores_config_t* cfg, domino_scores_t** out);

/* Scores of rows of logits, row i at logits + i * row_stride (elements, >= 0).  With
 * p = softmax(x) of a row's logits x:
 *   logprob  [rows] fp32: ln p(tokens[i]); -inf for a token outside [0, V) or of x = -inf
 *   entropy  [rows] fp32: -sum p ln p
 *   top_ids  [rows, top] int32, top_logprob [rows, top] fp32: the ids of the
 *            `top` largest x, largest first and the lower id first among equal
 *            ones, with ln p; ids of x = -inf are none, -1 and -inf in their place
 * Each is optional (NULL; top 0); tokens and logprob, and the outputs of top, go
 * together.  NaN logits count as -inf and +inf as the largest fp32 number.  A row
 * without x > -inf has entropy 0.  Sums are fp32. */
domino_status_t domino_scores_run(domino_scores_t* h, const void* logits, int64_t row_stride, int32_t rows,
                                  const int32_t* tokens, int32_t top, float* logprob, float* entropy,
                                  int32_t* top_ids, float* top_logprob, void* stream);

/* Frees the workspace.  NULL is a no-op. */
void domino_scores_destroy(domino_scores_t* h);

/* As domino_attention_last_error. */
const char* domino_scores_last_error(const domino_scores_t* h);

#ifdef __cplusplus
}
#endif
#endif /* DOMINO_VERIFY_H */
