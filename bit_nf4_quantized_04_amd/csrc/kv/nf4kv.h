/*
 * nf4kv.h -- C ABI of libnf4kv.so: a paged key/value cache held in 4 bits and
 * the operators around it, for models whose linear layers run on libnf4qlora.
 *
 *  - nf4_rope_*:       rotary positions (training and prompts; forward, backward)
 *  - nf4_kv_plan:      block tables and slot maps from request lengths
 *  - nf4_kv_append:    keys rotated, keys and values quantized into the cache
 *  - nf4_kv_read:      the stored values of given slots
 *  - nf4_kv_attention: causal attention over the cache, optionally through a
 *                      sliding window with the first tokens kept visible
 *
 * Conventions are those of nf4qlora.h: device pointers, bf16 as uint16_t bit
 * patterns, `stream` a hipStream_t, status codes of its enum, nothing
 * allocated, freed or synchronized, nothing enqueued on an error (except
 * NF4_ELAUNCH; the HIP error is then in nf4_kv_last_hip_error()).  Pointers
 * are aligned to 16 bytes and every stride of a bf16 tensor is a multiple of
 * 8 elements (fp32: 4), so that rows can be read 16 bytes at a time.  Outputs
 * do not alias inputs unless said otherwise.  The calls can be captured in a
 * HIP graph: nothing about them depends on device data, which the kernels
 * check themselves (an index outside its range never leads to an access).
 * A call of more than 2^31 threads (of the order of 10^7 tokens) is refused
 * with NF4_EINVAL.
 */
#ifndef NF4KV_H
#define NF4KV_H

#include "nf4qlora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache of n_pages pages, each holding page_size tokens of every head.  An
 * entry (one head of one token) is head_dim elements in blocks of 64: 4-bit
 * codes packed as in nf4_tensor (even element in the high nibble) and one
 * bf16 absmax per block.  An element is fl32(scale * level[code]), the levels
 * those of quant_type (nf4_levels()).  The scale of a cached bf16 block is
 * the magnitude of one of its elements, so 16 bits hold it exactly.  Scales
 * are non-negative, or NaN for a block that held Inf or NaN (its codes are
 * then the level-0 code, as in nf4_quantize).
 *   k_codes, v_codes:   [n_pages][n_heads][page_size][head_dim/2] uint8
 *   k_scales, v_scales: [n_pages][n_heads][page_size][head_dim/64] bf16
 * A token's slot is page * page_size + (position % page_size). */
typedef struct nf4_kv_cache {
    uint8_t* k_codes;
    uint16_t* k_scales;
    uint8_t* v_codes;
    uint16_t* v_scales;
    int64_t n_pages;    /* >= 1, at most 2^31 - 1 */
    int32_t n_heads;    /* 1 to 1024 */
    int32_t head_dim;   /* 64, 128 or 256 (NF4_EUNSUPPORTED otherwise) */
    int32_t page_size;  /* 16, 32, 64, 128 or 256 (NF4_EUNSUPPORTED otherwise) */
    int32_t quant_type; /* NF4_QUANT_NF4 or NF4_QUANT_FP4 */
} nf4_kv_cache;

/* The last hipError_t recorded by a failed launch of this library on the
 * calling thread. */
int nf4_kv_last_hip_error(void);

/* ---- rotary positions ---------------------------------------------------
 * The first `rot` elements of a head form rot/2 pairs: (i, i + rot/2) in the
 * half layout, (2i, 2i + 1) in the interleaved one; the others pass through.
 * Pair i of a token at position p turns by the angle p * theta_i. */
enum { NF4_ROPE_HALF = 0, NF4_ROPE_INTERLEAVED = 1 };

/* Frequencies for contexts longer than those trained on, with
 * theta_i = base^(-2i/rot):
 *   NONE:   theta_i
 *   LINEAR: theta_i / factor
 *   BASE:   base replaced by base * factor^(rot/(rot-2))  (rot > 2): the
 *           first pair keeps its frequency, the last one's is divided by factor
 *   PARTS:  pairs that turn at least `high` times within `original` tokens
 *           keep theta_i, those that turn at most `low` times get
 *           theta_i / factor, and the frequencies between are blended
 *           linearly in the number of turns n: w = (n - low)/(high - low),
 *           theta_i * (w + (1 - w)/factor)
 * `amplitude` multiplies every cosine and sine (1 for none). */
enum { NF4_ROPE_NONE = 0, NF4_ROPE_LINEAR = 1, NF4_ROPE_BASE = 2, NF4_ROPE_PARTS = 3 };
typedef struct nf4_rope_scaling {
    int32_t kind;
    float factor;      /* > 0; not read by NONE */
    float low, high;   /* PARTS: 0 <= low < high */
    float original;    /* PARTS: tokens trained on, > 0 */
    float amplitude;   /* finite */
} nf4_rope_scaling;

/* table[p][0, rot/2) = amplitude * cos(p theta_i), table[p][rot/2, rot) = the
 * sines, for p < max_pos: fp64 throughout, one rounding to fp32.  rot even,
 * 2 <= rot <= 512; base > 1. */
int nf4_rope_table(float* table, int64_t max_pos, int32_t rot, float base, const nf4_rope_scaling* scaling,
                   void* stream);

/* y = x with every head's pairs (a, b) turned:
 *   forward:  a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s))
 *   backward: the gradient of the forward, the same with -s
 * in fp32 without contraction, rounded once to the type of x.  x and y:
 * `tokens` rows, token_stride apart (elements), of n_heads heads, head_stride
 * apart (>= head_dim), of head_dim consecutive elements; `is_bf16` or fp32.
 * The heads of y do not overlap: a token's come before the next token's
 * (y_token_stride >= (n_heads - 1) * y_head_stride + head_dim), or a head's
 * tokens before the next head's (the same the other way round).
 * y may be x itself (same strides).  rot <= head_dim <= 512, head_dim a
 * multiple of 8.  positions: int32 [tokens]; the rotated elements of a token
 * outside [0, max_pos) are NaN.  tokens == 0 is a no-op. */
int nf4_rope_forward(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* y, int64_t y_token_stride,
                     int64_t y_head_stride, int64_t tokens, int32_t n_heads, int32_t head_dim, int32_t is_bf16,
                     const int32_t* positions, const float* table, int64_t max_pos, int32_t rot, int32_t layout,
                     void* stream);
int nf4_rope_backward(const void* dy, int64_t dy_token_stride, int64_t dy_head_stride, void* dx,
                      int64_t dx_token_stride, int64_t dx_head_stride, int64_t tokens, int32_t n_heads,
                      int32_t head_dim, int32_t is_bf16, const int32_t* positions, const float* table,
                      int64_t max_pos, int32_t rot, int32_t layout, void* stream);

/* ---- block tables and slot maps -----------------------------------------
 * One step's bookkeeping for `batch` requests (1 to 4096), on the device.
 * Request i holds kv_lens[i] tokens in the pages block_table[i][0 ..
 * ceil(kv_lens[i] / page_size)) and asks for new_lens[i] more; one with
 * done[i] != 0 (done may be NULL) ends instead.  Negative lengths count as 0.
 * Free pages stand in a ring of `capacity` entries: free_state = {head,
 * count}, entry j of it at free_pages[(head + j) % capacity].
 *
 * In request order, request i wants the pages its longer length needs beyond
 * those it holds.  It is refused (and keeps its length) if that length does
 * not fit table_width pages, if it wants pages and the wants up to and with
 * its own exceed `count`, or if it asks for tokens and the tokens asked for
 * up to and with its own exceed max_tokens (requests refused for the first
 * reason want and ask nothing; those refused for the others still count, so
 * no later request overtakes them).  The step's token list holds the granted
 * requests' tokens only, one request after the other: a caller whose rows lie
 * by new_lens gathers them, token t of request i from row
 * sum(new_lens[0 .. i)) + t - cu_new[i].  Then
 *   block_table   gains the granted pages, taken from the ring's head (in place)
 *   free_pages    gets the ended requests' pages at its tail, in request order (in place)
 *   free_out      {head, count} after both; not free_state itself
 *   kv_lens_out   the lengths with the new tokens, 0 for an ended request
 *   cu_new        [batch + 1] first new token of each request in the step's token list
 *   slots         [max_tokens] int64 slot of each token of the list, then -1
 *   positions     [max_tokens] int32 position of each token, then 0
 *   refused       [1] how many requests were refused
 * kv_lens_out, free_out and cu_new do not alias the inputs.  capacity and
 * max_tokens are at most 2^30. */
int nf4_kv_plan(const int32_t* kv_lens, const int32_t* new_lens, const int32_t* done, int32_t batch,
                int32_t* block_table, int32_t table_width, int32_t page_size, int32_t* free_pages, int32_t capacity,
                const int32_t* free_state, int32_t max_tokens, int32_t* kv_lens_out, int32_t* cu_new, int64_t* slots,
                int32_t* positions, int32_t* free_out, int32_t* refused, void* stream);

/* ---- the cache's write and read -----------------------------------------
 * Keys are rotated as nf4_rope_forward does (rounded to bf16, as a prompt's
 * attention would see them), then keys and values are quantized into the
 * slots: per 64-element block S = max |x|, code = the level nearest
 * fl32(x / S), an exact tie to the lower (FP4: even) one; an all-zero block
 * and one holding Inf or NaN as nf4_quantize.  A slot outside the cache (-1
 * for padding) writes nothing.  The slots of one call are distinct.
 *   k, v: bf16 [tokens][n_heads][head_dim], tokens *_stride elements apart
 *   q:    bf16 [tokens][q_heads][head_dim], or NULL; q_out (tokens
 *         q_out_stride apart) receives it rotated, padding included
 *   positions, table, max_pos, rot, layout: as nf4_rope_forward; rot == 0
 *         rotates nothing (positions and table may be NULL; q must be)
 * tokens == 0 is a no-op. */
int nf4_kv_append(const nf4_kv_cache* cache, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                  int64_t v_stride, const int64_t* slots, int64_t tokens, const uint16_t* q, int64_t q_stride,
                  uint16_t* q_out, int64_t q_out_stride, int32_t q_heads, const int32_t* positions,
                  const float* table, int64_t max_pos, int32_t rot, int32_t layout, void* stream);

/* The stored keys and values of slots, bf16(fl32(scale * level)), each
 * [tokens][n_heads][head_dim] contiguous (either may be NULL); zeros for a
 * slot outside the cache. */
int nf4_kv_read(const nf4_kv_cache* cache, const int64_t* slots, int64_t tokens, uint16_t* k_out, uint16_t* v_out,
                void* stream);

/* ---- attention ----------------------------------------------------------
 * Request i has queries cu_q[i] .. cu_q[i+1] (rows of q), the last tokens of
 * its kv_lens[i] cached ones: query j of n stands at position
 * p = kv_lens[i] - n + j and sees the cached tokens t <= p that are inside
 * the window, t > p - window (window == 0: all), or among the first, t < sinks.
 *   out = sum_t softmax_t(scale * q.k_t) v_t,
 * 0 for a query that sees nothing.  Query head h reads cache head
 * h / (q_heads / n_heads).  Sums and softmax statistics are fp32; products
 * take fp16 operands (the levels and the softmax weights, 11 bits) on the
 * matrix units, q scaled by a power of two per row so that fp16 holds every
 * bit of its bf16 values down to 2^-14 of the row's largest.  A query holding
 * Inf or NaN gives NaN, as does a visible block whose scale is NaN (a value's,
 * unless the token's weight is 0 in fp32); what a mask hides has no effect
 * whatever it holds.  A token's weight times its largest absmax is kept to 11
 * bits down to 2^-21 of the row's largest such product and to 2^-32 of it
 * below; values of blocks whose absmax is below 2^-110 lose bits, and below
 * 2^-122 count as 0.  Scores beyond 2^26 leave fp32 no bits to
 * weigh tokens by: the result is then of no meaning, and NaN once they, or the
 * products of a key whose absmax is 2^115 or more, overflow fp32.
 *   q, out: bf16 [total_q][q_heads][head_dim], tokens *_stride elements apart
 *   cu_q: int32 [batch + 1]; kv_lens: int32 [batch]
 *   block_table: int32 [batch][table_width]; the tokens of a page id outside
 *     the cache are not visible
 *   max_q: at least every request's queries (later ones are not computed)
 *   max_len: at least every request's length; at most table_width * page_size.
 *     A longer request is taken for one of max_len tokens: its queries stand at
 *     the last of those.  The bounds, not the lengths, decide how a call is
 *     cut up, so that tight ones are faster
 *   ws: nf4_kv_attention_ws_bytes() of workspace
 * 1 <= batch <= 65535, q_heads a multiple of n_heads, q_heads / n_heads <= 128;
 * with 96 rows (queries times q_heads / n_heads) or more, batch * n_heads times
 * the rows' blocks of 256 (128 at 256 elements a head) below 2^23.
 * Rows of out that no request has (before cu_q[0], from cu_q[batch] on: a step
 * whose token list has room to spare) and a request's queries past max_q are
 * left as they are by nf4_kv_attention, and made zeros by
 * nf4_kv_attention_padded, which is otherwise the same.
 * total_q == 0 is a no-op, and so is max_q == 0 but for those zeros. */
size_t nf4_kv_attention_ws_bytes(int32_t batch, int32_t q_heads, int32_t n_heads, int32_t head_dim, int32_t max_q,
                                 int32_t max_len, int32_t window, int32_t sinks);
int nf4_kv_attention(const nf4_kv_cache* cache, const uint16_t* q, int64_t q_stride, int64_t total_q,
                     int32_t q_heads, const int32_t* cu_q, const int32_t* kv_lens, const int32_t* block_table,
                     int32_t table_width, int32_t batch, int32_t max_q, int32_t max_len, float scale, int32_t window,
                     int32_t sinks, uint16_t* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream);
int nf4_kv_attention_padded(const nf4_kv_cache* cache, const uint16_t* q, int64_t q_stride, int64_t total_q,
                            int32_t q_heads, const int32_t* cu_q, const int32_t* kv_lens, const int32_t* block_table,
                            int32_t table_width, int32_t batch, int32_t max_q, int32_t max_len, float scale,
                            int32_t window, int32_t sinks, uint16_t* out, int64_t out_stride, void* ws,
                            size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NF4KV_H */
