/*
 * gdn_attention.h -- C ABI of a full-attention layer that is served beside
 * Gated DeltaNet layers on GB300 (sm_103a): the step's keys and values go into
 * a paged cache, and its queries attend over their requests' pages.
 *
 *   gdn_kv_append    norms and position rotation of queries and keys; keys and
 *                    values into the cache
 *   gdn_attn_paged   causal attention over the pages: one new token a request
 *                    (decode), a few (verify), or chunks of prompts
 *
 * gdn_slot_map (gdn_prefill.h) makes their offsets, positions, slots and block
 * tables; gdn_linear and gdn_linear_w4 are the layer's projections.
 *
 * Conventions (beside those of gdn_decode.h and gdn_prefill.h):
 *  - A cache is num_slots = num_blocks * block_size rows of num_kv_heads *
 *    head_dim bf16 values (head h at column h * head_dim); slots are `ld*`
 *    values apart. Block b holds slots b * block_size and on. Key position p of
 *    request s is in slot block_table[s][p / block_size] * block_size +
 *    p % block_size. Several requests may share blocks.
 *  - A ragged batch's rows and offsets are those of gdn_prefill.h: request s has
 *    rows cu_seqlens[s] .. cu_seqlens[s+1] - 1, rows past the last are pad rows,
 *    and whatever the offsets hold every row has one owner.
 *  - Query head h reads key/value head h / (num_q_heads / num_kv_heads).
 *  - Row strides (ld*) count elements and are multiples of 8; pointers of bf16
 *    matrices are 16-byte aligned.
 */
#ifndef GDN_ATTENTION_H_
#define GDN_ATTENTION_H_

#include "gdn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* For every token t with slots[t] in 0 .. num_slots - 1:
 *   q', k' = q, k; with norm weights each head's x is first
 *     x / sqrt(mean x^2 + norm_eps) * (1 + w)                (Gemma form)
 *   and its first rotary_dim values turn by angles token_pos[t] * inv_freq[i],
 *     (a, b) -> (a cos - b sin, b cos + a sin),
 *   with a, b the values i and i + rotary_dim / 2 of the head, or with
 *   `interleaved` 2 i and 2 i + 1;
 *   q_out[t] = q', k_cache[slots[t]] = k', v_cache[slots[t]] = v.
 * f32 throughout, one rounding to bf16; v is copied. An angle is within 2^-25 of a
 * turn at any position (its fraction in 64-bit fixed point, rounded to f32). A token with a
 * negative slot is a pad row: its q_out row is zero and nothing is appended. A
 * slot >= num_slots does the same and sets *error (a device word, optional) to
 * GDN_ERR_INDEX in bits 31..24, 1 in 23..16 and the token in 15..0, if it was
 * zero. Slots >= 0 must be distinct.
 * q [tokens][ldq >= num_q_heads * head_dim] and q_out, or both NULL (keys and
 * values alone; num_q_heads is then ignored), k, v [tokens][>= num_kv_heads *
 * head_dim] bf16; token_pos int32, slots int64 [tokens]; inv_freq f32
 * [rotary_dim / 2] (radians a position, of less than 2^40; NULL with rotary_dim 0);
 * rotary_dim a multiple of 16, at most head_dim; head_dim 64, 128 or 256;
 * q_norm_w, k_norm_w bf16 [head_dim], each or both NULL: no norm. q_out may be q
 * itself (same pointer and stride); otherwise outputs overlap no input. */
gdn_status gdn_kv_append(int32_t tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, const void* q,
                         int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* token_pos,
                         const int64_t* slots, int64_t num_slots, const float* inv_freq, int32_t rotary_dim,
                         int32_t interleaved, const void* q_norm_w, const void* k_norm_w, float norm_eps, void* q_out,
                         int64_t ldqo, void* k_cache, int64_t ldkc, void* v_cache, int64_t ldvc, uint32_t* error,
                         void* stream);

typedef struct {
  int32_t num_q_heads;   /* a multiple of num_kv_heads */
  int32_t num_kv_heads;
  int32_t head_dim;      /* 64, 128 or 256 */
  int32_t block_size;    /* slots of a block, any number >= 1 */
  int32_t max_tokens;    /* most rows of one call */
  int32_t max_seqs;      /* most requests of one call */
  float scale;           /* multiplies q . k; any finite number (chunks take longer with one of 0 or below) */
} gdn_attn_config;

typedef struct gdn_attn gdn_attn_t;

/* Device bytes of the workspace for this config on the current device; 0 if
 * the config is invalid or unsupported. It holds the parts of rows that several
 * CTAs work on, two for each CTA that runs at once. */
size_t gdn_attn_workspace_bytes(const gdn_attn_config* cfg);

/* Validate the config, bind the caller's workspace (256-byte aligned device
 * memory that outlives the handle) and clear its error word and counters on
 * `stream`. The handle holds host state only. It belongs to the device that is
 * current here; calls with another one current are GDN_ERR_ARG. Calls on another stream
 * are ordered after the clearing by the caller. */
gdn_status gdn_attn_create(const gdn_attn_config* cfg, void* workspace, size_t workspace_bytes, void* stream,
                           gdn_attn_t** out);

/* Causal attention of every request's new tokens over its context and
 * themselves: token j of request s, whose context is c = context_lens[s], has
 * position c + j and sees keys 0 .. c + j (its own among them, which
 * gdn_kv_append has put into the cache before):
 *   o = sum_p softmax_p(scale q . k_p) v_p,  and with gate: o * sigmoid(gate).
 * Scores, maxima, sums and outputs are f32; the weights of the values are
 * rounded to bf16 before they are multiplied. Sums of weights (of 2^8 at most, or for scores past 2^20
 * of 2^40) times values have to stay within f32's range. Keys a token does not see have no
 * part in its row, whatever they hold; a value that is not finite and is seen makes its
 * column of the row NaN or infinite; a row whose every score is minus infinity is zero.
 * max_len is an upper bound of the requests' new tokens known to the host
 * (tokens if nothing better is known); it chooses the form: where it times the query heads
 * of a key/value head is at most 16, that of few rows. A bound that is too high makes
 * single tokens take the chunks' form, which is up to half as long again.
 * A request longer than max_len, with a negative context, or with more keys
 * than max_blocks blocks hold records GDN_ERR_INDEX and is padding: zero rows.
 * A block outside 0 .. num_blocks - 1 that a request needs records GDN_ERR_INDEX
 * and is read as zeros. Pad rows and their outputs: not read, zero.
 * q, out [tokens][>= num_q_heads * head_dim], gate likewise or NULL, a row's query heads one
 * after another (where a projection has a head's query and gate side by side, its weights' rows are
 * put in this order once); k_cache,
 * v_cache [num_blocks * block_size][>= num_kv_heads * head_dim] bf16 (fewer
 * than 2^31 slots; ldq, ldk and ldv below 2^38); block_table int32 [seqs][max_blocks], cu_seqlens int32
 * [seqs + 1], context_lens int32 [seqs]. out must overlap no input.
 * One call at a time per handle (its calls share the workspace). */
gdn_status gdn_attn_paged(gdn_attn_t* h, int32_t seqs, int32_t tokens, int32_t max_len, const void* q, int64_t ldq,
                          const void* k_cache, int64_t ldk, const void* v_cache, int64_t ldv, int32_t num_blocks,
                          const int32_t* block_table, int32_t max_blocks, const int32_t* cu_seqlens,
                          const int32_t* context_lens, const void* gate, int64_t ldg, void* out, int64_t ldo,
                          void* stream);

/* Synchronise `stream` and read the sticky error word: GDN_OK or the first
 * recorded device status. *detail (optional) receives the raw word: bits 31..24
 * status, 23..16 what (1 a block outside the cache, 2 cu_seqlens as for
 * gdn_prefill_check, 3 a request longer than max_len, 4 a wait inside the kernel
 * that passed its limit, 5 a context that is negative or past the block table),
 * 15..0 the request. */
gdn_status gdn_attn_check(gdn_attn_t* h, void* stream, uint32_t* detail);

/* Clear the error word and the counters on `stream`. */
gdn_status gdn_attn_reset(gdn_attn_t* h, void* stream);

/* Free the host handle. The workspace stays the caller's. */
void gdn_attn_destroy(gdn_attn_t* h);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTENTION_H_ */
