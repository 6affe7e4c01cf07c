/*
 * gdn_prefill.h -- C ABI of the GB300 (sm_103a) prompt side of a Gated
 * DeltaNet (GDN) layer: the operators that take ragged batches of prompt
 * tokens to the conv and SSM states the decode step (gdn_decode.h) continues
 * from.
 *
 *   gdn_slot_map       offsets, block tables and slots of a ragged batch from
 *                      its request lengths, on the device
 *   gdn_linear         act(x W^T + bias) + residual (in_proj, out_proj)
 *   gdn_prefill_conv   causal depthwise conv1d + SiLU, conv state in and out
 *   gdn_prefill_delta  L2-normalised q/k, gates, the gated delta rule and
 *                      optionally the gated RMSNorm x SiLU(z), SSM state in
 *                      and out; requests of one token are its recurrent form
 *
 * The layouts, the state pools and the status codes are those of
 * gdn_decode.h, so a slot written here is one gdn_decode_step can take.
 *
 * Conventions (beside those of gdn_decode.h: device pointers owned by the
 * caller, no allocation, asynchronous and stream-ordered, capturable in a
 * CUDA graph, host-side argument errors before any launch):
 *  - A ragged batch is `tokens` rows holding `seqs` sequences one after the
 *    other: sequence s has rows cu_seqlens[s] .. cu_seqlens[s+1] - 1.
 *    cu_seqlens is int32 [seqs + 1] on the device, starts at 0 and does not
 *    decrease; a sequence may be empty. Rows from cu_seqlens[seqs] on are pad
 *    rows: they are not read and their output rows are zero.
 *  - state_in and state_out are int32 [seqs] slots on the device. Sequence s
 *    starts from slot state_in[s], or from zero state when state_in[s] <= 0,
 *    and leaves its state in slot state_out[s]; state_out[s] <= 0 makes it
 *    padding: zero output rows, no state read or written. An empty sequence
 *    passes its state on. The two may be the same slot; several sequences may
 *    start from one slot (a shared prefix), but state_out slots must be
 *    distinct and none may be another sequence's state_in.
 *  - Row strides (ld*) count elements; rows need not be packed. Outputs may be
 *    columns beside an input's in the same rows (an equal stride); that is not
 *    an overlap.
 */
#ifndef GDN_PREFILL_H_
#define GDN_PREFILL_H_

#include "gdn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t num_k_heads;   /* Hk */
  int32_t num_v_heads;   /* Hv, a multiple of Hk */
  int32_t head_k_dim;    /* dk: 64 or 128 */
  int32_t head_v_dim;    /* dv = dk */
  int32_t conv_kernel;   /* must be 4 */
  int32_t num_slots;
  int32_t max_tokens;    /* most rows of one call */
  int32_t max_seqs;      /* most sequences of one call */
  int32_t ssm_dtype;     /* gdn_state_dtype */
  float gated_norm_eps;  /* gated RMSNorm eps */
  float l2_eps;          /* q/k L2 norm: x / sqrt(sum(x^2) + l2_eps) */
  float q_scale;         /* multiplies the L2-normalised q */
} gdn_prefill_config;

typedef struct gdn_prefill gdn_prefill_t;

/* Device bytes of the workspace for this config; 0 if the config is invalid
 * or unsupported. It holds what a call prepares for every chunk of 64 tokens
 * (34 KB a value head and 256 x dk bytes a key head): 41 KB a token with 64
 * value and 16 key heads of 128; and up to 24 bytes a sequence. */
size_t gdn_prefill_workspace_bytes(const gdn_prefill_config* cfg);

/* Validate the config, bind the caller's workspace (256-byte aligned device
 * memory that outlives the handle) and clear its error word on `stream`. The
 * handle holds host state only. It belongs to the device that is current here;
 * calls with another one current are GDN_ERR_ARG. */
gdn_status gdn_prefill_create(const gdn_prefill_config* cfg, void* workspace, size_t workspace_bytes,
                              void* stream, gdn_prefill_t** out);

/* Causal depthwise conv1d over the C = 2*Hk*dk + Hv*dv channels, and SiLU:
 *   out[t][c] = silu(sum_{j<4} conv_w[c][j] x[t-3+j][c])
 * where rows before the sequence's first are the slot's three taps, oldest
 * first (zero when state_in <= 0). f32 sums, one rounding to bf16. The slot
 * state_out receives the sequence's last three inputs.
 * x [tokens][ldx >= C] bf16, out [tokens][ldo >= C] bf16, conv_w [C][4] bf16,
 * conv_state [num_slots][C][3] bf16. ldx and ldo are multiples of 8, pointers
 * 16-byte aligned. out must overlap no input. */
gdn_status gdn_prefill_conv(gdn_prefill_t* h, int32_t seqs, int32_t tokens, const void* x, int64_t ldx,
                            const void* conv_w, const int32_t* cu_seqlens, const int32_t* state_in,
                            const int32_t* state_out, void* conv_state, void* out, int64_t ldo,
                            void* stream);

/* The gated delta rule over every sequence, for each value head (value head h
 * reads key head h / (Hv/Hk)):
 *   k = k / sqrt(sum k^2 + l2_eps), q likewise and times q_scale,
 *   g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b),
 *   S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = S q,
 * and with z: core = o / sqrt(mean o^2 + gated_norm_eps) * gated_norm_w *
 * silu(z) per value head; without (z NULL, gated_norm_w ignored): core = o.
 * States, sums and gates are f32 throughout a sequence; a bf16 state is
 * rounded once, when it is stored. Sequences of up to 14 tokens run token by
 * token, all in f32. Longer ones run in chunks of 64 on the tensor cores, where
 * what is multiplied is two f16 terms, 22 bits (q and k as they are): on
 * ordinary inputs an f32 state ends within 2.3e-7 of the 64-bit result, token by
 * token within 0.6e-7. Within a chunk a row of the state keeps what is above
 * 2^-39 of the largest of its own values and of its state there, and q and k
 * what is above 2^-25 of the token's largest element (exact above 2^-17). A
 * caller that needs f32 products throughout passes a prompt in pieces of up to 14
 * tokens. The gate's SiLU is within a few 2^-22, and 0 where it is below 2^-126.
 * max_len is an upper bound of the sequences' lengths known to the host
 * (tokens if nothing better is known); sequences longer than it record
 * GDN_ERR_INDEX and are padding.
 * qkv [tokens][ldqkv >= C] bf16, rows q | k | v; z [tokens][ldz >= Hv*dv]
 * bf16 or NULL; ba [tokens][ldba >= 2*Hv] bf16, rows b | a; A_log [Hv] f32;
 * dt_bias [Hv] bf16; gated_norm_w [dv] bf16; ssm_state [num_slots][Hv][dv][dk]
 * f32 or bf16; core_out [tokens][ldcore >= Hv*dv] bf16. ldqkv, ldz and ldcore
 * are multiples of 8, the pointers of qkv, z, core_out, gated_norm_w and
 * ssm_state 16-byte aligned. core_out must overlap no input. One call at a time per handle
 * (its calls share the workspace; so do calls of gdn_prefill_conv with more than
 * 128 sequences among themselves). */
gdn_status gdn_prefill_delta(gdn_prefill_t* h, int32_t seqs, int32_t tokens, int32_t max_len,
                             const void* qkv, int64_t ldqkv, const void* z, int64_t ldz, const void* ba,
                             int64_t ldba, const float* A_log, const void* dt_bias,
                             const void* gated_norm_w, const int32_t* cu_seqlens,
                             const int32_t* state_in, const int32_t* state_out, void* ssm_state,
                             void* core_out, int64_t ldcore, void* stream);

/* Synchronise `stream` and read the sticky error word: GDN_OK or the first
 * recorded device status. *detail (optional) receives the raw word: bits
 * 31..24 status, 23..16 what (1 a state slot >= num_slots, 2 cu_seqlens not from
 * 0 on, out of order or past `tokens`, 3 a sequence longer than max_len, 4 a wait inside
 * the kernel that passed its limit), 15..0 the sequence. A sequence with an
 * index error is treated as padding; the others are not affected. Offsets that
 * lie outside the rows concern the two sequences that they bound alone. After
 * an offset that goes back, every sequence that starts before the largest
 * offset so far would have rows of an earlier one: it is padding as well, and
 * the sequence whose end went back is the one recorded. */
gdn_status gdn_prefill_check(gdn_prefill_t* h, void* stream, uint32_t* detail);

/* Clear the error word on `stream`. */
gdn_status gdn_prefill_reset(gdn_prefill_t* h, void* stream);

/* Free the host handle. The workspace stays the caller's. */
void gdn_prefill_destroy(gdn_prefill_t* h);

typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_GELU_TANH = 2 } gdn_activation;

/* out[m][n] = bf16(act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n]) with
 * f32 sums and one rounding. The sums are the tensor cores', which cut where an
 * f32 addition rounds: 1e-5 of the result at an inner size of 8192, a hundredth of
 * the last rounding. The activations are within a few 2^-22, and 0 where they
 * are below 2^-126. x [rows][ldx >= inner], w [cols][ldw >= inner],
 * bias [cols] or NULL, residual [rows][ldr >= cols] or NULL, out [rows][ldo >=
 * cols], all bf16. GELU is the tanh form. x and w are 16-byte aligned with ldx
 * and ldw multiples of 8; bias, residual and out have no alignment rule beyond
 * their type's. out may be residual itself (same pointer and stride) and must
 * overlap no other input. Non-finite values in x or w reach the outputs of
 * their own row or column only. No workspace, no handle. */
gdn_status gdn_linear(int32_t rows, int32_t cols, int32_t inner, const void* x, int64_t ldx, const void* w,
                      int64_t ldw, const void* bias, int32_t activation, const void* residual, int64_t ldr,
                      void* out, int64_t ldo, void* stream);

/* Synchronise `stream`, read the error word of this device's gdn_linear calls
 * and clear it: GDN_OK, or GDN_ERR_DEADLINE when a wait inside a kernel passed
 * its limit (the call's outputs are then not all written). *detail (optional)
 * receives the raw word, as for gdn_prefill_check. */
gdn_status gdn_linear_check(void* stream, uint32_t* detail);

/* Offsets, block tables and slots of a ragged step from its request lengths.
 * Request r holds context_lens[r] tokens in blocks of block_size slots (its
 * first ceil(context / block_size) table entries) and brings new_lens[r] more.
 * In request order each takes the blocks it still needs,
 *   need = ceil((context + new) / block_size) - ceil(context / block_size),
 * from the end of the free list (free_list[*free_count - 1] first), and its new
 * entries of block_table are written. Then
 *   cu_seqlens[r]  = sum of new_lens before r          [requests + 1]
 *   token_seq[t]   = the request of token t             [tokens]
 *   token_pos[t]   = its position, context + offset     [tokens]
 *   slots[t]       = block_table[r][pos / block_size] * block_size
 *                    + pos % block_size  (64 bits)      [tokens]
 *   *free_count_out = blocks left.
 * block_size 1 gives every token a slot of its own (a verify step's
 * state_out); a block_size no shorter than any request gives one block per
 * request (its state slot); in between, a paged cache.
 * Tokens at or past the last offset have request, position and slot -1; a sum
 * past `tokens` is cut there and recorded. A request with a negative length,
 * of more than max_blocks blocks or of more than 2^31 - 1 tokens gets no
 * blocks (a negative new length counts as 0 tokens, and a position stops at
 * 2^31 - 1); when the free list is short, so does the first request
 * that does not fit, and every later one that needs any. Their tokens' slots
 * are -1, no entry of theirs is written, and *error (a device word, optional)
 * receives GDN_ERR_INDEX in bits 31..24, what in 23..16 (1 a bad length, 2 the
 * free list is short, 3 more tokens than `tokens`) and the request in 15..0,
 * if it was zero. A free_count below 0 counts as 0 and above free_cap as
 * free_cap.
 * new_lens, context_lens int32 [requests]; block_table int32
 * [requests][max_blocks], updated; free_list int32 [free_cap]; free_count and
 * free_count_out int32, two different words. Outputs overlap no input. */
gdn_status gdn_slot_map(int32_t requests, int32_t tokens, const int32_t* new_lens,
                        const int32_t* context_lens, int32_t block_size, int32_t max_blocks,
                        int32_t* block_table, const int32_t* free_list, int32_t free_cap,
                        const int32_t* free_count, int32_t* free_count_out, int32_t* cu_seqlens,
                        int32_t* token_seq, int32_t* token_pos, int64_t* slots, uint32_t* error,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_PREFILL_H_ */
