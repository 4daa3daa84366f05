/*
 * ninfer_layer.h -- the operators that complete a model's step around the
 * projections (ninfer_ternary.h), the cache and the logit controls
 * (ninfer_decode.h); same library, libninfer_ternary.so:
 *
 *   ninfer_norm                  root-mean-square norm, with the residual's addition and a gate
 *   ninfer_rotary                rotary positions of queries and keys, with their norms
 *   ninfer_rotary_frequencies    the table of frequencies it reads (host), scaled for long contexts
 *   ninfer_gated_delta           the gated delta rule over a state per head: single tokens and prompts
 *   ninfer_sample                the next token: temperature, top-k, top-p, min-p, given random numbers
 *
 * The conventions are those of ninfer_decode.h: an ninfer_status comes back; on
 * any but NINFER_OK nothing was launched or written; device work is asynchronous
 * on the caller's stream, in programmatic dependent launches that touch no buffer
 * before the preceding work is done; no memory is allocated and no pointer kept.
 * Sizes and strides are element counts. Values that only the device sees
 * (positions, offsets, slots, controls) never take an access out of the buffers.
 */
#ifndef NINFER_LAYER_H
#define NINFER_LAYER_H

#include "ninfer_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more bit of *status. */
enum {
    NINFER_DELTA_BAD_SLOT = 64    /* gated delta: a slot at or past `slots` */
};

/*
 * ninfer_norm -- for every group of `group` neighbouring elements of every row:
 *   s = x + residual (residual NULL: x),  sum = round(s),
 *   out = round(s / sqrt(mean of s^2 + eps) * (weight[e] + weight_offset) * gate / (1 + e^-gate))
 * with e the element's place in its group (weight NULL: 1 for weight + offset; gate NULL: no gate). All in fp32; s enters the
 * norm unrounded. A row of one group is a hidden state, `cols / group` groups are the heads of a row.
 *   x, residual, gate, sum, out: device, row r at r * their own stride, f32, bf16 or f16 each; sum has the
 *     residual's type and may be the residual itself (same stride), out may be x or gate (same stride and
 *     type); outputs overlap neither each other nor anything else. sum NULL: not written (it needs a residual).
 *   weight: device, `group` elements. eps >= 0; weight_offset finite (1 for weights stored around zero).
 * Rows whose bases and strides are multiples of 16 bytes, with groups of a multiple of 8, are the fast ones.
 * Errors: INVALID_ARGUMENT, SHAPE (rows, cols or group 0; cols no multiple of group; a stride below cols),
 *   ALIGNMENT (a pointer not aligned to its element), OVERFLOW (rows * groups over 2^31 - 1).
 */
typedef struct {
    const void *x, *residual, *gate, *weight;
    void *sum, *out;
    uint64_t rows, cols, group;
    uint64_t x_stride, residual_stride, gate_stride, sum_stride, out_stride;
    float eps, weight_offset;
    int32_t x_dtype, residual_dtype, gate_dtype, weight_dtype, out_dtype, reserved;   /* reserved: 0 */
} ninfer_norm_args;

int ninfer_norm(const ninfer_norm_args *args, ninfer_stream stream);

/*
 * ninfer_rotary -- every head of q and k turned by its token's position, pair by pair:
 *   h = x (with weights: x / sqrt(mean of x^2 + eps) * (weight + weight_offset) over the head),
 *   a = h[i], b = h[i + rotary_dim / 2]   (interleaved: h[2 i], h[2 i + 1]),   i < rotary_dim / 2,
 *   angle = 2 pi * positions[t] * frequencies[i] / 2^64,
 *   a' = magnitude * (a cos - b sin),  b' = magnitude * (b cos + a sin); elements from rotary_dim on stay h.
 * The fraction of a turn is exact (products of whole numbers modulo 2^64), so that far positions lose nothing.
 *   q, k, q_out, k_out: device, one dtype (f32, bf16, f16), element e of head h of token t at
 *     t * token_stride + h * head_stride + e, each with strides of its own, multiples of 16 bytes; an output may be its
 *     input (same strides), and overlaps nothing else that the call reads or writes. k NULL: queries alone.
 *   positions: device int32[tokens]; a token with a negative one is left out: nothing of it is written.
 *   frequencies: device uint64[rotary_dim / 2], turns a position times 2^64.
 *   q_weight, k_weight: device, head_dim elements of weight_dtype; NULL: no norm. magnitude, weight_offset
 *     finite, eps >= 0.
 *   head_dim: a multiple of 8 up to 256; rotary_dim: even, 2 .. head_dim.
 * Errors: INVALID_ARGUMENT, SHAPE, ALIGNMENT, OVERFLOW.
 *
 * ninfer_rotary_frequencies -- host: that table from f_i = base^(-2 i / rotary_dim) radians a position, and the magnitude:
 *   NINFER_ROTARY_NONE        f_i; magnitude 1
 *   NINFER_ROTARY_LINEAR      f_i / factor; magnitude 1
 *   NINFER_ROTARY_DIMENSIONS  (1 - r) f_i + r f_i / factor, r rising from 0 to 1 in i between the pair that turns `fast`
 *                             times within `context` positions and the one that turns `slow` times (rounded outwards);
 *                             magnitude 0.1 ln(factor) + 1
 *   NINFER_ROTARY_TURNS       the same with r falling from 1 to 0 in the turns context f_i / (2 pi) between slow and fast; magnitude 1
 *   base > 1; factor >= 1; context > 0 and 0 < slow < fast for the last two.
 */
typedef enum {
    NINFER_ROTARY_NONE = 0,
    NINFER_ROTARY_LINEAR = 1,
    NINFER_ROTARY_DIMENSIONS = 2,
    NINFER_ROTARY_TURNS = 3
} ninfer_rotary_scaling;

typedef struct {
    const void *q, *k, *q_weight, *k_weight;
    void *q_out, *k_out;
    const int32_t *positions;
    const uint64_t *frequencies;
    uint64_t tokens, q_heads, kv_heads, head_dim, rotary_dim;
    uint64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
    uint64_t q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride;
    float magnitude, eps, weight_offset;
    int32_t dtype, weight_dtype, interleaved;
} ninfer_rotary_args;

int ninfer_rotary_frequencies(uint64_t rotary_dim, double base, int scaling, double factor, double context, double slow,
                              double fast, uint64_t *frequencies, float *magnitude);
int ninfer_rotary(const ninfer_rotary_args *args, ninfer_stream stream);

/*
 * ninfer_gated_delta -- the gated delta rule. Every value head h of a request has a state S of k_dim x v_dim;
 * for each of the request's tokens, in order, with key head h / (v_heads / k_heads):
 *   S <- e^log_decay S;  u = beta (v - S^T k);  S <- S + k u^T;  out = scale S^T q
 * (norm_eps >= 0: with q / sqrt(sum of q^2 + norm_eps) for q and the same for k; negative: as they are).
 *   q, k: device, element e of head h of token t at t * token_stride + h * head_stride + e, k_heads heads of k_dim;
 *   v: the same with v_heads heads of v_dim; one dtype (f32, bf16, f16), strides multiples of 16 bytes.
 *   log_decay, beta: device float, token t at t * decay_stride (beta_stride), v_heads elements. Natural logarithms,
 *     at most 0 in earnest.
 *   state: device float, head h of slot s at s * slot_stride + h * k_dim * v_dim, [k_dim][v_dim], read and written in
 *     place; slot_stride a multiple of 4 and at least v_heads * k_dim * v_dim.
 *   state_slots: device int32[requests] (NULL: request i has slot i); a negative one leaves the request out, one at or past
 *     `slots` does so and sets NINFER_DELTA_BAD_SLOT. Slots of one call differ from each other (the results of requests that
 *     share one are undefined).
 *   offsets: device int32[requests + 1], tokens offsets[i] .. offsets[i + 1] - 1 belong to request i (cut to
 *     [0, tokens]) and to no other (the results of requests that share some are undefined); NULL: one token each, token i of request i (tokens = requests).
 *   lengths: device int32[requests], tokens that the request's state has seen; one that has seen none (0 and less) begins
 *     with zeros, whatever its slot holds. NULL: every state is read.
 *   out: device [tokens][v_heads][v_dim] of out_dtype; rows of no request are left as they were, and so are the states of
 *     requests without tokens.
 *   workspace: with offsets, device, 256-byte aligned, at least ninfer_gated_delta_workspace() bytes; its contents need no
 *     initial value and are not preserved, and no other call may use it at the same time. Without offsets it is not used (NULL will do).
 *     It grows by what 32 tokens take (1.1 MB with 16 key and 48 value heads of 128: 270 MB for a prompt of 8001 tokens), whatever the type.
 *     A prompt that is given in parts of multiples of 32 tokens, one call after another with the same state, has the same results.
 *   out may be v itself (of one dtype, v without gaps). Beside that out, state, status and workspace overlap nothing that the call reads or writes.
 *   k_dim, v_dim: multiples of 8 up to 256; v_heads a multiple of k_heads; scale finite.
 * States and sums are fp32. With offsets, a request's tokens go 32 at a time through the tensor cores: operands hold 22 bits of each
 * value (q and k of 16-bit types all of theirs). Each token's q and k has a scale of its own, for each column of a state the state, the values
 * and what the tokens add to it have one: nothing counts that is under 2^-38 of the largest state, value or addition of its column among those 32
 * tokens, before it or behind it. (Without offsets there is no such limit.) Infinities and NaN make NaN of what the formulas give them to, and reach no earlier
 * token, other column, head or request, as long as finite operands' products are within fp32's range. No bit of a request's results
 * depends on the others of the call. (Without offsets the order of sums goes by the number of states.)
 * If a kernel's bounded wait runs out (ninfer_set_wait_limit), the device error word is set and the results are incomplete.
 * Errors: INVALID_ARGUMENT, SHAPE, SIZE_MISMATCH (workspace), ALIGNMENT, OVERFLOW, CUDA.
 */
typedef struct {
    const void *q, *k, *v;
    const float *log_decay, *beta;
    float *state;
    const int32_t *state_slots, *offsets, *lengths;
    void *out;
    int32_t *status;
    uint64_t tokens, requests, slots, k_heads, v_heads, k_dim, v_dim;
    uint64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    uint64_t decay_stride, beta_stride, slot_stride;
    float scale, norm_eps;
    int32_t dtype, out_dtype;
} ninfer_gated_delta_args;

int ninfer_gated_delta_workspace(uint64_t tokens, uint64_t requests, uint64_t k_heads, uint64_t v_heads, uint64_t k_dim,
                                 uint64_t v_dim, uint64_t *bytes);
int ninfer_gated_delta(const ninfer_gated_delta_args *args, void *workspace, uint64_t workspace_bytes, ninfer_stream stream);

/*
 * ninfer_sample -- one token for every row of logits x, m the row's largest (NaN counts as -infinity, and tokens
 * of -infinity take no part):
 *   w_v = e^((x_v - m) / temperature);  the tokens in falling order of x, equal ones in rising order of v;
 *   A = the first top_k of them (top_k <= 0: all),
 *   B = the shortest beginning of A whose w add up to at least top_p times A's sum (top_p >= 1 or NaN: A; <= 0: the first),
 *   C = those of B with w_v >= min_p (NaN: all; at most 1 counts);
 *   token = the first v of C, in rising order of v, for which the w of C up to and with v add up to more than random * (C's sum);
 *   logprob = ln(w_token / C's sum).
 * temperature <= 0 (or NaN): the largest logit, the lowest of equal ones, logprob 0; one below 2^-119 counts as that. A row without a logit above
 * -infinity: token -1, logprob -infinity. If m is +infinity, w is 1 where x is and 0 elsewhere.
 *   logits: device, dtype f32, bf16 or f16, row b at b * stride.
 *   temperature, top_p, min_p: device float[rows], NULL: 1, 1, 0; top_k: device int32[rows], NULL: 0.
 *   random: device float[rows], in [0, 1) (cut to it).
 *   tokens: device int32[rows]; logprobs: device float[rows] or NULL. Each may be one of the controls' arrays; else they overlap nothing.
 * Weights are whole multiples of 2^(vocab's bits - 62) of the largest one, each off by less than 2^-29 and the rounding of x - m (2^-24 of
 * the exponent; 0 where x - m overflows) of itself; their sums are exact and do not depend on an order: equal rows give equal tokens, however they are divided.
 * Errors: INVALID_ARGUMENT, SHAPE (rows or vocab 0, vocab over 2^30, stride below vocab), ALIGNMENT, OVERFLOW, CUDA.
 */
typedef struct {
    const void *logits;
    const float *temperature, *top_p, *min_p;
    const int32_t *top_k;
    const float *random;
    int32_t *tokens;
    float *logprobs;
    uint64_t rows, vocab, stride;
    int32_t dtype, reserved;   /* reserved: 0 */
} ninfer_sample_args;

int ninfer_sample(const ninfer_sample_args *args, ninfer_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* NINFER_LAYER_H */
