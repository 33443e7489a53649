/*
 * conv_seq.h -- C ABI of the sequence operators: the causal depthwise
 * convolution, the gated linear recurrence and 8-bit activation checkpoints,
 * in the same library and with the same conventions as conv_fwd.h (element
 * types, error codes, streams, ownership: every buffer is the caller's, no
 * call allocates, synchronises or keeps anything).
 *
 * Sequences.  Tokens are rows of C channels, channels last.
 *  - A batch (cu == NULL): N sequences of L tokens each, [N, L, C].
 *  - Packed (cu != NULL): N sequences in one run of L rows, [L, C]; cu is a
 *    device array of N + 1 non-decreasing int32, sequence s being the rows
 *    cu[s] .. cu[s+1]-1 (it may be empty).  Rows in no sequence (behind the
 *    last, or before the first) are unused: never read into a result, and
 *    their output rows are left as they are, or with fill = 1 set to zero.
 *    cu is read on the device and not checked; entries that decrease or lie
 *    outside [0, L] give unspecified results but no access out of bounds.
 * N, L and the step functions' B may be 0; C is at least 1; none is above
 * 2^31 - 4097.  The step functions take at most 65535 blocks of 128 channels, of
 * 512 where C and the rows are aligned to four (CONV_EUNSUPPORTED).  A workspace
 * is in use until the call's kernels are done: calls that may overlap (other
 * streams, graphs replayed side by side) need one each.
 * Inputs documented with strides have unit channel stride, a token stride and
 * a batch stride in elements (batch stride unused when packed); every other
 * tensor is contiguous.  Buffers need only their element type's alignment;
 * 16-byte aligned rows run faster.  An output must not overlap an input or
 * another output (CONV_EALIAS), except where a state is said to be updated in
 * place.
 *
 * Checkpoints.  Where an argument has a `_scale` beside it and that is not
 * NULL, the tensor is an 8-bit checkpoint (act8_pack): `x` then points to its
 * int8 values and its strides count those; the scales are contiguous.
 */
#ifndef CONV_SEQ_H_
#define CONV_SEQ_H_

#include "conv_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- causal depthwise convolution ---------------------------------------
 *
 *   z[t, c] = bias[c] + sum_{j < K} w[c, j] * x[t - (K-1) + j, c]
 *   y[t, c] = z (CONV_ACT_NONE) or z / (1 + exp(-z)) (CONV_ACT_SILU)
 *
 * within each sequence: a cross-correlation along time that sees no later
 * token.  Rows before a sequence's first token come from its window `state`
 * [N, K-1, C] (oldest first), or are zero without one.  state_out (may be
 * NULL) receives each sequence's last K-1 rows, the window that continues it.
 * w: [C, K]; bias: [C] or NULL; x, w, bias, state, y of one type; 1 <= K <= 8.
 * Sums are fp32, rounded once. */
#define CONV_CAUSAL_MAX_K 8
enum { CONV_ACT_NONE = 0, CONV_ACT_SILU = 1 };

int conv_causal(const void* x, const void* w, const void* bias, const void* state, const int* cu, void* y,
                void* state_out, int N, long long L, int C, int K, long long x_batch, long long x_token,
                int activation, int fill, int dtype, conv_stream_t stream);

/* Its gradients.  From dy (with strides) and the forward pass's inputs (x may
 * be a checkpoint of type `dtype`): dx, dw [C, K], dbias [C] (NULL without
 * bias), dstate [N, K-1, C] (NULL, or the gradient of `state`; needs state).
 * dstate_out (may be NULL) is the gradient of the forward pass's state_out.
 * dw and dbias are sums over all tokens: fp32 partial sums of fixed ranges of
 * tokens in `workspace` (conv_causal_grad_workspace_size bytes, 16-byte
 * aligned), added in order, so a result is the same bits on every run.  Eight
 * ranges take K + 1 rows of C there, and in a batch each sequence has ranges of its
 * own: many sequences of a few tokens take less packed. */
int conv_causal_grad(const void* x, const unsigned char* x_scale, const void* w, const void* bias, const void* state,
                     const int* cu, const void* dy, const void* dstate_out, void* dx, void* dw, void* dbias,
                     void* dstate, int N, long long L, int C, int K, long long x_batch, long long x_token,
                     long long dy_batch, long long dy_token, int activation, int fill, int dtype, void* workspace,
                     unsigned long long workspace_bytes, conv_stream_t stream);
int conv_causal_grad_workspace_size(int N, long long L, int C, int K, int packed, unsigned long long* bytes);

/* One token for each of B sequences.  Row b uses window slot index[b] of
 * `state` [slots, K-1, C] (slot b when index is NULL), which is shifted by the
 * new row in place.  A row whose index is negative or >= slots is skipped: its
 * y row is left as it is (fill = 1: zero).  Rows that name one slot are taken
 * one after the other, in row order, as that sequence's consecutive tokens. */
int conv_causal_step(const void* x, const void* w, const void* bias, void* state, const int* index, void* y, int B,
                     int slots, int C, int K, long long x_token, int activation, int fill, int dtype,
                     conv_stream_t stream);

/* ---- gated linear recurrence ---------------------------------------------
 *
 *   s = sigmoid(r), g = sigmoid(i), a = exp(-decay * s)
 *   h[t] = a * h[t-1] + sqrt(1 - a^2) * g * x[t],   y[t] = h[t]
 *
 * for each channel within each sequence, from h0 [N, C] (fp32; zero if NULL).
 * decay: [C] fp32, >= 0; an infinite one counts as fp32's largest number.  A
 * sigmoid below fp32's least normal number (a gate under -87.3) is 0.  The state
 * and all sums are fp32; y is h rounded to the type of x, r and i.  h_last [N, C]
 * (fp32, may be NULL) receives each sequence's last state (h0 for an empty one).
 * states (fp32, may be NULL) receives the state in front of every
 * GATED_SCAN_STATE_EVERY-th token, [N, ceil(L/64), C] (packed: of every 64th row,
 * [ceil(L/64), C]): the backward pass starts from them.  Entries in front of a
 * sequence's first token, or of unused rows, are written but have no meaning. */
#define GATED_SCAN_STATE_EVERY 64

int gated_scan(const void* x, const void* r, const void* i, const float* decay, const float* h0, const int* cu, void* y,
               float* h_last, float* states, int N, long long L, int C, long long x_batch, long long x_token,
               long long r_batch, long long r_token, long long i_batch, long long i_token, int fill, int dtype,
               conv_stream_t stream);

/* Its gradients.  From dy (with strides), the forward pass's inputs (x, r and i
 * all tensors, or all contiguous checkpoints; CONV_EUNSUPPORTED where they are
 * mixed or strided) and its `states`: dx, dr, di (like y), ddecay
 * [C] and dh0 [N, C] (fp32; dh0 may be NULL).  dh_last (fp32, may be NULL) is
 * the gradient of h_last.  Where 1 - a^2 is below fp32's least normal number
 * (decay * s under 6e-39, or 0) it counts as 0, as in the forward pass, and the
 * square root's derivative is taken as 0.  ddecay is summed as dw above is, from a
 * row of C partial sums of each CTA: one at least of each sequence of a batch. */
int gated_scan_grad(const void* x, const unsigned char* x_scale, const void* r, const unsigned char* r_scale,
                    const void* i, const unsigned char* i_scale, const float* decay, const float* states,
                    const float* h0, const int* cu, const void* dy, const float* dh_last, void* dx, void* dr, void* di,
                    float* ddecay, float* dh0, int N, long long L, int C, long long x_batch, long long x_token,
                    long long r_batch, long long r_token, long long i_batch, long long i_token, long long dy_batch,
                    long long dy_token, int fill, int dtype, void* workspace, unsigned long long workspace_bytes,
                    conv_stream_t stream);
int gated_scan_grad_workspace_size(int N, long long L, int C, int packed, unsigned long long* bytes);

/* One token for each of B sequences, their states in h [slots, C] (fp32,
 * updated in place); index, skipped rows and repeated slots as for
 * conv_causal_step. */
int gated_scan_step(const void* x, const void* r, const void* i, const float* decay, float* h, const int* index, void* y,
                    int B, int slots, int C, long long x_token, long long r_token, long long i_token, int fill,
                    int dtype, conv_stream_t stream);

/* ---- 8-bit activation checkpoints ----------------------------------------
 *
 * Each row's channels in blocks of 32 (the last may be shorter).  A block has
 * one power of two 2^e, the least with |x| <= 127 * 2^e for all its elements
 * and e >= -126, and its elements are q = x / 2^e rounded to the nearest
 * integer (ties to even), held within the type's largest value: x is given
 * back as q * 2^e, off by at most 2^(e-1), or by less than 2^e where the nearest
 * is past that value (65504 in f16 is 63 * 2^10).  scale holds e + 127; 0 for a block
 * of zeros; 255 for a block with an infinity or NaN, whose elements all come
 * back as NaN (q = 0 there).
 * x: [rows, C] with a row stride; q: [rows, C] int8; scale: [rows, ceil(C/32)]
 * uint8; both contiguous. */
#define ACT8_BLOCK 32

int act8_pack(const void* x, signed char* q, unsigned char* scale, long long rows, int C, long long x_row, int dtype,
              conv_stream_t stream);
int act8_unpack(const signed char* q, const unsigned char* scale, void* y, long long rows, int C, int dtype,
                conv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_SEQ_H_ */
