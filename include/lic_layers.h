/*
 * lic_layers.h -- C ABI of the gfx950 (MI355X) network operators that stand
 * around the coder of rans_hip.h in a learned image codec: group norm with an
 * activation (transforms), RMS norm with the residual's addition, rotary
 * positions, attention and linear attention (entropy models over the latent's
 * positions), each forward and backward, and clipping of gradients.
 *
 * Memory and ownership are the coder's: every array is a DEVICE pointer owned
 * by the caller, the library allocates nothing and keeps no state, all work
 * is enqueued on `hstream` and no call synchronises with the host.
 * `workspace` is device memory of at least the matching *_workspace_bytes,
 * 256-byte aligned; it needs no filling and keeps nothing from one call to the
 * next.  Calls that share a workspace or an output must not overlap in time.
 *
 * Results do not depend on timing nor on where the values lie (addresses, strides):
 * every sum is taken in an order that a call's sizes, windows and key lengths
 * alone decide, so an encoder and a decoder that make the same call get the same
 * bits.  Calls of other sizes take other orders: a position by itself (a single
 * token over a cache, another batch) differs in its last bits from the same
 * position within a longer call, so a decoder that steps needs an encoder that
 * steps.
 *
 * Errors: the return value is a rans_status.  Sizes, pointers and types are
 * checked on the host before any launch (RANS_E_ARG, RANS_E_WORKSPACE); a
 * failed launch is RANS_E_HIP.  The data cannot make a call fail, with one
 * exception that lic_rotary reports in *status.
 *
 * Strides are in elements and at least 0; the innermost extent (channels, a
 * head's values) always has stride 1.  Outputs have to be free of overlap.
 */
#ifndef LIC_LAYERS_H
#define LIC_LAYERS_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "rans_hip.h"

#ifdef __cplusplus
extern "C" {
#endif

enum lic_dtype { LIC_F32 = 0, LIC_F16 = 1, LIC_BF16 = 2 };

enum lic_activation { LIC_ACT_NONE = 0, LIC_ACT_RELU = 1, LIC_ACT_SILU = 2, LIC_ACT_GELU = 3 };

/* ---- group norm with an activation, channels last ----------------------
 *
 * x holds `samples` samples of `positions` rows of `channels` values; row p
 * of sample n starts at x + n * x_sample + p * x_row (elements).  The channels
 * form `groups` groups of channels / groups neighbours, and
 *   mean, var  over a group's values of one sample (var without Bessel's
 *              correction), rstd = 1 / sqrt(var + eps)
 *   y = act(weight[c] * (x - mean) * rstd + bias[c]).
 * weight and bias (param_dtype, `channels` values each) may be null for 1 and
 * 0.  mean and rstd (float, samples * groups) are outputs that the backward
 * call takes.  gelu is u * Phi(u), the Gaussian's own distribution function.
 *
 * Statistics and sums are held in 32 bits; the sums of squares are taken
 * about a value of the data, so a large mean costs no precision.
 *
 * The backward call gives dx, and dweight and dbias (param_dtype; either may
 * be null) summed over samples and positions. */
#define LIC_MAX_CHANNELS 65536
#define LIC_MAX_SAMPLES 65535

uint64_t lic_group_norm_workspace_bytes(int32_t samples, int64_t positions, int32_t channels,
                                        int32_t groups);

int lic_group_norm_forward(const void *x, int64_t x_sample, int64_t x_row, int32_t samples,
                           int64_t positions, int32_t channels, int32_t groups, int32_t dtype,
                           const void *weight, const void *bias, int32_t param_dtype, float eps,
                           int32_t activation, void *y, int64_t y_sample, int64_t y_row,
                           float *mean, float *rstd, void *workspace, uint64_t workspace_bytes,
                           hipStream_t hstream);

int lic_group_norm_backward(const void *dy, int64_t dy_sample, int64_t dy_row, const void *x,
                            int64_t x_sample, int64_t x_row, int32_t samples, int64_t positions,
                            int32_t channels, int32_t groups, int32_t dtype, const void *weight,
                            const void *bias, int32_t param_dtype, int32_t activation,
                            const float *mean, const float *rstd, void *dx, int64_t dx_sample,
                            int64_t dx_row, void *dweight, void *dbias, void *workspace,
                            uint64_t workspace_bytes, hipStream_t hstream);

/* ---- RMS norm with the residual's addition ------------------------------
 *
 * x holds `samples` x `positions` rows of `channels` values next to each other; every
 * array of such rows has strides of its own (sample, row).
 *   h = x + residual, rounded to their type (residual null: h = x)
 *   rstd = 1 / sqrt(mean over the row of h^2 + eps),  y = weight[c] h rstd
 * weight (param_dtype) may be null for 1.  sum receives h; it has to be null where
 * residual is.  rstd (float [samples][positions]) may be null in the forward call; the
 * backward call takes it, and h as x:
 *   a = weight dy,  dx = rstd (a - xh mean(a xh)) + dsum,  dweight = sum over rows of dy xh
 * with xh = h rstd; dx is the gradient of x and of residual alike, dsum the one
 * that comes to h from elsewhere (null: 0).  dweight (param_dtype) may be null.
 * An output may be an input of the same strides (y and sum: x or residual; dx: dy or dsum).
 * y and sum must not overlap each other, and y in 8 bits no input.
 *
 * format != LIC_FORMAT_NONE (forward only): y has one byte a value, an e4m3 number (up
 * to 448) or a whole number (up to 127), and scales (float [samples][positions]) what
 * one stands for:
 *   top = max(max over the row of |weight h rstd|, 1e-30), scale = top / most,
 *   y = round(weight h rstd * (most / top)), ties to even
 * Where a row of weight h rstd is not all finite, neither is its scale, and all that the row
 * stands for is NaN.  Sums are held in 32 bits; a row whose squares overflow them has an rstd of 0. */
enum lic_format { LIC_FORMAT_NONE = 0, LIC_FORMAT_E4M3 = 1, LIC_FORMAT_INT8 = 2 };

typedef struct lic_rms_norm_args {
    const void *x, *residual, *weight;
    void *y, *sum;
    float *rstd, *scales;
    const void *dy, *dsum;
    void *dx, *dweight;
    int64_t x_stride[2], residual_stride[2], y_stride[2], sum_stride[2]; /* sample, row */
    int64_t dy_stride[2], dsum_stride[2], dx_stride[2];
    int64_t samples, positions, channels, dtype, param_dtype, format;
    double eps;
} lic_rms_norm_args;

/* Bytes for lic_rms_norm_backward with a dweight (without one none are needed). */
uint64_t lic_rms_norm_workspace_bytes(int64_t samples, int64_t positions, int64_t channels);

int lic_rms_norm_forward(const lic_rms_norm_args *args, hipStream_t hstream);

int lic_rms_norm_backward(const lic_rms_norm_args *args, void *workspace, uint64_t workspace_bytes,
                          hipStream_t hstream);

/* ---- rotary positions ---------------------------------------------------
 *
 * lic_rotary_table: cosine and sine of every angle, once for a model.  Row r
 * has `axes` coordinates coords[r * axes ..] (double: a token's index, or an
 * image position's row and column); the pairs = rotary_dim / 2 angles of a
 * row are split evenly over the axes (pairs must divide by axes), and the
 * j-th of an axis' n is
 *   coordinate * freq_j,  freq_j = base^(-j / n) * (g_j + (1 - g_j) / factor)
 * with g_j = 1 for no scaling (factor 1), 0 for linear interpolation by
 * `factor` (low >= high), else the ramp clamp((turns_j - low) / (high - low),
 * 0, 1), turns_j = original * base^(-j / n) / (2 pi): angles that turn often
 * within the `original` length stay, slow ones are interpolated.  Cosine and
 * sine are multiplied by `amplitude`.  Angles are formed and reduced in double
 * precision: in single precision a position of a million would be off by
 * a twentieth of a radian.  cos, sin: float [rows][pairs].
 *
 * lic_rotary: of each head's `dim` values the first rotary_dim form pairs,
 * (j, j + rotary_dim / 2) or, with interleaved != 0, (2 j, 2 j + 1), and
 *   a' = a cos - b sin, b' = a sin + b cos
 * with row positions[b * pos_batch + s] of the tables (positions null: row s);
 * the others are copied.  inverse != 0 takes -sin, which is also the
 * gradient.  Both q (heads) and k (kv_heads; k may be null with kv_heads 0)
 * are done in one launch; an output may be its input.  A position outside
 * [0, table_rows) gives a token of NaN and *status = RANS_E_INDEX; status may
 * be null, and otherwise is only ever written in that case. */
typedef struct lic_rotary_args {
    const void *q, *k;
    void *q_out, *k_out;
    const float *cos, *sin;
    const int32_t *positions;
    int32_t *status;
    int64_t pos_batch;
    int64_t q_stride[3], k_stride[3], q_out_stride[3], k_out_stride[3]; /* batch, token, head */
    int64_t batch, tokens, heads, kv_heads, dim, rotary_dim, table_rows;
    int64_t dtype, interleaved, inverse;
} lic_rotary_args;

int lic_rotary_table(const double *coords, int64_t rows, int32_t axes, int32_t rotary_dim,
                     double base, double factor, double low, double high, double original,
                     double amplitude, float *cos, float *sin, hipStream_t hstream);

int lic_rotary(const lic_rotary_args *args, hipStream_t hstream);

/* ---- attention -----------------------------------------------------------
 *
 * q, out, dout, dq are [batch][queries][heads][dim], k, v, dk, dv
 * [batch][keys][kv_heads][dim] with any batch, row and head strides; heads is
 * a multiple of kv_heads and head h reads kv head h / (heads / kv_heads).
 *   s_ij = scale q_i . k_j,  lse_i = log sum_j exp s_ij,  p_ij = exp(s_ij - lse_i),
 *   out_i = sum_j p_ij v_j                       over the visible j.
 * Batch b has n = key_lengths[b] keys (all of them where key_lengths is null;
 * held to [0, keys]) and its queries are its last positions: query i stands at
 * i + n - queries.  Key j < n is visible to a query at position t unless
 * window_left >= 0 and j < t - window_left, or window_right >= 0 and
 * j > t + window_right (0: causal), or mask (one byte an entry, strides by
 * batch, head, query and key, 0 to share it) holds 0 there.
 *
 * A key that a query does not see has no part in that query's row, nor the
 * query in its gradients, whatever their values: NaN and infinity in masked
 * places stay there.  Rows past key_lengths[b] are not read; their dk and dv
 * are 0.  A query that sees no key gives out 0, lse -inf and no gradient.
 *
 * lse is float [batch][heads][queries].  Scores, sums and accumulators are held
 * in 32 bits, products of 32-bit inputs in 32 bits; probabilities (and, in the
 * backward call, their gradients) are rounded to q's type for the second
 * product, as its operands; in half precision a power of two of each row lifts those
 * gradients there, so their precision does not depend on the size of dout or v.
 *
 * dim is 1 .. 128 (16-bit types: vector loads for multiples of 8, with strides and
 * addresses to match; 32-bit: of 4), scale positive.  The backward call recomputes
 * the probabilities from q, k and lse and takes what the forward call took. */
#define LIC_MAX_HEAD_DIM 128

typedef struct lic_attention_args {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const void *dout;
    void *dq, *dk, *dv;
    const uint8_t *mask;
    const int32_t *key_lengths;
    int64_t q_stride[3], k_stride[3], v_stride[3]; /* batch, row, head */
    int64_t out_stride[3], dout_stride[3], dq_stride[3], dk_stride[3], dv_stride[3];
    int64_t mask_stride[4];
    int64_t batch, queries, keys, heads, kv_heads, dim;
    int64_t dtype, window_left, window_right;
    double scale;
} lic_attention_args;

/* Bytes for lic_attention_forward (backward == 0) or lic_attention_backward of these
 * sizes and windows: batch, queries, keys, heads, kv_heads, dim, dtype, window_left and
 * window_right are read and have to be the call's (other windows split the work otherwise).
 * 0 is possible: the workspace may then be null; it is also the answer to sizes or windows
 * that a call refuses. */
uint64_t lic_attention_workspace_bytes(const lic_attention_args *args, int32_t backward);

int lic_attention_forward(const lic_attention_args *args, void *workspace,
                          uint64_t workspace_bytes, hipStream_t hstream);

int lic_attention_backward(const lic_attention_args *args, void *workspace,
                           uint64_t workspace_bytes, hipStream_t hstream);

/* ---- linear attention with a decay for each head ------------------------
 *
 * q, out, dout, dq are [batch][tokens][heads][..], k, v, dk, dv
 * [batch][tokens][kv_heads][..] with any batch, row and head strides; q and k have
 * `dim` values, v and out `value_dim`; heads is a multiple of kv_heads and head h
 * reads kv head h / (heads / kv_heads).  With g = exp(log_decay[head]) and a state of
 * dim x value_dim numbers for each batch and head,
 *   S_t = g S_(t-1) + k_t v_t',   out_t = scale q_t S_t
 * that is out_t = scale (sum over s <= t of g^(t-s) (q_t . k_s) v_s + g^(t+1) q_t S_(-1)),
 * where S_(-1) is `state` (null: 0) and state_out (may be null) receives the last S.
 * state_out may be `state` itself, with its strides; no other output may be an input.
 * lengths (null: all) are the tokens in use of each batch, held to [0, tokens]: the state
 * stops there, rows behind it are not read, and their out (dq, dk, dv) is 0.
 *
 * A token has no part in what comes before it, whatever its values are: a NaN or an
 * infinity shows from its own row on (in gradients: up to it).
 *
 * States are float, [batch][head][dim][value_dim] with strides by batch, head and
 * row of their own.  Sums and states are held in 32 bits, and a state that leaves the call has
 * that precision.  16-bit types: an operand that is no input (a power of g times one, a score,
 * a state) goes into a product as parts of q's type that add up to it: off by 2^-17 in
 * bfloat16 and 2^-23 in half precision in what forms outputs and gradients of q's type,
 * which are rounded once at the end, and by less in states that leave the call.  In half
 * precision a power of two lifts each column of a state (of what it takes in), and each token's
 * scores, so this holds for values of any size that are not below 2^-16 of the largest beside them
 * (the smaller are off by 2^-38 of that).  Products of 32-bit inputs are in 32 bits.
 *
 * The backward call takes what the forward call took, dout, and dstate, the gradient
 * that comes to state_out (null: 0).  dlog_decay (float [heads], summed over the batch)
 * and dstate_in (the gradient of `state`) may be null.  dk and dv of heads that share a
 * kv head are their sums.
 *
 * Long calls of few heads are split along the tokens; how is decided by the sizes
 * alone.  tokens up to 2^28, dim and value_dim 1 .. 128, scale positive. */
typedef struct lic_linear_attention_args {
    const void *q, *k, *v;
    const float *log_decay, *state;
    const int32_t *lengths;
    void *out;
    float *state_out;
    const void *dout;
    const float *dstate;
    void *dq, *dk, *dv;
    float *dlog_decay, *dstate_in;
    int64_t q_stride[3], k_stride[3], v_stride[3], out_stride[3]; /* batch, row, head */
    int64_t dout_stride[3], dq_stride[3], dk_stride[3], dv_stride[3];
    int64_t state_stride[3], state_out_stride[3], dstate_stride[3], dstate_in_stride[3]; /* batch, head, row */
    int64_t batch, tokens, heads, kv_heads, dim, value_dim, dtype;
    double scale;
} lic_linear_attention_args;

/* Bytes for lic_linear_attention_forward (backward == 0) or lic_linear_attention_backward:
 * batch, tokens, heads, kv_heads, dim, value_dim and dtype are read. */
uint64_t lic_linear_attention_workspace_bytes(const lic_linear_attention_args *args, int32_t backward);

int lic_linear_attention_forward(const lic_linear_attention_args *args, void *workspace,
                                 uint64_t workspace_bytes, hipStream_t hstream);

int lic_linear_attention_backward(const lic_linear_attention_args *args, void *workspace,
                                  uint64_t workspace_bytes, hipStream_t hstream);

/* ---- clipping of gradients by their global norm --------------------------
 *
 *   norm = sqrt(sum over all values of all tensors of x^2)
 *   out = x * min(1, max_norm / (norm + 1e-6))
 * `tensors` is a HOST array of `count` entries, read before the call returns; x and out
 * (which may be x) are device memory of n values next to each other, each of its own
 * type.  Outputs must not overlap each other, nor an x but their own.  norm is one float on
 * the device.  Squares are summed and the factor is formed in 64 bits, so no size of the values
 * overflows or leaves the factor without its bits (a norm past 32 bits' range is written as infinity).  An infinity
 * among the values makes the factor 0 (and itself NaN), a NaN makes all outputs NaN.
 * lic_gradient_norm leaves `out` alone (it may be null). */
typedef struct lic_gradient {
    const void *x;
    void *out;
    int64_t n, dtype;
} lic_gradient;

uint64_t lic_clip_gradients_workspace_bytes(const lic_gradient *tensors, int64_t count);

int lic_gradient_norm(const lic_gradient *tensors, int64_t count, float *norm, void *workspace,
                      uint64_t workspace_bytes, hipStream_t hstream);

int lic_clip_gradients(const lic_gradient *tensors, int64_t count, double max_norm, float *norm,
                       void *workspace, uint64_t workspace_bytes, hipStream_t hstream);

/* Static text that names the library's build target. */
const char *lic_layers_target(void);

#ifdef __cplusplus
}
#endif

#endif /* LIC_LAYERS_H */
