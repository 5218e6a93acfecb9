/*
 * fm_ops.h -- C ABI of the frame models' operators (GB300, sm_103a).
 *
 * What a model over mel frames needs next to the spectrogram of fm_mel.h:
 * layer norm, a learned position bias by distance buckets, and attention
 * whose scores may be capped, biased by distance and masked by recording; for
 * recurrent blocks root-mean-square norm with the residual's addition, a gated
 * linear layer and a gated recurrence; each with its backward pass, and the norm
 * and the gated layer in 8 bits for serving. Same library (libfm_mel.so), same conventions
 * as fm_mel.h: errors come back as fm_status, nothing is thrown or printed, a
 * failing call has no side effects, work is queued on `stream` and nothing is
 * allocated (callers pass workspaces whose sizes the *_workspace calls give).
 * A call needs its device current. Results are the same bits on every call:
 * no sum's order depends on timing.
 *
 * Element types: FM_F32, FM_F16 and FM_BF16. Every sum, mean, softmax
 * statistic and gradient sum is held in 32 bits.
 */
#ifndef FM_OPS_H
#define FM_OPS_H

#include "fm_mel.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Layer norm over the last dimension:
 *   y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(var + eps)
 * with mean and var = mean((x - mean)^2) of each row.
 *
 *   rows, width : rows >= 0, width 1 .. 2^24.
 *   dtype       : type of x, y, dy and dx.
 *   param_dtype : type of weight, bias, dweight and dbias: dtype or FM_F32.
 *   *_stride    : elements between rows, >= width (any for rows <= 1); the
 *                 elements of a row are adjacent.
 *   weight,bias : [width]; NULL means ones / zeros.
 *   mean, rstd  : [rows] f32; forward writes them (NULL: not wanted),
 *                 backward reads them.
 *   dx, dweight, dbias : each may be NULL where it is not wanted.
 *   workspace   : backward only, fm_layer_norm_workspace() bytes, 16-byte
 *                 aligned (needed where dweight or dbias is wanted).
 */
typedef struct {
  int64_t rows, width;
  int64_t dtype, param_dtype;
  int64_t x_stride, y_stride, dy_stride, dx_stride;
  double eps;
  const void *x, *weight, *bias;
  void* y;
  float *mean, *rstd;
  const void* dy;
  void *dx, *dweight, *dbias;
  void* workspace;
  int64_t workspace_bytes;
} fm_layer_norm_args;

fm_status fm_layer_norm_forward(const fm_layer_norm_args* args, fm_stream_t stream);
fm_status fm_layer_norm_backward(const fm_layer_norm_args* args, fm_stream_t stream);
int64_t fm_layer_norm_workspace(const fm_layer_norm_args* args);

/* ------------------------------------------------------------------------
 * Distance buckets. An offset is a key's place minus a query's. With
 * side = num_buckets / 2 where both directions have buckets of their own
 * (bidirectional; num_buckets even) and num_buckets otherwise, e = side / 2,
 * L = side - e and n the distance (|offset|, or max(-offset, 0) one-sided):
 *   bucket = n                                        for n < e
 *   bucket = e + the largest m <= L - 1 with n^L >= e^(L-m) * max_distance^m
 * (the whole-number form of e + floor(L log(n/e) / log(max_distance/e))), and
 * `side` more for keys after the query where bidirectional.
 *
 * fm_buckets_create builds the map for the offsets -max_distance ..
 * max_distance (beyond them it is constant) in whole numbers on the host and
 * copies it to the current device (it waits for that copy alone; allowed while a
 * graph is being recorded); the handle is read-only afterwards, usable
 * from several threads and streams on that device, and owned by the caller
 * until fm_buckets_destroy.
 *   num_buckets  : 4 .. 4096 bidirectional (even), 2 .. 4096 one-sided.
 *   max_distance : e + 1 .. 2048.
 * fm_buckets_map copies the map, 2 * max_distance + 1 int32, to host memory.
 */
typedef struct fm_buckets fm_buckets;
fm_status fm_buckets_create(fm_buckets** out, int num_buckets, int max_distance, int bidirectional);
fm_status fm_buckets_map(const fm_buckets* buckets, int32_t* map);
fm_status fm_buckets_destroy(fm_buckets* buckets);

/*
 * The dense bias:  out[h][i][j] = table[bucket(j - (q_start + i))][h]
 * and its gradient: dtable[c][h] = sum of dout[h][i][j] with that bucket = c.
 *
 *   table, dtable : [num_buckets][heads], dense; out, dout: [heads][q_len][k_len].
 *   dtype         : type of all four.
 *   q_start       : place of the first query on the keys' axis.
 *   workspace     : backward only, fm_relative_bias_workspace() bytes, 16-byte
 *                   aligned.
 */
typedef struct {
  int64_t heads, q_len, k_len, q_start, dtype;
  const fm_buckets* buckets;
  const void* table;
  void* out;
  const void* dout;
  void* dtable;
  void* workspace;
  int64_t workspace_bytes;
} fm_relative_bias_args;

fm_status fm_relative_bias_forward(const fm_relative_bias_args* args, fm_stream_t stream);
fm_status fm_relative_bias_backward(const fm_relative_bias_args* args, fm_stream_t stream);
int64_t fm_relative_bias_workspace(const fm_relative_bias_args* args);

/* ------------------------------------------------------------------------
 * Attention over frames.
 *
 *   z[i][j]  = scale * q_i . k_j
 *   z        = softcap * tanh(z / softcap)                where softcap > 0
 *   z       += table[bucket(o)][h]                        where buckets != NULL
 *   z       -= slopes[h] * |o|                            where slopes != NULL
 *   out_i    = sum_j softmax_j(z[i][j] over the keys i may see) v_j
 *
 * with o = j - (start + i) the offset and start the place of the row's first
 * query among its keys. Query i of row b may see key j when all of these hold:
 *   j < k_lens[b]                     (NULL: k_len)
 *   q_docs[b][i] == k_docs[b][j] >= 0 (NULL: any; a negative id is padding)
 *   o <= 0, or j < prefix[b]          (causal only; prefix NULL: 0)
 * A query that may see no key gets out = 0, lse = -inf and no gradient, and
 * keys that nothing sees get zero gradients. Keys at or past k_lens[b], and
 * frames whose document id is negative, are never used: their memory may hold
 * anything, infinities and NaN included.
 * A key that one query may see and another may not changes nothing of the
 * latter, whatever its k and v hold (in the backward pass, whatever the
 * query's q and dout hold). Near a mask's border a query that does see a key
 * whose v is not finite returns NaN in all of its elements.
 *
 *   batch, q_len, k_len, heads, kv_heads, dim : heads a multiple of kv_heads
 *            (query head h reads key head h / (heads / kv_heads)); dim 1 .. 256.
 *   dtype  : type of q, k, v, out, dout, dq, dk, dv.
 *   *_s    : strides {batch, token, head} in elements; the dim elements of one
 *            token's head are adjacent. Strides of q, k, v and dout are free
 *            (0 for broadcast inputs too); out, dq, dk, dv must not overlap
 *            themselves.
 *   q_start: [batch] int32, NULL for q_start_all; q_start_all =
 *            FM_Q_START_END means the queries are the last q_len of the
 *            row's k_lens[b] keys.
 *   table  : [num_buckets][heads], dense, of type table_dtype (dtype or F32).
 *   slopes : [heads] f32.
 *   lse    : [batch][heads][q_len] f32, log of the softmax's sum; the forward
 *            writes it (NULL: not wanted), the backward reads it.
 *   out    : the backward reads what the forward wrote.
 *   out_rest: of dtype and out's strides, what rounding took from out; NULL:
 *            not wanted. Where the backward gets the one that the forward
 *            wrote, its sum of dout * out is that of the unrounded output.
 *   dtable : [num_buckets][heads] of table_dtype; NULL where not wanted.
 *   workspace: fm_attention_workspace(args, backward) bytes, 16-byte aligned.
 */
#define FM_Q_START_END INT64_MIN

typedef struct {
  int64_t batch, q_len, k_len, heads, kv_heads, dim;
  int64_t dtype, causal;
  double scale, softcap;
  const void *q, *k, *v;
  void* out;
  int64_t q_s[3], k_s[3], v_s[3], out_s[3];
  float* lse;
  void* out_rest;
  const int32_t *q_docs, *k_docs, *k_lens, *q_start, *prefix;
  int64_t q_start_all;
  const fm_buckets* buckets;
  const void* table;
  int64_t table_dtype;
  const float* slopes;
  const void* dout;
  void *dq, *dk, *dv;
  int64_t dout_s[3], dq_s[3], dk_s[3], dv_s[3];
  void* dtable;
  void* workspace;
  int64_t workspace_bytes;
} fm_attention_args;

fm_status fm_attention_forward(const fm_attention_args* args, fm_stream_t stream);
fm_status fm_attention_backward(const fm_attention_args* args, fm_stream_t stream);
/* Bytes of workspace of the forward (backward = 0) or backward (1) call; -1
 * where the call itself would refuse the arguments. Pointers may be NULL here
 * except those whose presence changes the computation (masks, buckets,
 * slopes, dtable). */
int64_t fm_attention_workspace(const fm_attention_args* args, int backward);

/* ------------------------------------------------------------------------
 * Root-mean-square norm over the last dimension, after a residual's addition:
 *   total = x + residual, rounded to dtype (x itself where residual == NULL)
 *   y     = total * rstd * weight,  rstd = 1 / sqrt(mean(total^2) + eps)
 * of each row. In 8 bits (y_dtype FM_E4M3) a row has one scale:
 *   scale = max(max |y| / 448, 2^-126),  values = y / scale rounded to FM_E4M3
 * from the unrounded y; a row with an infinity or NaN gets a scale of NaN. The mean of
 * squares is 32-bit: magnitudes beyond 1e18 overflow it, those below 1e-18 vanish in it.
 *
 * Backward: with n = total * rstd and h = dy * weight,
 *   dx = dtotal + rstd * (h - n * mean(h n)),  dweight = sum of dy * n
 * (the gradient of the residual is the same dx).
 *
 *   rows, width : rows 0 .. 2^31 - 1, width 1 .. 2^24.
 *   dtype       : type of x, residual, total, dy, dtotal, dx, and of y.
 *   param_dtype : type of weight and dweight: dtype or FM_F32.
 *   y_dtype     : dtype or FM_E4M3 (forward only).
 *   *_stride    : elements between rows, >= width (any for rows <= 1); the
 *                 elements of a row are adjacent.
 *   residual    : NULL: nothing is added, total is not written.
 *   total       : needed with residual; may be the memory of x or of residual.
 *   weight      : [width]; NULL means ones.
 *   scales      : [rows] f32, FM_E4M3 only.
 *   rstd        : [rows] f32; forward writes it (NULL: not wanted), backward
 *                 reads it.
 *   dtotal      : gradient that reaches total besides; NULL: none.
 *   dx, dweight : each may be NULL where it is not wanted.
 *   The backward call reads total through x; it reads no residual.
 *   workspace   : backward only, fm_rms_norm_workspace() bytes, 16-byte aligned
 *                 (needed where dweight is wanted).
 */
typedef struct {
  int64_t rows, width;
  int64_t dtype, param_dtype, y_dtype;
  int64_t x_stride, residual_stride, total_stride, y_stride, dy_stride, dtotal_stride, dx_stride;
  double eps;
  const void *x, *residual, *weight;
  void *total, *y;
  float *scales, *rstd;
  const void *dy, *dtotal;
  void *dx, *dweight;
  void* workspace;
  int64_t workspace_bytes;
} fm_rms_norm_args;

fm_status fm_rms_norm_forward(const fm_rms_norm_args* args, fm_stream_t stream);
fm_status fm_rms_norm_backward(const fm_rms_norm_args* args, fm_stream_t stream);
int64_t fm_rms_norm_workspace(const fm_rms_norm_args* args);

/*
 * Rows in 8 bits: values and scales as above, of x itself.
 *   x : [rows][width] of dtype, rows x_stride apart; values: [rows][width]
 *   FM_E4M3, rows values_stride apart; scales: [rows] f32.
 */
typedef struct {
  int64_t rows, width, dtype, x_stride, values_stride;
  const void* x;
  void* values;
  float* scales;
} fm_rows_8bit_args;

fm_status fm_rows_8bit(const fm_rows_8bit_args* args, fm_stream_t stream);

/* ------------------------------------------------------------------------
 * Gated linear layer, the first half of a gated feed-forward part:
 *   g = x w_gate^T,  u = x w_up^T,  h = act(g) * u
 * with act(g) = g / (1 + exp(-g))  (FM_ACT_SILU), g (1 + erf(g / sqrt 2)) / 2
 * (FM_ACT_GELU), 1 / (1 + exp(-g)) (FM_ACT_SIGMOID) or max(g, 0) (FM_ACT_RELU, slope
 * 0 at 0). Neither g nor u is ever in memory; the backward pass works them out again:
 *   dg = dh * u * act'(g),  du = dh * act(g)
 *   dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x
 * Products of 16-bit inputs are summed in 32 bits; dg and du are rounded to dtype
 * for the second products (FM_F16: each row's scaled by a power of two before, so that
 * what they can reach at most is just below what the type holds, and for the weights'
 * gradients x alike, which is taken out of the results again: nothing becomes infinite
 * where dx, dw_gate or dw_up would not, and small rows and projections keep their digits).
 *
 * In 8 bits (in_dtype FM_E4M3, forward only) x, w_gate and w_up are FM_E4M3 values with
 * a scale a row, as fm_rms_norm_forward and fm_rows_8bit write them:
 *   g[m][f] = x_scales[m] * gate_scales[f] * sum of products, and u alike.
 *
 *   rows, width, hidden : x [rows][width], w_* [hidden][width], h [rows][hidden];
 *             rows 0 .. 2^30, width and hidden 1 .. 2^24.
 *   dtype   : type of h, dh, dx, dw_*, and of x and w_* where in_dtype is the same.
 *             With FM_E4M3: FM_F16, FM_BF16 or FM_F32, of h.
 *   in_dtype: dtype or FM_E4M3.
 *   *_stride: elements between rows, >= the row's length (any for one row); the
 *             elements of a row are adjacent.
 *   dx, dw_gate, dw_up : each may be NULL where it is not wanted.
 *   workspace: fm_gated_workspace(args, backward) bytes, 16-byte aligned.
 */
enum { FM_ACT_SILU = 0, FM_ACT_GELU = 1, FM_ACT_SIGMOID = 2, FM_ACT_RELU = 3 };

typedef struct {
  int64_t rows, width, hidden;
  int64_t dtype, in_dtype, act;
  int64_t x_stride, gate_stride, up_stride, h_stride, dh_stride, dx_stride, dgate_stride, dup_stride;
  const void *x, *w_gate, *w_up;
  const float *x_scales, *gate_scales, *up_scales;
  void* h;
  const void* dh;
  void *dx, *dw_gate, *dw_up;
  void* workspace;
  int64_t workspace_bytes;
} fm_gated_args;

fm_status fm_gated_forward(const fm_gated_args* args, fm_stream_t stream);
fm_status fm_gated_backward(const fm_gated_args* args, fm_stream_t stream);
/* Bytes of workspace of the forward (backward = 0) or backward (1) call; -1 where
 * the call itself would refuse the sizes or types. Pointers and strides count: they
 * decide which kernels run. */
int64_t fm_gated_workspace(const fm_gated_args* args, int backward);

/* ------------------------------------------------------------------------
 * Gated linear recurrence over frames, each channel by itself:
 *   a_t = 1 / (1 + exp(-gate_t))
 *   h_t = a_t * h_(t-1) + (1 - a_t) * x_t,   y_t = h_t
 * in the order of time, or against it (reverse). The recurrence is held in 32 bits.
 *
 * Frame t of row b is used when
 *   t < lens[b]             (NULL: all)
 *   docs[b][t] >= 0         (NULL: all)
 * Frames that are not used get y = 0 and no gradient, leave the state as it is, and
 * their memory may hold anything. The row's first frame in the order of the walk
 * goes on from `state`; a later one whose document id differs from the one before
 * it (a padding frame's included) starts from 0.
 *
 * Backward: with dh_t = dy_t + what comes back from the next frame (dend behind the
 * last one), dx_t = (1 - a_t) dh_t, dgate_t = dh_t (h_(t-1) - x_t) a_t (1 - a_t), and
 * a_t dh_t goes back to the frame before; what leaves the first is dstate.
 *
 *   batch, frames, channels : each >= 0, channels 1 .. 2^24, frames up to 2^30,
 *             batch up to 2^31 - 1 (FM_ERR_UNSUPPORTED where batch times channels
 *             takes more blocks than a launch has).
 *   dtype   : type of x, gate, y, dy, dx and dgate.
 *   *_s     : strides {batch, frame} in elements; channels are adjacent. Free for
 *             x, gate and dy (0 for broadcast inputs too); y, dx and dgate must not
 *             overlap themselves.
 *   state, end, dend, dstate : [batch][channels] f32, dense; NULL: zeros, or not
 *             wanted. end (the state after the last frame) may be state's memory.
 *   lens    : [batch] int32.  docs: [batch][frames] int32, dense.
 *   marks   : fm_scan_marks() bytes, 16-byte aligned, states along the row that the
 *             forward leaves (NULL: not wanted) and the backward reads.
 *   workspace : fm_scan_workspace() bytes, 16-byte aligned, the same for both
 *             directions; without it, or with fewer bytes, few channels of long rows
 *             take longer (and sums are joined in another order). Not touched where
 *             fm_scan_workspace() is 0.
 */
typedef struct {
  int64_t batch, frames, channels;
  int64_t dtype, reverse;
  int64_t x_s[2], gate_s[2], y_s[2], dy_s[2], dx_s[2], dgate_s[2];
  const void *x, *gate;
  const float* state;
  const int32_t *lens, *docs;
  void* y;
  float *end, *marks;
  const void* dy;
  const float* dend;
  void *dx, *dgate;
  float* dstate;
  void* workspace;
  int64_t workspace_bytes;
} fm_scan_args;

fm_status fm_scan_forward(const fm_scan_args* args, fm_stream_t stream);
fm_status fm_scan_backward(const fm_scan_args* args, fm_stream_t stream);
int64_t fm_scan_marks(const fm_scan_args* args);
int64_t fm_scan_workspace(const fm_scan_args* args);

/* Where a bounded wait inside a kernel of the attention, the gated layer or the
 * gated recurrence gives up (after two seconds; never in ordinary running), the
 * results of its call are not valid. From when the host can see it the calls of
 * those three on that device that would wait start nothing and return
 * FM_ERR_KERNEL_TIMEOUT, until the error is taken; calls under way by then, and
 * replays of recorded ones, may give up early too.
 *
 * fm_ops_poll_error waits for all work queued on the current device, on any
 * stream, then takes and clears that error: FM_ERR_KERNEL_TIMEOUT or FM_OK. Not
 * allowed while a graph is being recorded.
 *
 * fm_ops_selftest_wait -- diagnostic: queues a kernel of one warp whose wait
 * runs out, so that the two ways of learning of it can be tested. */
fm_status fm_ops_poll_error(void);
fm_status fm_ops_selftest_wait(fm_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif
