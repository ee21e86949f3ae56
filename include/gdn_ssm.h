/*
 * gdn_ssm.h -- C ABI of the state space layer that stands beside Gated
 * DeltaNet layers in hybrid models: the short causal convolution, the
 * selective scan, the single-token step and the gated group norm.
 *
 *   gdn_ssm_conv    K-tap causal depthwise conv over the packed x|B|C channels
 *                   with a carried history, bias and SiLU.
 *   gdn_ssm_scan    the selective state space recurrence on a per-head fp32
 *                   state, for whole prompts.
 *   gdn_ssm_step    one decode token per sequence: conv and recurrence.
 *   gdn_group_norm  per-token group norm (RMS or centred) with a SiLU gate
 *                   before or after it.
 *
 * The conventions of gdn.h hold: device pointers on the current HIP device,
 * a host `shape` read during the call only, a hipStream_t passed as void*,
 * nothing synchronises or allocates, the library keeps no state, every
 * argument check runs before anything is enqueued, and the return value is a
 * gdn_status.  A call that enqueues several kernels returns GDN_E_LAUNCH when
 * the runtime refuses one of them; its outputs are then undefined.
 *
 * Symbols and layouts (row-major).  H = heads, P = head_dim, G = groups,
 * N = state_dim, K = conv_width, C = H*P + 2*G*N; "io" = shape->io_dtype.
 *   cu_seqlens [n_seq+1] int32  sequence n owns tokens [cu[n], cu[n+1]); cu[0]
 *                               = 0, non-decreasing, no sequence longer than
 *                               max_T, cu[n_seq] <= total_T.  Token rows from
 *                               cu[n_seq] on belong to no sequence: they are
 *                               not read and their outputs are left as they
 *                               were.  These device contents are a
 *                               precondition; a value outside [0, total_T] is
 *                               taken as the nearer end, so that no access
 *                               leaves the buffers.
 *   xbc     [total_T][C]      io   channel blocks x (H heads of P) | B (G
 *                                  groups of N) | C (G groups of N); head h
 *                                  reads B and C of group h / (H/G)
 *   conv_w  [C][K]            io   tap K-1 multiplies the current token
 *   conv_b  [C]               io   or NULL (no bias)
 *   hist    [n_seq][K-1][C]   io   the K-1 rows before the first token, oldest
 *                                  first; NULL: zeros
 *   dt      [total_T][H]      io   raw step sizes
 *   A_log, dt_bias, D  [H]    fp32 (as such models keep them); D may be NULL
 *   state   [n_seq][H][P][N]  fp32 NULL: zeros
 *   y       [total_T][H][P]   shape->out_dtype
 * The raw xbc and dt of gdn_ssm_conv and gdn_ssm_step, and dt of gdn_ssm_scan,
 * may be column blocks of a wider projection: xbc_stride and dt_stride give
 * the elements between token rows.  Every other buffer is dense.
 * Alignment: workspaces 256-byte; xbc (rows too), conv_w, conv_b, hist, state,
 * y and the norm's rows 16-byte; cu_seqlens, A_log, dt_bias and D 4-byte; dt
 * by its element (GDN_E_ALIGN otherwise).
 * No two buffers may overlap, except hist_out == hist and state_out == state
 * (updated in place).
 */
#ifndef GDN_SSM_H
#define GDN_SSM_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A dtype code of the entry points of this header only, beside GDN_F32 and
 * GDN_F16: bfloat16. */
#define GDN_BF16 2

/* Sizes of one call.  Supported: 1 <= groups, heads % groups == 0, heads <=
 * 4096; head_dim a multiple of 16 up to 256; state_dim 32, 64, 128 or 256;
 * conv_width 2, 3 or 4; out_dtype GDN_F32 or io_dtype; 1 <= n_seq <= 2^20;
 * 0 <= max_T <= total_T <= 2^27; strides 0 or a row's elements up to 2^40;
 * 0 <= dt_min <= dt_max (dt_max may be +infinity). */
typedef struct gdn_ssm_shape {
    int32_t heads, head_dim, groups, state_dim;
    int32_t conv_width; /* read by gdn_ssm_conv and gdn_ssm_step, checked by all */
    int32_t n_seq;
    int32_t io_dtype;   /* of xbc, conv_w, conv_b, hist, dt and the conv's output */
    int32_t out_dtype;  /* of y */
    int64_t total_T;    /* token rows of the buffers */
    int64_t max_T;      /* host copy of max_n (cu[n+1] - cu[n]), or more */
    int64_t xbc_stride; /* elements between rows of the raw xbc; 0: C */
    int64_t dt_stride;  /* elements between rows of dt; 0: heads */
    float dt_min, dt_max;
} gdn_ssm_shape;

/*
 * gdn_ssm_conv -- per sequence, with X = [hist; token rows] ((K-1+T) x C):
 *   out[t][c] = SiLU(conv_b[c] + sum_{k<K} conv_w[c][k] X[t+k][c])
 *   hist_out <- the last K-1 rows of X (bit for bit)
 * Sums in fp32, one rounding to io.  In: cu_seqlens, xbc, conv_w, conv_b,
 * hist.  Out: out [total_T][C] io, dense; hist_out [n_seq][K-1][C] (NULL: not
 * kept; may be hist itself).  With total_T == 0 the history is copied.
 */
int gdn_ssm_conv(const gdn_ssm_shape *shape, const int32_t *cu_seqlens, const void *xbc,
                 const void *conv_w, const void *conv_b, const void *hist, void *hist_out,
                 void *out, void *stream);

/*
 * gdn_ssm_scan -- per sequence and head h, over its tokens in order, with S
 * the P x N state and x, B, C the token's convolved channels:
 *   dt = clamp(softplus(dt[t][h] + dt_bias[h]), dt_min, dt_max)
 *   S <- exp(-exp(A_log[h]) dt) S + dt x B^T
 *   y[t][h] = S C + D[h] x
 * The state, the decays and every sum are held in fp32 (sums of log decays in
 * 64 bits), whatever out_dtype is.  As operands of the matrix products the fp32
 * quantities keep all of their bits where io is fp32 or bf16; where it is fp16
 * they are off by at most 2^-23 of their value or 2^-38 of the largest of their
 * row or column.  A decay below e^-200 is taken as e^-200, which is 0 in fp32, and a
 * token that the decays after it bring below e^-104 no longer counts.  A value
 * that is not finite leaves every output before its token and every other sequence
 * as they are; from its token on it makes outputs undefined: x those of its channel,
 * dt those of its head, B those of its group's heads, C its token's of that group.
 * In: cu_seqlens, xbc [total_T][C] dense (gdn_ssm_conv's output), dt, A_log,
 * dt_bias, D, state.  Out: y; state_out (NULL: not kept; may be state itself).
 * A sequence of no tokens keeps its state.
 * workspace: device scratch of >= gdn_ssm_scan_workspace_bytes(shape) bytes,
 * 256-byte aligned (NULL where that is 0); its contents are undefined after
 * the call, and it must not be shared by calls in flight at the same time.
 */
int gdn_ssm_scan(const gdn_ssm_shape *shape, const int32_t *cu_seqlens, const void *xbc,
                 const void *dt, const float *A_log, const float *dt_bias, const float *D,
                 const float *state, float *state_out, void *y, void *workspace,
                 size_t workspace_bytes, void *stream);

/* Bytes of scratch gdn_ssm_scan needs for `shape` (0 also if the shape is
 * invalid, which gdn_ssm_scan reports). */
size_t gdn_ssm_scan_workspace_bytes(const gdn_ssm_shape *shape);

/*
 * gdn_ssm_step -- one token for each of n_seq sequences: the arithmetic of
 * gdn_ssm_conv and gdn_ssm_scan with total_T == n_seq and max_T == 1 (token row
 * n belongs to sequence n, no cu_seqlens), x, B and C staying in fp32 between
 * the two.  One kernel with a separate hist_out; with hist_out == hist two
 * (the step, then the history shift, since every head of a group reads the
 * group's old B and C rows).  hist, hist_out, state and state_out as above.
 */
int gdn_ssm_step(const gdn_ssm_shape *shape, const void *xbc, const void *conv_w,
                 const void *conv_b, const void *dt, const float *A_log, const float *dt_bias,
                 const float *D, const void *hist, void *hist_out, const float *state,
                 float *state_out, void *y, void *stream);

/* gdn_norm_shape.flags */
#define GDN_NORM_CENTRE 1    /* subtract the group's mean (else RMS)            */
#define GDN_NORM_GATE_LAST 2 /* gate after the norm (else before it)            */

/* Sizes of one gdn_group_norm call: 0 <= rows <= 2^27, channels a multiple of
 * 8*groups, at most 16384 channels a group and 65536 a row; x_dtype GDN_F32 or
 * io_dtype; eps finite and >= 0. */
typedef struct gdn_norm_shape {
    int64_t rows;
    int32_t channels, groups;
    int32_t x_dtype;  /* of x */
    int32_t io_dtype; /* of z, weight, bias and y */
    int64_t x_stride; /* elements between rows of x; 0: channels */
    int64_t z_stride; /* elements between rows of z; 0: channels */
    int32_t flags;
    float eps;
} gdn_norm_shape;

/*
 * gdn_group_norm -- per row and group of channels/groups consecutive channels:
 *   v = x * SiLU(z)       (x alone with GDN_NORM_GATE_LAST or z NULL)
 *   m = mean(v) with GDN_NORM_CENTRE, else 0
 *   y = (v - m) / sqrt(mean((v - m)^2) + eps) * weight + bias
 *   y = y * SiLU(z)       (with GDN_NORM_GATE_LAST and z)
 * in fp32, rounded once to io.  z, weight [channels] and bias [channels] may
 * be NULL (no gate, 1 and 0).  y [rows][channels] is dense.
 */
int gdn_group_norm(const gdn_norm_shape *shape, const void *x, const void *z, const void *weight,
                   const void *bias, void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SSM_H */
