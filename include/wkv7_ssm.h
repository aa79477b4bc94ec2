/*
 * wkv7_ssm.h - C ABI of the state-space mixer's operators in libwkv7.so: the
 * short causal convolution, the selective state-space scan, the RMS norm with
 * the residual's addition, and 8-bit activation checkpoints.
 *
 * The scan is the library's second recurrence.  Where the WKV7 state decays per
 * key channel and takes a rank-one transition (wkv7.h), a scan channel d holds
 * N numbers that decay each by its own rate:
 *
 *     dt_t  = softplus(delta_t + dt_bias)                  (per channel)
 *     h_t   = exp(dt_t A) h_{t-1} + dt_t u_t B_t           (h, A, B: N numbers)
 *     s_t   = C_t . h_t + D u_t
 *     y_t   = s_t z_t sigmoid(z_t)
 *
 * The convolution mixes each channel with its last W - 1 inputs (width 2 without
 * activation is a token shift); its output is the scan's u.
 *
 * Conventions are wkv7.h's (device pointers, caller-owned scratch, asynchronous
 * on `stream`, host checks before any launch, no exception) with these
 * differences:
 *  - Per-token inputs are read through strides, in elements: *_bs from one
 *    sequence to the next, *_ts from one token to the next (both >= 0; a
 *    token's channels are contiguous), so a slice of a projection's output is
 *    taken as it is.  They need their element's alignment only; 16-byte aligned
 *    pointers with strides and widths that are multiples of 8 elements run the
 *    vector loads.  Outputs and gradients are contiguous.
 *  - fp32 parameters, states and workspaces are contiguous; workspaces and
 *    [.., N] states are 16-byte aligned.
 *  - Any D >= 0 up to WKV7_SSM_MAX_D, any 1 <= N <= 64, W = 2, 3 or 4; other
 *    sizes return WKV7_ERR_UNSUPPORTED.
 *  - Outputs overlap no input, except where a call says so.
 *  - Every sum runs in a fixed order: the same call on the same device gives
 *    the same bits.
 */
#ifndef WKV7_SSM_H
#define WKV7_SSM_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WKV7_SSM_MAX_D 1048576      /* channels */
#define WKV7_NORM_MAX_D 16384       /* channels of the RMS norm's row */
#define WKV7_ACT8_BLOCK 128         /* channels that share a scale */

/*
 * 8-bit activations.  A [rows, D] activation is kept as e4m3 codes [rows, D]
 * and fp32 scales [rows, ceil(D / 128)]: for each row and block of 128
 * channels the scale is the least power of two >= amax / 448 (448: the largest
 * e4m3 number), at least 2^-117, and a code is x / scale rounded to nearest
 * even.  A power-of-two scale divides exactly, so a value is rounded once, to
 * within 2^-4 of itself (2^-10 of the scale below 2^-6 of it), and code * scale is exact
 * in bf16 and fp32 (a value that would round to 2^128 takes the code below).
 * An infinite or NaN element becomes a NaN code and does not
 * touch its block's scale.
 *   x    : rows of x_dtype, x_ld elements apart
 *   out  : [rows, D] of out_dtype, contiguous
 */
WKV7_API wkv7_status wkv7_act8_save(long long rows, int D, wkv7_dtype x_dtype, const void *x, long long x_ld,
                                    void *codes, float *scales, cudaStream_t stream);
WKV7_API wkv7_status wkv7_act8_load(long long rows, int D, const void *codes, const float *scales,
                                    wkv7_dtype out_dtype, void *out, cudaStream_t stream);

/*
 * RMS norm with the residual's addition, per row:
 *     s = x + residual,   rstd = 1 / sqrt(mean(s^2) + eps),   y = weight s rstd
 * The sum is normalised as it is, before it is rounded to residual_out's type.
 *   x            : rows of x_dtype, x_ld elements apart
 *   residual     : [rows, D] of r_dtype, or NULL (s = x)
 *   weight       : [D] fp32
 *   eps          : >= 0; the mean square is taken in fp64, so a row may be as large or
 *                  small as its type allows.  A row with an infinity has rstd = 0, and
 *                  one with mean(s^2) + eps = 0, or so small that rstd is above fp32's
 *                  range, has rstd = inf; y follows from the formula
 *   residual_out : [rows, D] of r_dtype (s rounded), or NULL; may be residual
 *   y            : [rows, D] of y_dtype; WKV7_E4M3 writes 8-bit codes, with
 *                  y_scales [rows, ceil(D / 128)] (NULL otherwise)
 *   s_codes, s_scales : the 8-bit activation of s (rounded once from the exact
 *                  sum), which the backward reads, or both NULL
 *   rstd         : [rows] fp32, or NULL
 */
WKV7_API wkv7_status wkv7_rmsnorm_forward(long long rows, int D, wkv7_dtype x_dtype, wkv7_dtype r_dtype,
                                          wkv7_dtype y_dtype, const void *x, long long x_ld, const void *residual,
                                          const float *weight, float eps, void *residual_out, void *y,
                                          float *y_scales, void *s_codes, float *s_scales, float *rstd,
                                          cudaStream_t stream);

/* Bytes of scratch wkv7_rmsnorm_backward needs (the weight gradient's partial sums). */
WKV7_API size_t wkv7_rmsnorm_backward_workspace_size(long long rows, int D);

/*
 * Gradients of the norm from dy (of y) and dresidual (of residual_out).  With
 * xh = s rstd and c = mean(weight dy xh):
 *     dx = dresidual + rstd (weight dy - c xh)   (of x and of residual alike)
 *     dweight = sum over rows of dy xh
 *   s          : what the forward normalised: [rows, D] of s_dtype (its
 *                residual_out, or x), or WKV7_E4M3 codes with s_scales
 *   rstd       : [rows] fp32 of the forward
 *   dy         : [rows, D] of dy_dtype
 *   dresidual  : [rows, D] of grad_dtype, or NULL for zeros; dx may be dresidual
 *   dx         : [rows, D] of grad_dtype
 *   dweight    : [D] fp32
 */
WKV7_API wkv7_status wkv7_rmsnorm_backward(long long rows, int D, wkv7_dtype s_dtype, wkv7_dtype dy_dtype,
                                           wkv7_dtype grad_dtype, const void *s, const float *s_scales,
                                           const float *rstd, const float *weight, const void *dy,
                                           const void *dresidual, void *dx, float *dweight, void *workspace,
                                           size_t workspace_bytes, cudaStream_t stream);

/*
 * Short causal convolution, per channel:
 *     p_t = bias + sum_{j < W} weight[j] x_{t - W + 1 + j},
 *     y_t = p_t sigmoid(p_t) with silu, else p_t
 * x before the first token comes from `state`: the last W - 1 inputs, oldest
 * first.
 *   x         : [B, T, D] of x_dtype, strided; or WKV7_E4M3 codes, contiguous
 *               (strides ignored), with x_scales [B, T, ceil(D / 128)]
 *   weight    : [D, W] fp32;   bias : [D] fp32, or NULL for zeros
 *   state     : [B, W - 1, D] of x_dtype (of y_dtype when x is codes), or NULL
 *               for zeros
 *   lens      : [B] tokens of each sequence (clamped to 0 .. T), or NULL for T.
 *               Rows of y behind a sequence's end stay as they are.
 *   y         : [B, T, D] of y_dtype; not x itself
 *   state_out : [B, W - 1, D] of x_dtype, the last W - 1 inputs of each
 *               sequence, or NULL; not with codes, and not `state` itself
 *   codes, scales : the 8-bit activation of x, written in the same pass, or
 *               both NULL; not with lens, nor when x is codes
 */
WKV7_API wkv7_status wkv7_conv_forward(int B, int T, int D, int W, wkv7_dtype x_dtype, wkv7_dtype y_dtype,
                                       const void *x, long long x_bs, long long x_ts, const float *x_scales,
                                       const float *weight, const float *bias, const void *state, const int *lens,
                                       int silu, void *y, void *state_out, void *codes, float *scales,
                                       cudaStream_t stream);

/* One token for every sequence; the state [B, W - 1, D] of x_dtype moves on in
 * place.  x : [B, D] rows x_bs elements apart;  y : [B, D] of y_dtype. */
WKV7_API wkv7_status wkv7_conv_step(int B, int D, int W, wkv7_dtype x_dtype, wkv7_dtype y_dtype, const void *x,
                                    long long x_bs, const float *weight, const float *bias, void *state, int silu,
                                    void *y, cudaStream_t stream);

/* Bytes of scratch wkv7_conv_backward needs (the parameter gradients' partial sums). */
WKV7_API size_t wkv7_conv_backward_workspace_size(int B, int T, int D, int W);

/*
 * Gradients of the convolution: L = sum(dy * y) + sum(dstate_out * state_out).
 *   x, x_scales, weight, bias, state : the forward's, or x's 8-bit activation
 *                (p_t is computed again from it); state is of x_dtype, of
 *                grad_dtype when x is codes
 *   dy         : [B, T, D] of dy_dtype, contiguous
 *   dstate_out : [B, W - 1, D] fp32, or NULL for zeros
 *   dx         : [B, T, D] of grad_dtype; not x or dy itself
 *   dweight    : [D, W] fp32;  dbias : [D] fp32, or NULL
 *   dstate     : [B, W - 1, D] fp32, or NULL; not dstate_out itself
 */
WKV7_API wkv7_status wkv7_conv_backward(int B, int T, int D, int W, wkv7_dtype x_dtype, wkv7_dtype dy_dtype,
                                        wkv7_dtype grad_dtype, const void *x, long long x_bs, long long x_ts,
                                        const float *x_scales, const float *weight, const float *bias,
                                        const void *state, const void *dy, const float *dstate_out, int silu,
                                        void *dx, float *dweight, float *dbias, float *dstate, void *workspace,
                                        size_t workspace_bytes, cudaStream_t stream);

/* Bytes of scratch with which wkv7_ssm_forward splits a long sequence over few
 * channels into segments that run side by side (0 when it would not).  Depends
 * on the current device's SM count. */
WKV7_API size_t wkv7_ssm_forward_workspace_size(int B, int T, int D, int N, int G);

/* Bytes of the states that wkv7_ssm_forward can keep for the backward: h before
 * every 16th token, [B, ceil(T / 16), D, N] fp32. */
WKV7_API size_t wkv7_ssm_saved_states_size(int B, int T, int D, int N);

/*
 * Selective scan over whole sequences (the formulas above).
 *   u, delta, z : [B, T, D] of in_dtype, strided; z NULL leaves the gate out
 *   A           : [D, N] fp32 rates (negative for a state that decays)
 *   Bm, Cm      : [B, T, G, N] of in_dtype, strided, a token's [G, N]
 *                 contiguous; channel d takes group d / (D / G), D % G = 0
 *   Dskip, dt_bias : [D] fp32, or NULL for zeros
 *   state0      : [B, D, N] fp32, or NULL for zeros
 *   softplus    : 0 takes dt_t = delta_t + dt_bias as it is
 *   lens        : [B] tokens of each sequence (clamped to 0 .. T), or NULL.
 *                 Rows of y behind a sequence's end stay as they are, and
 *                 stateT is the state at its end.
 *   y           : [B, T, D] of y_dtype
 *   stateT      : [B, D, N] fp32, or NULL; may be state0
 *   states      : wkv7_ssm_saved_states_size() bytes for wkv7_ssm_backward, or
 *                 NULL; not with lens
 *   workspace   : wkv7_ssm_forward_workspace_size() bytes; without it (NULL or
 *                 smaller) the sequence runs in one piece
 */
WKV7_API wkv7_status wkv7_ssm_forward(int B, int T, int D, int N, int G, wkv7_dtype in_dtype, wkv7_dtype y_dtype,
                                      const void *u, long long u_bs, long long u_ts, const void *delta,
                                      long long delta_bs, long long delta_ts, const float *A, const void *Bm,
                                      long long b_bs, long long b_ts, const void *Cm, long long c_bs, long long c_ts,
                                      const float *Dskip, const void *z, long long z_bs, long long z_ts,
                                      const float *dt_bias, const float *state0, int softplus, const int *lens,
                                      void *y, float *stateT, float *states, void *workspace,
                                      size_t workspace_bytes, cudaStream_t stream);

/* One token for every sequence: u, delta, z [B, D] and Bm, Cm [B, G, N], rows
 * *_bs elements apart; the state [B, D, N] fp32 is updated in place; y [B, D]. */
WKV7_API wkv7_status wkv7_ssm_step(int B, int D, int N, int G, wkv7_dtype in_dtype, wkv7_dtype y_dtype,
                                   const void *u, long long u_bs, const void *delta, long long delta_bs,
                                   const float *A, const void *Bm, long long b_bs, const void *Cm, long long c_bs,
                                   const float *Dskip, const void *z, long long z_bs, const float *dt_bias,
                                   float *state, int softplus, void *y, cudaStream_t stream);

/* Bytes of scratch wkv7_ssm_backward needs; with_states = 0 adds the states it
 * then computes itself.  Depends on the current device's SM count. */
WKV7_API size_t wkv7_ssm_backward_workspace_size(int B, int T, int D, int N, int G, int with_states);

/*
 * Gradients of the scan: L = sum(dy * y) + sum(dstateT * stateT).
 *   u .. state0 : the forward's
 *   states      : what the forward kept, or NULL to compute it here (state0 is
 *                 read only then)
 *   dy          : [B, T, D] of in_dtype, contiguous
 *   dstateT     : [B, D, N] fp32, or NULL for zeros
 *   du, ddelta  : [B, T, D] of grad_dtype;  dz : the same (required with z,
 *                 NULL without)
 *   dA          : [D, N] fp32
 *   dB, dC      : [B, T, G, N] of grad_dtype
 *   dD, ddt_bias: [D] fp32, or NULL
 *   dstate0     : [B, D, N] fp32, or NULL; may be dstateT
 */
WKV7_API wkv7_status wkv7_ssm_backward(int B, int T, int D, int N, int G, wkv7_dtype in_dtype,
                                       wkv7_dtype grad_dtype, const void *u, long long u_bs, long long u_ts,
                                       const void *delta, long long delta_bs, long long delta_ts, const float *A,
                                       const void *Bm, long long b_bs, long long b_ts, const void *Cm,
                                       long long c_bs, long long c_ts, const float *Dskip, const void *z,
                                       long long z_bs, long long z_ts, const float *dt_bias, const float *state0,
                                       int softplus, const float *states, const void *dy, const float *dstateT,
                                       void *du, void *ddelta, float *dA, void *dB, void *dC, float *dD, void *dz,
                                       float *ddt_bias, float *dstate0, void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WKV7_SSM_H */
