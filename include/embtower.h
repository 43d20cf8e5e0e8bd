/*
 * embtower.h -- C ABI of the dense-tower operators that stand next to the embedding core of
 * embcore.h: a dense layer with bias, activation, dropout and residual in its epilogue and
 * its backward, the same epilogue on its own, and a channels-last group norm with an
 * activation.  They build the layers of a deeper (residual, regularised, normalised) tower
 * around the pooled embeddings.  Built into the same library; every convention of embcore.h
 * holds (device pointers unless marked [host], caller-owned memory, work enqueued on
 * `stream`, host-side validation before anything is enqueued, no aliasing of outputs with
 * inputs, bitwise reproducible results, round to nearest even), with two differences: data
 * pointers need only the alignment of their element type (each call takes the vector path
 * that the alignment allows), and row strides are 64-bit.
 */
#ifndef EMBTOWER_H
#define EMBTOWER_H

#include "embcore.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations, next to EL_ACT_NONE and EL_ACT_RELU:
 *   EL_ACT_GELU  u Phi(u) = u (1 + erf(u / sqrt 2)) / 2
 *                (absolute error in fp32 at most 2.2e-7 for |u| <= 8; the error relative to the
 *                value passes 1e-3 below u = -4.6, where the value is smaller than 1e-5)
 *   EL_ACT_SILU  u / (1 + exp(-u)) */
enum { EL_ACT_GELU = 2u, EL_ACT_SILU = 3u };

/*
 * Dropout whose mask is a function of the element's place and is never stored.  Philox4x32-10
 * (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) with
 *   key     = (seed low, seed high)
 *   counter = (n / 8, m, o low, o high),  o = offset + step[0]
 * gives four 32-bit words, read as eight 16-bit numbers, low half of a word first: number n % 8
 * belongs to column n of row m.  With T = round(65536 p) the element is kept where its number
 * is >= T and then multiplied by 65536 / (65536 - T); a dropped element is +0 whatever it held
 * (infinities and NaN too).  p is thus used to 16 bits; T = 0 keeps everything.  The mask does
 * not depend on strides, launch shape or dtype, so the backward draws the forward's mask again
 * from the same (p, seed, offset, step).
 */
typedef struct {
  double p;              /* in [0, 1] */
  uint64_t seed;
  uint64_t offset;       /* a number of its own for every layer (and step, without `step`) */
  const uint64_t* step;  /* device, or NULL (0): read when the work runs, so that every replay of
                            a captured graph can draw another mask */
} el_dropout;

/*
 * Activation, dropout and residual on their own:
 *   y[m][n] = residual[m][n] + drop(act(x[m][n])),   m < M, n < N
 * act: EL_ACT_*; drop NULL: no dropout; residual NULL: none.  x, residual, y: rows of strides
 * ldx, ldr, ldy (elements), all of dtype; fp32 arithmetic, one rounding.  A call with
 * M ceil(N / 8) > 2^32 - 256 is refused (EL_ERR_UNSUPPORTED).
 */
EL_API el_status el_act_dropout_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                    int32_t M, int32_t N, uint32_t act, const el_dropout* drop,
                                    void* y, int64_t ldy, el_dtype dtype, hipStream_t stream);

/*
 * Its gradient with respect to x:  dx[m][n] = drop(dy[m][n] * act'(x[m][n])), the same mask.
 * (The residual's gradient is dy.)  x may be NULL with EL_ACT_NONE.  ReLU'(0) = 0.
 */
EL_API el_status el_act_dropout_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                    int32_t M, int32_t N, uint32_t act, const el_dropout* drop,
                                    void* dx, int64_t lddx, el_dtype dtype, hipStream_t stream);

/* [host, pure] Bytes of device workspace el_dense_fwd / el_dense_bwd can need for these sizes,
 * whatever the strides and alignments; 0 for invalid or unsupported sizes or M == 0. */
EL_API size_t el_dense_fwd_workspace_bytes(int32_t M, int32_t K, int32_t N);
EL_API size_t el_dense_bwd_workspace_bytes(int32_t M, int32_t K, int32_t N);

/*
 * Dense layer with an epilogue:
 *   z[m][n] = sum_k x[m][k] w[n][k] + bias[n]
 *   y[m][n] = residual[m][n] + drop(act(z[m][n]))
 *   pre[m][n] = z[m][n]                             (pre may be NULL: not stored)
 * x: [M] rows of stride ldx (first K used); w: [N][K] row-major; bias: fp32 [N] or NULL;
 * residual, pre, y: [M] rows of strides ldr, ldpre, ldy.  dtype: EL_BF16 or EL_F16 (one for x,
 * w, residual, pre and y).  Products accumulate in fp32 (MFMA); y is computed from the fp32 z,
 * one rounding each.  Any K, N from 1 to 2^20 with N K < 2^29 and ceil(M/256) ceil(N/256) < 2^21
 * (EL_ERR_UNSUPPORTED beyond).  x and w are copied to the workspace where their rows are not
 * whole 16-byte aligned vectors; such operands may have fewer than 2^35 elements together.
 * workspace: >= el_dense_fwd_workspace_bytes(M, K, N), 256-byte aligned, contents irrelevant
 * (NULL when that is 0).
 */
EL_API el_status el_dense_fwd(const void* x, int64_t ldx, int32_t M, int32_t K, const void* w,
                              const float* bias, int32_t N, uint32_t act, const el_dropout* drop,
                              const void* residual, int64_t ldr, void* pre, int64_t ldpre, void* y,
                              int64_t ldy, el_dtype dtype, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);

/*
 * Dense layer backward from dz = dL/dz:
 *   dw[n][k]  = sum_m dz[m][n] x[m][k]       fp32 [N][K], overwritten
 *   db[n]     = sum_m dz[m][n]               fp32 [N], overwritten (NULL: not computed)
 *   dx[m][k]  = sum_n dz[m][n] w[n][k] + dres[m][k]
 *                                            (dx may be NULL; dres NULL: nothing added)
 *   dzb[m][k] = drop(dx[m][k] * act'(pre[m][k]))
 *                                            (dzb may be NULL)
 * dres is the gradient that reaches x by another way (the skip connection of a residual
 * layer).  dzb is the dz of the layer below, whose output is x: act, drop and pre are that
 * layer's; it is computed from the fp32 dx, so a tower's backward is one call per layer.  pre
 * may be NULL with EL_ACT_NONE; dzb needs dx.  The sums over m are split into fixed slices (by
 * the sizes, and by whether dx is asked for) whose fp32 partials are added in a fixed order:
 * bitwise reproducible.  M == 0 gives zero dw, db.  K and N as in the
 * forward, and ceil(M/256) ceil(K/256) < 2^21 where dx is asked for; dz, x and (for dx) w are
 * copied as x and w are there, with the same limit.
 * workspace: >= el_dense_bwd_workspace_bytes(M, K, N), 256-byte aligned.
 */
EL_API el_status el_dense_bwd(const void* x, int64_t ldx, int32_t M, int32_t K, const void* w,
                              int32_t N, const void* dz, int64_t lddz, const void* dres,
                              int64_t lddres, void* dx, int64_t lddx, uint32_t act,
                              const el_dropout* drop, const void* pre, int64_t ldpre, void* dzb,
                              int64_t lddzb, float* dw, float* db, el_dtype dtype, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/* [host, pure] Bytes of device workspace el_group_norm_fwd / _bwd need for B samples of S
 * positions, C channels in G groups; 0 for invalid or empty sizes.  The forward's are at most
 * 8 MiB for up to 2048 channels. */
EL_API size_t el_group_norm_fwd_workspace_bytes(int32_t B, int32_t S, int32_t C, int32_t G);
EL_API size_t el_group_norm_bwd_workspace_bytes(int32_t B, int32_t S, int32_t C, int32_t G);

/*
 * Group norm with an activation, channels last.  Sample b's positions are rows b*S .. b*S+S-1
 * of x, C channels each; group g is the channels [g C/G, (g+1) C/G).  Over the n = len[b] C/G
 * values of a group in the first len[b] positions (len[b] = lengths[b], or S when lengths is
 * NULL; values outside [0, S] are clamped to it):
 *   mean[b][g] = sum x / n,   rstd[b][g] = 1 / sqrt(sum (x - mean)^2 / n + eps)
 *   u = gamma[c] (x - mean) rstd + beta[c],   y = act(u)
 * Positions from len[b] on are padding: they are not read, and y is +0 there.  An empty sample
 * has mean 0 and rstd 1 / sqrt(eps).  G = 1 and S = 1 is a layer norm of each row; x = the
 * pooled vectors [B][F][D] normalises each sample's embeddings over its F tables.
 * x, y: rows of strides ldx, ldy, dtype EL_F32 / EL_F16 / EL_BF16; gamma, beta: fp32 [C] or
 * NULL (1, 0); mean, rstd: fp32 [B][G], overwritten; statistics and arithmetic in fp32, the
 * variance from centred values.  C % G == 0, eps >= 0 finite.  Up to C = 2^20 and S = 2^30, with
 * B G < 2^25 (EL_ERR_UNSUPPORTED beyond, as for batches that one launch cannot hold: B below 2^22
 * always fits where a sample has at most 512 vectors of eight channels, and rows, S = 1, of up to
 * 2048 channels with G = 1 below 2^24; longer samples B G < 2^22).  workspace: >=
 * el_group_norm_fwd_workspace_bytes(B, S, C, G), 256-byte aligned (NULL when that is 0).
 */
EL_API el_status el_group_norm_fwd(const void* x, int64_t ldx, int32_t B, int32_t S, int32_t C,
                                   int32_t G, const int32_t* lengths, const float* gamma,
                                   const float* beta, float eps, uint32_t act, void* y, int64_t ldy,
                                   float* mean, float* rstd, el_dtype dtype, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/*
 * Its backward, from the forward's inputs and mean / rstd.  With xh = (x - mean) rstd,
 * du = dy act'(u), dh = du gamma and averages over the n values of a group:
 *   dx        = rstd (dh - avg(dh) - xh avg(dh xh));   +0 at padded positions
 *   dgamma[c] = sum_{b, s} du xh,   dbeta[c] = sum_{b, s} du      (fp32 [C], overwritten;
 *                                                                  either may be NULL)
 * Sums over samples are added in a fixed order: bitwise reproducible.
 */
EL_API el_status el_group_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                   int32_t B, int32_t S, int32_t C, int32_t G,
                                   const int32_t* lengths, const float* gamma, const float* beta,
                                   const float* mean, const float* rstd, uint32_t act, void* dx,
                                   int64_t lddx, float* dgamma, float* dbeta, el_dtype dtype,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EMBTOWER_H */
