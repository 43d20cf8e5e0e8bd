/*
 * embblock.h -- C ABI of the operators of a normalised residual block, next to the tower operators
 * of embtower.h: the norms behind one block and before the next with the block's gate and residual
 * scale, activations kept in 8 bits between the forward and the backward pass, and the dense layer
 * on microscaled 4-bit weights and activations.  Built into the same library; every convention of
 * embtower.h holds (device pointers unless marked [host], caller-owned memory, work enqueued on
 * `stream`, host-side validation before anything is enqueued, no aliasing of outputs with inputs,
 * bitwise reproducible results, round to nearest even, data pointers aligned to their elements,
 * 64-bit row strides), except that packed data has the alignment stated for it.
 */
#ifndef EMBBLOCK_H
#define EMBBLOCK_H

#include "embtower.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Norms of a row of C values: n(v) = (v - mean) rstd,
 *   EL_NORM_RMS    mean = 0,            rstd = 1 / sqrt(sum v^2 / C + eps)
 *   EL_NORM_LAYER  mean = sum v / C,    rstd = 1 / sqrt(sum (v - mean)^2 / C + eps)
 *   EL_NORM_NONE   n(v) = v */
enum { EL_NORM_NONE = 0u, EL_NORM_RMS = 1u, EL_NORM_LAYER = 2u };

/* What is done to the gate's values before they multiply: nothing, or 1 / (1 + exp(-u)). */
enum { EL_GATE_NONE = 0u, EL_GATE_SIGMOID = 1u };

/* The parameters of the norms around one residual block. */
typedef struct {
  uint32_t post, pre; /* EL_NORM_*: behind this block; before the next (EL_NORM_RMS or _LAYER) */
  uint32_t gate_act;  /* EL_GATE_* */
  int32_t gate_rows;  /* rows m that share row m / gate_rows of the gate, >= 1 */
  float scale, eps;   /* both finite, eps >= 0 */
  const float *post_gamma, *post_beta; /* fp32 [C] or NULL (1, 0) */
  const float *pre_gamma, *pre_beta;   /* fp32 [C] or NULL (1, 0) */
} el_block_norm;

/*
 * The seam between two residual blocks, in one pass over the rows:
 *   t = post_gamma post(f) + post_beta
 *   y = x + scale gate_act(gate[m / gate_rows]) t          (y is the residual stream)
 *   h = pre_gamma pre(y) + pre_beta                        (h is the next block's input)
 * f NULL: y = x, so only h is computed (gate and y are then NULL).  x NULL: y = scale gate t.
 * gate NULL: 1.  y, h: either may be NULL, not both.  x, f, gate, y, h: rows of strides ldx, ..., of
 * dtype (EL_F32 / EL_F16 / EL_BF16), C columns; the gate has ceil(M / gate_rows) rows.
 * post_stats, pre_stats: fp32 [M][2], mean and rstd of each row (8-byte aligned), or NULL: not
 * stored; pre_stats needs h, post_stats needs post != EL_NORM_NONE.  fp32 arithmetic; h comes from
 * the fp32 y; one rounding each.  C from 1 to 32768 (EL_ERR_UNSUPPORTED beyond).  Values beyond
 * 2^63 / sqrt(C) in magnitude overflow the sums of squares.
 */
EL_API el_status el_block_norm_fwd(const el_block_norm* p, const void* x, int64_t ldx, const void* f,
                                   int64_t ldf, const void* gate, int64_t ldg, int32_t M, int32_t C,
                                   void* y, int64_t ldy, void* h, int64_t ldh, float* post_stats,
                                   float* pre_stats, el_dtype dtype, hipStream_t stream);

/* [host, pure] Bytes of device workspace el_block_norm_bwd needs; 0 for invalid sizes or M == 0. */
EL_API size_t el_block_norm_bwd_workspace_bytes(int32_t M, int32_t C, int32_t gate_rows);

/*
 * Its backward, from the stored y (x where f was NULL), f, gate and statistics.  With
 * yh = pre(y), fh = post(f), a = pre_gamma dh, averages over a row's C values (avg(.) of the first
 * power only for EL_NORM_LAYER):
 *   D  = dy + rstd (a - avg(a) - yh avg(a yh))              dx = D
 *   u  = scale gate_act(gate) D,   b = post_gamma u
 *   df = rstd' (b - avg(b) - fh avg(b fh))                  (df = b for EL_NORM_NONE)
 *   dgate[r]    = gate_act'(gate[r]) sum over its rows of scale D t
 *   dpre_gamma  = sum_m dh yh,  dpre_beta  = sum_m dh       (fp32 [C], overwritten)
 *   dpost_gamma = sum_m u fh,   dpost_beta = sum_m u        (fp32 [C], overwritten)
 * dy or dh may be NULL (0), not both; dh NULL: y and pre_stats are not needed.  Every output may be
 * NULL; df, dgate and the dpost_* need f (and the gate for dgate); dpre_* need dh.  Sums are added in
 * a fixed order, which depends on the sizes, on gate_rows with a gate, on whether every row is 16-byte
 * aligned and on whether post_beta is given or a beta's gradient asked for (the other outputs may be
 * asked for one at a time or together).  workspace: >= el_block_norm_bwd_workspace_bytes, 256-byte
 * aligned.
 */
EL_API el_status el_block_norm_bwd(const el_block_norm* p, const void* dy, int64_t lddy, const void* dh,
                                   int64_t lddh, const void* y, int64_t ldy, const void* f, int64_t ldf,
                                   const void* gate, int64_t ldg, int32_t M, int32_t C,
                                   const float* post_stats, const float* pre_stats, void* dx,
                                   int64_t lddx, void* df, int64_t lddf, void* dgate, int64_t lddg,
                                   float* dpost_gamma, float* dpost_beta, float* dpre_gamma,
                                   float* dpre_beta, el_dtype dtype, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/*
 * Microscaled numbers (the MX formats of the Open Compute Project): 32 consecutive columns of a row
 * share a scale 2^e, stored as the byte e + 127 with e >= -126: the smallest for which the largest
 * finite magnitude of the block is at most T 2^e.  Every value / 2^e is rounded to the nearest
 * number of the format, ties to even.
 *   8 bits: e4m3, T = 448.  A NaN or an infinity becomes the NaN of e4m3, its neighbours stay.
 *   4 bits: e2m1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives), T = 6, two to a byte, the even
 *           column in the low half.  A block that holds a NaN or an infinity has the scale byte 255
 *           and stands for NaN altogether.
 * Magnitudes that round to 2^128 (from 2^128 (1 - 2^-5) in 8 bits, 2^128 (1 - 2^-3) in 4) stand for
 * infinity in fp32; in 8 bits, fp16's magnitudes from 63488 round to 2^16, infinity in EL_F16.
 * Columns behind the last are zeros up to the padded width Kp: whole blocks.
 *   8 bits: codes [M][Kp], scales [M][Kp / 32], Kp = K rounded up to 32.
 *   4 bits: in the order that the matrix instructions take, rows padded with zeros to 32, Kp = K
 *           rounded up to 128 for the codes and to 512 for the scales.  Codes [M / 32][Kp / 128][2]
 *           [64][16]: lane l of fragment i holds the 16 bytes of block l / 16 (of a step of 128
 *           columns) of row 8 (l % 16 / 4) + 4 i + l % 4 (of 32).  Scales [M / 32][Kp / 512][2][64][4]:
 *           the same lanes, their blocks' scales of four steps.
 * Codes are 16-byte aligned, scales 4-byte aligned.  K from 1 to 2^20, padded rows times padded
 * columns of codes <= 2^34 (EL_ERR_UNSUPPORTED beyond).
 */

/* x [M] rows of stride ldx, K columns, of dtype -> 8 bits. */
EL_API el_status el_ckpt_pack(const void* x, int64_t ldx, int32_t M, int32_t K, el_dtype dtype,
                              uint8_t* codes, uint8_t* scales, hipStream_t stream);

/* From a kept activation xq, y = drop(act(xq)) (the forward's output computed again; with
 * EL_ACT_NONE and no dropout the kept values themselves) and its gradient dx = drop(dy act'(xq)),
 * the masks of el_act_dropout_fwd / _bwd.  ReLU'(0) = 0 and ReLU(NaN) = 0, as theirs (an infinity is
 * kept as NaN).  GELU for EL_F32 is accurate relative to its value, also in the negative tail. */
EL_API el_status el_ckpt_act_dropout_fwd(const uint8_t* codes, const uint8_t* scales, int32_t M, int32_t K,
                                         uint32_t act, const el_dropout* drop, void* y, int64_t ldy,
                                         el_dtype dtype, hipStream_t stream);
EL_API el_status el_ckpt_act_dropout_bwd(const void* dy, int64_t lddy, const uint8_t* codes,
                                         const uint8_t* scales, int32_t M, int32_t K, uint32_t act,
                                         const el_dropout* drop, void* dx, int64_t lddx, el_dtype dtype,
                                         hipStream_t stream);

/* [host, pure] Bytes of device workspace el_dense_bwd_ckpt can need; 0 for invalid or unsupported
 * sizes or M == 0. */
EL_API size_t el_dense_bwd_ckpt_workspace_bytes(int32_t M, int32_t K, int32_t N);

/*
 * el_dense_bwd with the layer's input x and the layer below's pre-activation read from 8 bits:
 *   dw = dz^T xq,  db = sum dz,  dx = dz w + dres,  dzb = drop(dx act'(preq))
 * x_codes, x_scales, pre_codes, pre_scales: [M] rows of K columns as el_ckpt_pack writes them
 * (pre_* NULL with EL_ACT_NONE or without dzb).  xq enters the products in dtype: exactly where it
 * was packed from dtype, but for EL_F16 the magnitudes that round to 2^16, as infinities; otherwise
 * rounded (EL_BF16: magnitudes below its subnormals alone).  Everything else as in el_dense_bwd, its
 * limits and reproducibility included.
 */
EL_API el_status el_dense_bwd_ckpt(const uint8_t* x_codes, const uint8_t* x_scales, int32_t M, int32_t K,
                                   const void* w, int32_t N, const void* dz, int64_t lddz,
                                   const void* dres, int64_t lddres, void* dx, int64_t lddx, uint32_t act,
                                   const el_dropout* drop, const uint8_t* pre_codes,
                                   const uint8_t* pre_scales, void* dzb, int64_t lddzb, float* dw,
                                   float* db, el_dtype dtype, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/* x [M] rows of stride ldx, K columns, of dtype -> 4 bits, and back: y holds the values that the
 * codes stand for, rounded once to dtype. */
EL_API el_status el_fp4_pack(const void* x, int64_t ldx, int32_t M, int32_t K, el_dtype dtype,
                             uint8_t* codes, uint8_t* scales, hipStream_t stream);
EL_API el_status el_fp4_unpack(const uint8_t* codes, const uint8_t* scales, int32_t M, int32_t K, void* y,
                               int64_t ldy, el_dtype dtype, hipStream_t stream);

/* [host, pure] Bytes of device workspace el_dense_fwd_fp4 can need; 0 for invalid or unsupported
 * sizes or M == 0, and where the rows are rounded within the product's launch. */
EL_API size_t el_dense_fwd_fp4_workspace_bytes(int32_t M, int32_t K, int32_t N);

/*
 * The serving form of el_dense_fwd on 4 bits:
 *   y[m][n] = residual[m][n] + act(sum_k x4[m][k] w4[n][k] + bias[n])
 * x: [M] rows of stride ldx of dtype (EL_BF16 or EL_F16), rounded to 4 bits within the call (x4 is
 * what el_fp4_pack makes of it); w_codes, w_scales: [N] rows of K columns from el_fp4_pack; bias:
 * fp32 [N] or NULL; residual (or NULL), y: rows of strides ldr, ldy, of dtype.  Products of 4-bit
 * numbers are exact and accumulate in fp32 (block-scaled MFMA); one rounding.  A NaN block makes
 * every output of its row (of x) or column (of w) NaN, under every activation.  N, K <= 2^20, N K < 2^29 and
 * ceil(M/256) ceil(N/256) < 2^21 (EL_ERR_UNSUPPORTED beyond).  workspace: >=
 * el_dense_fwd_fp4_workspace_bytes(M, K, N), 256-byte aligned (NULL when that is 0).
 */
EL_API el_status el_dense_fwd_fp4(const void* x, int64_t ldx, int32_t M, int32_t K, const uint8_t* w_codes,
                                  const uint8_t* w_scales, const float* bias, int32_t N, uint32_t act,
                                  const void* residual, int64_t ldr, void* y, int64_t ldy, el_dtype dtype,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EMBBLOCK_H */
