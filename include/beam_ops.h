/*
 * beam_ops.h -- operators around the MoE block (beam_moe.h) that need no
 * handle: the norm in front of a block, microscaled 4- and 8-bit operands
 * (making, reading and multiplying them) and routing from scores.
 *
 * Memory, streams and errors as in beam_moe.h: every pointer is a device
 * pointer that the caller owns, `stream` is a cudaStream_t passed as void*,
 * calls are stream-ordered and asynchronous, and a call whose arguments are
 * invalid returns a negative beam_status and launches nothing; the text of
 * the last such error on the calling thread is beam_ops_error().  The current
 * CUDA device must be the one that the pointers and the stream belong to.
 * No call allocates memory or keeps any between calls (the one exception is a
 * status word per device, beam_ops_status), so calls may overlap on several
 * streams and be captured into graphs.  Inputs and outputs must not overlap
 * unless a call says so.  Rows that lie `ld` elements apart have ld >= their
 * length; pointers have the alignment of their element type unless stated
 * (16-byte alignment of pointers and rows selects the vector kernels).
 */
#ifndef BEAM_OPS_H
#define BEAM_OPS_H

#include <stdint.h>

#include "beam_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BEAM_BF16 = 0, BEAM_F16 = 1, BEAM_F32 = 2 } beam_dtype;

/*
 * Microscaled formats: blocks of consecutive elements of a row share a scale.
 *   NVFP4  E2M1 elements, an E4M3 scale per 16 (sign bit 0), an FP32 scale per tensor;
 *   MXFP4  E2M1 elements, a power of two (UE8M0 byte: 2^(byte - 127)) per 32;
 *   MXFP8  E4M3 elements, a power of two per 32.
 * Codes: two E2M1 a byte, element 2j of a row in the low nibble of byte j
 * (uint8 [rows, K/2]), as beam_moe_create_nvfp4 takes them; one E4M3 a byte
 * (uint8 [rows, K]).
 */
typedef enum { BEAM_NVFP4 = 0, BEAM_MXFP4 = 1, BEAM_MXFP8 = 2 } beam_mx_format;

/*
 * Layouts of the scale bytes.
 *   ROWS   [rows, K/block], as beam_moe_create_nvfp4 takes them;
 *   TILED  what the tensor cores read: 512-byte tiles of 128 rows x 4 scales,
 *          [ceil(rows/128)][ceil(K/block/4)][32][4][4]: the scale j of row r
 *          is byte (r % 32) * 16 + (r / 32 % 4) * 4 + j % 4 of tile
 *          (r / 128, j / 4).  Bytes of rows and scales past the end are zero.
 */
typedef enum { BEAM_SCALES_ROWS = 0, BEAM_SCALES_TILED = 1 } beam_scale_layout;

/* Bytes of the scales of a [rows, K] operand, or a negative beam_status.
 * K must be a positive multiple of the format's block, rows * K at most 2^60. */
long long beam_mx_scale_bytes(int format, long long rows, int K, int layout);

/*
 * The NVFP4 scale of a tensor x [rows, K] (rows ldx elements apart): the least
 * power of two g with amax <= 6 * 448 * g, where amax is the largest finite
 * magnitude, taken as 2^-100 at least.  A power of two costs at most one of
 * the E4M3 scale's 17 binades and keeps every decision of beam_mx_quantize
 * and every product element * scale * g exact.
 * Elements above 6 * 448 * 2^112 (1.4e37) give a g above 2^112, which
 * beam_mx_quantize does not take; beam_mx_quantize_nvfp4 stops there.
 * tensor_scale  fp32 [1] (out).  rows >= 0, K >= 1; an empty tensor gives the
 *               scale of amax = 2^-100.
 */
int beam_mx_tensor_scale(void *stream, const void *x, int dtype, long long rows, int K,
                         long long ldx, float *tensor_scale);

/*
 * x [rows, K] (dtype, rows ldx elements apart) to codes and scales.
 *   NVFP4   s = E4M3(amax / (6 g)) per block of 16, element = E2M1(x / (s g)),
 *           with g = *tensor_scale (fp32 [1], device; required for NVFP4,
 *           NULL for the others), the quotients rounded to FP32 first (exact
 *           decisions where g is a power of two and x has 16 bits);
 *   MXFP4, MXFP8   the least power of two s = 2^k, k in [-127, 127], with
 *           amax <= 6 s (448 s), element = E2M1(x / s) (E4M3(x / s)): no
 *           finite element saturates.
 * All roundings are to nearest, ties to even.  A block that holds an infinity
 * or a NaN gets the scale NaN (byte 0x7f, UE8M0 0xff) and elements of zero,
 * so each of its values reads back as NaN; so do all blocks of an NVFP4
 * tensor whose g is outside [2^-112, 2^112].  A block of zeros gets the
 * scale byte 0.
 * codes 16-byte and scales 4-byte aligned.  K a positive multiple of the
 * block, rows >= 0 (0: nothing to do).
 */
int beam_mx_quantize(void *stream, const void *x, int dtype, long long rows, int K, long long ldx,
                     int format, int layout, const float *tensor_scale, uint8_t *codes,
                     uint8_t *scales);

/*
 * x to NVFP4 under the scale that beam_mx_tensor_scale finds, 2^112 at most:
 * finite elements beyond 6 * 448 * 2^112 saturate there.  One more pass over x.
 * tensor_scale  fp32 [1], device (out).  The rest as in beam_mx_quantize; with
 *               rows = 0 only tensor_scale is written.
 */
int beam_mx_quantize_nvfp4(void *stream, const void *x, int dtype, long long rows, int K,
                           long long ldx, int layout, float *tensor_scale, uint8_t *codes,
                           uint8_t *scales);

/*
 * The values that codes and scales stand for, out [rows, K] (dtype, rows ldo
 * elements apart): element * block scale * tensor scale (NULL: 1), the
 * product formed in FP32 and rounded once.  Alignment as beam_mx_quantize.
 */
int beam_mx_dequantize(void *stream, const uint8_t *codes, const uint8_t *scales,
                       const float *tensor_scale, int format, int layout, long long rows, int K,
                       void *out, int dtype, long long ldo);

/*
 * Scales in ROWS layout to TILED (a checkpoint's scales, once, for
 * beam_mx_matmul).  tiled 4-byte aligned.
 */
int beam_mx_tile_scales(void *stream, int format, const uint8_t *scales, long long rows, int K,
                        uint8_t *tiled);

/*
 * out [T, N] = a [T, K] . w [N, K]^T, both operands microscaled, on the
 * block-scaled tensor cores (products exact, sums in FP32), times the tensor
 * scales (fp32 [1], device; NULL: 1), rounded once to dtype.
 * Formats (a, w): (NVFP4, NVFP4), (MXFP4, MXFP4), (MXFP8, MXFP4) and
 * (MXFP8, MXFP8); others return BEAM_ERR_UNSUPPORTED.  Scales TILED; codes
 * contiguous rows.  K a positive multiple of 64 for 4-bit a, of 128 for 8-bit
 * a, else BEAM_ERR_UNSUPPORTED.  codes and scales 32-byte aligned.
 * 0 <= T, N < 2^27 (T or N 0: nothing to do).  Results do not depend on the
 * run; a NaN scale gives NaN in the rows or columns it scales.
 */
int beam_mx_matmul(void *stream, int a_format, const uint8_t *a_codes, const uint8_t *a_scales,
                   const float *a_tensor_scale, int w_format, const uint8_t *w_codes,
                   const uint8_t *w_scales, const float *w_tensor_scale, int T, int N, int K,
                   void *out, int dtype, long long ldo);

/*
 * Residual addition and root-mean-square norm of T rows of H elements:
 *     s = alpha * residual + beta * x       (s = beta * x without residual)
 *     y = s / sqrt(mean(s^2) + eps) * gamma
 * in FP32 (where the sum of s^2 overflows, at elements of 1.8e19 and more, the
 * finite elements of the row give y = 0); residual_out = s and out = y, each
 * rounded once.  With
 * alpha = sqrt((k-1)/k), beta = 1/sqrt(k) this is the depth-scaled residual
 * update that beam_moe_forward applies after a block, in front of the next.
 * x            [T, H] x_dtype, rows ldx apart.
 * residual     [T, H] residual_dtype, rows ldr apart, or NULL.
 * residual_out same type, rows ldro apart; may be the same memory as residual
 *              (same ld); required with residual, NULL without.
 *              residual_dtype is BEAM_F32 or x_dtype.
 * gamma        fp32 [H].  eps >= 0.
 * out          [T, H] out_dtype, rows ldo apart, or NULL when codes is given.
 * codes, scales  MXFP8 of y (from FP32, not from the rounded out), as
 *              beam_mx_quantize writes them, in `layout`; both or neither.
 *              H must be a multiple of 32 then.
 * 1 <= H <= 32768 and T <= 2^31 - 256 (else BEAM_ERR_UNSUPPORTED), T >= 0 (0:
 * nothing to do).
 */
int beam_rms_norm(void *stream, const void *x, int x_dtype, long long ldx, const void *residual,
                  int residual_dtype, long long ldr, void *residual_out, long long ldro,
                  float alpha, float beta, const float *gamma, float eps, int T, int H, void *out,
                  int out_dtype, long long ldo, uint8_t *codes, uint8_t *scales, int layout);

typedef enum { BEAM_SCORE_SIGMOID = 0, BEAM_SCORE_SOFTMAX = 1 } beam_score;

/*
 * Experts and weights of T tokens from router logits fp32 [T, E] (rows ldl
 * apart), for routers of other forms than the handle's (beam_moe_route_logits):
 *   p    sigmoid(logit), or the softmax over the row's experts;
 *   key  p + bias (fp32 [E] or NULL: p); the bias steers the choice only;
 *   with topk_group < n_group: the experts form n_group groups of
 *        E / n_group consecutive ones, a group's score is the sum of its
 *        group_top (1 or 2) largest keys, the topk_group best groups stay;
 *   the top_k largest keys are chosen, in descending order;
 *   w    p of the chosen, divided by their sum if renormalize, times scale.
 * Ties go to the lower index.  The choices are those of 64-bit arithmetic on
 * the FP32 logits and biases: where FP32 keys are too close to tell, the row
 * is decided in 64 bits, and keys or group scores that are equal there (sums
 * with sigmoids that saturate at 1, groups whose softmax is below 2^-1074) tie.
 * Without a bias experts are ordered by their logits, which are exact.
 * The handle's router (beam_moe_route, beam_moe_route_logits) decides such near
 * ties in FP32, so the two may choose differently there (below 1% of rows of
 * random logits).  Use the handle's with a handle's block, so that routing and
 * block agree with what the block does by itself, and this one for logits of
 * other routers, softmax, masks and other group rules.
 * An expert whose logit is -inf is masked: it has p = 0, is never chosen, and
 * counts for no group; a bias of -inf does the latter two.  Slots that no
 * expert is left for get index -1 and weight 0.  A row that holds a NaN, or +inf under softmax, or
 * is given a NaN bias, gets index -1 and weight NaN in every slot.
 * 1 <= E <= 1024, n_group <= 32 and a divisor of E, 1 <= topk_group <=
 * n_group, group_top 1 or 2, 1 <= top_k <= min(32, topk_group * E / n_group),
 * scale finite.  T == 0 launches nothing.
 */
int beam_route_scores(void *stream, const float *logits, int T, int E, long long ldl, int score,
                      const float *bias, int n_group, int topk_group, int group_top, int top_k,
                      int renormalize, float scale, int32_t *topk_idx, float *topk_w);

/*
 * Synchronise `stream`, then return and clear the current device's status
 * word of these operators: BEAM_OK, or BEAM_ERR_TIMEOUT when a bounded wait
 * inside beam_mx_matmul ran out since the last call.  The result of that
 * product, and of those that ran after it before this call, is not valid.  The
 * word is read and cleared in one step: one of several callers gets an event.
 * A stream that is being captured is refused (BEAM_ERR_INVALID_ARG) and its
 * capture goes on.
 */
int beam_ops_status(void *stream);

/*
 * For tests of the bounded waits: the calling thread's next beam_mx_matmul that
 * launches waits in stage `stage` of K (256 4-bit or 128 8-bit elements a stage;
 * -1: none) for bytes that do not come, limit_ms (1 .. 2000) at a wait.  Where it
 * has that stage it ends within some 20 such limits, its result is not valid
 * and beam_ops_status reports BEAM_ERR_TIMEOUT.
 */
int beam_ops_debug_withhold(int stage, int limit_ms);

/* Text of the last host-side error of a call above on the calling thread. */
const char *beam_ops_error(void);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_OPS_H */
