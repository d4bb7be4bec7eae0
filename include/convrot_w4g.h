/*
 * convrot_w4g.h -- C ABI of the group-scaled few-token variant of the rotated
 * linear layer (library libconvrot_w4g.so): bf16 activations times packed
 * INT4 weights that carry one bf16 scale per group of 32, 64 or 128 channels
 * instead of one per row.
 *
 * Weights (offline):
 *   1. y = w R, R = I (x) H_group as in convrot.h (group = 64 or 256), or
 *      y = w with group = 0 (weights that are not rotated, or already are);
 *   2. for every block b of scale_group channels of a row, a = max |y|,
 *          s = bf16_rne(a / 7)   (0 where that is below 2^-100),
 *          q = clamp(round_half_away(y * (1 / s)), -7, 7)   (fp32; s = 0: 0),
 *      packed as in convrot.h (two codes per byte, low nibble = even channel,
 *      4-bit two's complement).  The scale is rounded before the codes are
 *      chosen, so the codes make up for its rounding.
 * Activations: xr = x R (fp32), or x with group = 0, held as 16-bit whole
 * numbers with one fp32 factor for every 256 channels of a row: off by at most
 * 2^-16 of the largest of the 256.  Product:
 *      y[m][n] = bf16_rne( sum_b s[n][b] (sum_{k in b} xr[m][k] q[n][k])
 *                          + bias[n] ),
 * with exact sums inside a scale group and fp32 beyond.  256 channels whose
 * largest value is below 2^-100 count as 0; a row with a NaN or an infinity,
 * or whose sums over a group are not finite (of values beyond 2^119 they may
 * not be), gives NaN.
 *
 * Conventions are those of convrot.h: device pointers on the current device,
 * row-major, contiguous, 16-byte aligned; the caller owns every buffer and the
 * library allocates nothing; work is enqueued on `stream`; arguments are
 * validated before any launch; M = 0 or N = 0 is a no-op; results are
 * deterministic.  A buffer that a call writes overlaps no other
 * (CONVROT_ERR_OVERLAP).  64 <= K <= CONVROT_MAX_K, K a multiple of 64, of `group`
 * where that is not 0, and of scale_group.  CONVROT_ERR_GROUP: group is not
 * 0, 64 or 256, or scale_group is not 32, 64 or 128.
 */
#ifndef CONVROT_W4G_H_
#define CONVROT_W4G_H_

#include "convrot.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Weights: w_bf16 [N][K] bf16 -> qw [N][K/2] codes and sg_bf16
 * [N][K/scale_group] bf16 scales.  One kernel.
 */
convrot_status convrot_w4g_quantize_weight(const void *w_bf16, int64_t N, int64_t K, int group,
                                           int scale_group, uint8_t *qw, void *sg_bf16,
                                           convrot_stream_t stream);

/* Bytes of workspace convrot_w4g_linear needs for the activations' numbers
 * and factors, or 0 where a few short rows need none (and for M <= 0 or
 * K <= 0).  Host-only. */
size_t convrot_w4g_workspace_size(int64_t M, int64_t K);

/*
 * The whole layer: x_bf16 [M][K] bf16, qw [N][K/2], sg_bf16
 * [N][K/scale_group], bias_bf16 [N] bf16 or NULL (zeros), y_bf16 [M][N].
 * workspace: at least convrot_w4g_workspace_size(M, K) bytes, 256-byte
 * aligned (CONVROT_ERR_WORKSPACE otherwise; may be NULL where that is 0).
 * Made for few tokens: every 16 tokens read the weights once.  Any M is
 * accepted.
 */
convrot_status convrot_w4g_linear(const void *x_bf16, const uint8_t *qw, const void *sg_bf16,
                                  const void *bias_bf16, int64_t M, int64_t N, int64_t K,
                                  int group, int scale_group, void *workspace, size_t ws_bytes,
                                  void *y_bf16, convrot_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_W4G_H_ */
