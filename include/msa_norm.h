/*
 * msa_norm.h -- the norm ahead of an MSA layer's projection, as a C ABI, for NVIDIA
 * GB300 (sm_103a): RMSNorm of the hidden states with the residual's addition, and an
 * output in FP8 E4M3 with one scale for each token, in bf16, or both.
 *
 * Per token t, over K = hidden_size elements:
 *
 *     h[j]            = x[t, j] + residual[t, j]            (x[t, j] without a residual)
 *     residual_out    = bf16_rne(h)
 *     y[j]            = h[j] * weight[j] / sqrt(sum_j h[j]^2 / K + rms_eps)
 *     out             = bf16_rne(y)
 *     scales[t]       = max(max_j |y[j]|, 2^-100) * (1 / 448)
 *     codes           = e4m3_rne(y * (1 / scales[t]))
 *
 * codes and scales are an E4M3 operand of msa_projection_forward (hidden and
 * hidden_scales).  The norm is taken of h before its rounding to bf16.  Arithmetic is
 * fp32, the two reciprocals among it: a quotient is right to 2^-22, so that a code as near to
 * a tie may be its neighbour.  y is (h * weight) times the reciprocal root: h * weight has to be in
 * the range of fp32.  A row whose sum of squares leaves that range is scaled by a power of two
 * first, so its norm is right too.  A row that holds a NaN or an infinity gets the scale
 * NaN (and out as the formula gives it); a row of zeros with rms_eps 0 gives NaN.
 *
 * Ownership and threading: as for msa_producer_forward.  One kernel is enqueued, which
 * reads and writes memory only after the kernels ahead of it on the stream are complete.
 */
#ifndef MSA_NORM_H
#define MSA_NORM_H

#include <stdint.h>

#include "msa_producer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t hidden_size;  /* K: 1..16384 */
    float rms_eps;        /* >= 0, finite */
    int32_t reserved[2];  /* must be 0 */
} msa_norm_cfg;

/*
 * x              device bf16 [num_tokens, x_stride].
 * residual       device bf16 [num_tokens, residual_stride], or NULL: none.
 * weight         device bf16 [K], 16-byte aligned.
 * residual_out   device bf16 [num_tokens, residual_out_stride], or NULL: not written; NULL
 *                without a residual.
 * out            device bf16 [num_tokens, out_stride], or NULL: not written.
 * codes, scales  device E4M3 [num_tokens, codes_stride] and fp32 [num_tokens], or both
 *                NULL: not written.  At least one of out and codes is given.
 * launch_flags   MSA_LAUNCH_PDL: accepted; the kernel is launched with programmatic dependent
 *                launch in any case.
 *
 * Row strides are in elements, at least K, and multiples of 8 (of codes: 16); the five
 * arrays of rows are 16-byte aligned.  Elements of a row from K on are neither read nor
 * written.  residual_out may be residual or x, and out may be x or residual, with the same
 * row stride as the array that it takes the place of; no other arrays may overlap.
 * num_tokens at most 2^31 - 1; 0 returns MSA_OK and launches nothing.
 */
msa_status msa_norm_forward(const msa_norm_cfg *cfg, int64_t num_tokens, const void *x, int64_t x_stride,
                            const void *residual, int64_t residual_stride, const void *weight,
                            void *residual_out, int64_t residual_out_stride, void *out, int64_t out_stride,
                            void *codes, int64_t codes_stride, float *scales, int32_t launch_flags,
                            cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_NORM_H */
