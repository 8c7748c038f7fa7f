/*
 * msa_adapter.h -- low-rank adapters of many requests at once beside a shared packed
 * projection, as a C ABI, for NVIDIA GB300 (sm_103a).
 *
 * A projection's rows [Q | K | V | index-Q | index-K] (msa_projection_forward's rows_out,
 * or any GEMM's) are of width W, cut into slices; each slice has a down-projection of its
 * own.  Per token t with a = adapter_ids[t], for output j in slice s:
 *
 *     u[t, i]   = hidden_scales[t] * sum_k hidden[t, k] * down[a, s * rank + i, k]     i < rank
 *     out[t, j] = bf16_rne(rows[t, j] + adapter_scales[a] * sum_i up[a, j, i] * u[t, i])
 *
 * and out[t, :] = rows[t, :] where a is not in [0, num_adapters): a request without an
 * adapter.  What one request's adapter holds, NaN and infinities among it, never reaches
 * another request's row.  An adapter of a smaller rank is padded with zero rows of down
 * and zero columns of up.  msa_producer_forward (or msa_producer_axes_forward) of out is
 * the layer's producer with every request's adapter.
 *
 * Arithmetic: sums are fp32.  The second product runs on the tensor cores, where u is split
 * into three bf16 parts that hold all of its bits; a part may be 0, so that an infinite element of
 * up gives NaN where the formula in fp32 has an infinity.  Results do not depend on which
 * other calls run, and a call repeated with the same arguments gives the same bits.  A wait inside
 * a kernel that runs out of time (a failure of the hardware, never expected) makes the outputs of
 * its tokens NaN.
 *
 * Ownership and threading: as for msa_producer_forward; the workspace as the attention
 * operators' (it need not be initialised and carries nothing from one call to the next;
 * calls or graph replays that may run at the same time need separate ones).  The kernels
 * read and write memory only after the kernels ahead of them on the stream are complete.
 */
#ifndef MSA_ADAPTER_H
#define MSA_ADAPTER_H

#include <stdint.h>

#include "msa_producer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MSA_ADAPTER_MAX_SLICES 8

typedef struct {
    int32_t hidden_size;    /* K: 1..2^30 */
    int32_t rank;           /* a multiple of 8, 8..128 */
    int32_t num_adapters;   /* 1..16384 */
    int32_t hidden_dtype;   /* msa_dtype of hidden: bf16 or E4M3 */
    int32_t num_slices;     /* 1..MSA_ADAPTER_MAX_SLICES; num_slices * rank <= 512 */
    int32_t slice_end[MSA_ADAPTER_MAX_SLICES]; /* ascending; all but the last multiples of 64,
                               the last (the width W) a multiple of 8, at most
                               2^30; then 0 */
    int32_t reserved[3];    /* must be 0 */
} msa_adapter_cfg;

/* Bytes of workspace that serve msa_adapter_forward for any number of tokens up to num_tokens
 * under cfg: less than 2 MB and 512 bytes an adapter, and at most 32 * num_slices * rank + 80
 * bytes a token.  Host-side; enqueues nothing. */
msa_status msa_adapter_workspace_bytes(const msa_adapter_cfg *cfg, int64_t num_tokens, int64_t *bytes);

/*
 * hidden         device bf16 or E4M3 [num_tokens, hidden_stride]; 16-byte aligned, the row
 *                stride (elements) a multiple of 16 bytes, >= K.  Elements from K on are not read.
 * hidden_scales  device fp32 [num_tokens], or NULL: 1.
 * down           device bf16 [num_adapters, num_slices * rank, down_stride], 16-byte aligned,
 *                down_stride a multiple of 8, >= K, below 2^39.
 * up             device bf16 [num_adapters, W, rank], 16-byte aligned.
 * adapter_ids    device int32 [num_tokens], in any order.
 * adapter_scales device fp32 [num_adapters], or NULL: 1.
 * rows, out      device bf16 [num_tokens, rows_stride], [num_tokens, out_stride]; 16-byte
 *                aligned, strides multiples of 8, >= W.  out may be rows (with the same
 *                stride); otherwise they must not overlap.
 * workspace      device, 256-byte aligned; msa_adapter_workspace_bytes(cfg, num_tokens) bytes do.
 * launch_flags   MSA_LAUNCH_PDL: accepted; the kernels are launched with programmatic dependent
 *                launch in any case.
 *
 * num_tokens at most 2^24; 0 returns MSA_OK and launches nothing.
 */
msa_status msa_adapter_forward(const msa_adapter_cfg *cfg, int64_t num_tokens, const void *hidden,
                               int64_t hidden_stride, const float *hidden_scales, const void *down,
                               int64_t down_stride, const void *up, const int32_t *adapter_ids,
                               const float *adapter_scales, const void *rows, int64_t rows_stride, void *out,
                               int64_t out_stride, void *workspace, int64_t workspace_bytes,
                               int32_t launch_flags, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_ADAPTER_H */
