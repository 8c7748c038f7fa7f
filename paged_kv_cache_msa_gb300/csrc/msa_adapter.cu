// Low-rank adapters of many requests beside a shared projection (include/msa_adapter.h).
//
// Two kernels: the down-projection of every token with its own adapter into a workspace, and
// the up-projection added to the rows.

#include "msa_adapter.h"
#include "msa_internal.h"

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

namespace {

struct Params {
    const uint8_t *hidden;
    const float *hidden_scales;
    const uint16_t *down, *up;
    const int32_t *ids;
    const float *adapter_scales;
    const uint16_t *rows;
    uint16_t *out;
    float *u;                        // [T, S * r]
    int64_t hidden_stride, down_stride, rows_stride, out_stride;   // elements
    int64_t num_tokens;
    int32_t hidden_size, width, rank, num_adapters, num_slices, fp8;
    int32_t slice_end[MSA_ADAPTER_MAX_SLICES];
};

__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float x)
{
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    return h;
}

// A warp for each (token, row of down): lanes along K.
__global__ void __launch_bounds__(256) msa_adapter_down_kernel(const __grid_constant__ Params p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const int64_t t = blockIdx.x;
    const int a = p.ids[t];
    if (a < 0 || a >= p.num_adapters)
        return;
    const int n = p.num_slices * p.rank;
    const float c = (p.hidden_scales ? p.hidden_scales[t] : 1.0f) * (p.adapter_scales ? p.adapter_scales[a] : 1.0f);
    for (int i = threadIdx.x / 32; i < n; i += 8) {
        const uint16_t *row = p.down + ((int64_t)a * n + i) * p.down_stride;
        float s = 0.0f;
        for (int k = threadIdx.x % 32; k < p.hidden_size; k += 32) {
            const int64_t e = t * p.hidden_stride + k;
            __nv_fp8_e4m3 code;
            code.__x = p.fp8 ? p.hidden[e] : 0;
            const float x = p.fp8 ? float(code) : bf16_to_f32(reinterpret_cast<const uint16_t *>(p.hidden)[e]);
            s = fmaf(x, bf16_to_f32(row[k]), s);
        }
        for (int o = 16; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x % 32 == 0)
            p.u[t * n + i] = s * c;
    }
}

// A thread for each output.
__global__ void __launch_bounds__(256) msa_adapter_up_kernel(const __grid_constant__ Params p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const int64_t t = blockIdx.x;
    const int a = p.ids[t];
    const bool on = a >= 0 && a < p.num_adapters;
    for (int j = threadIdx.x; j < p.width; j += 256) {
        const uint16_t r = p.rows[t * p.rows_stride + j];
        if (!on) {
            p.out[t * p.out_stride + j] = r;
            continue;
        }
        int s = 0;
        while (j >= p.slice_end[s])
            ++s;
        const uint16_t *up = p.up + ((int64_t)a * p.width + j) * p.rank;
        const float *u = p.u + (t * p.num_slices + s) * p.rank;
        float d = 0.0f;
        for (int i = 0; i < p.rank; ++i)
            d = fmaf(u[i], bf16_to_f32(up[i]), d);
        p.out[t * p.out_stride + j] = f32_to_bf16(bf16_to_f32(r) + d);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t kMaxTokens = 1 << 24;

msa_status fail(msa_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
msa_status fail(msa_status s, const char *fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    msa_internal_set_detail(buf);
    return s;
}

msa_status check_cfg(const msa_adapter_cfg *cfg, int64_t T)
{
    msa_internal_set_detail("");
    if (!cfg)
        return fail(MSA_ERR_INVALID_ARGUMENT, "cfg is NULL");
    if (cfg->hidden_size < 1)
        return fail(MSA_ERR_INVALID_ARGUMENT, "hidden_size %d", cfg->hidden_size);
    if (cfg->rank < 1)
        return fail(MSA_ERR_INVALID_ARGUMENT, "rank %d", cfg->rank);
    if (cfg->rank % 8 || cfg->rank > 128)
        return fail(MSA_ERR_UNSUPPORTED, "rank %d (multiples of 8, at most 128)", cfg->rank);
    if (cfg->num_adapters < 1)
        return fail(MSA_ERR_INVALID_ARGUMENT, "num_adapters %d", cfg->num_adapters);
    if (cfg->hidden_dtype != MSA_DTYPE_BF16 && cfg->hidden_dtype != MSA_DTYPE_FP8_E4M3)
        return fail(MSA_ERR_UNSUPPORTED, "hidden_dtype %d", cfg->hidden_dtype);
    if (cfg->num_slices < 1 || cfg->num_slices > MSA_ADAPTER_MAX_SLICES)
        return fail(MSA_ERR_INVALID_ARGUMENT, "num_slices %d (1..%d)", cfg->num_slices, MSA_ADAPTER_MAX_SLICES);
    if (cfg->num_slices * cfg->rank > 512)
        return fail(MSA_ERR_UNSUPPORTED, "num_slices * rank is %d (at most 512)", cfg->num_slices * cfg->rank);
    for (int s = 0; s < MSA_ADAPTER_MAX_SLICES; ++s) {
        const int end = cfg->slice_end[s], last = s == cfg->num_slices - 1;
        if (s >= cfg->num_slices ? end != 0 : end <= (s ? cfg->slice_end[s - 1] : 0))
            return fail(MSA_ERR_INVALID_ARGUMENT, "slice_end[%d] is %d", s, end);
        if (end % (last ? 8 : 64))
            return fail(MSA_ERR_UNSUPPORTED, "slice_end[%d] is %d (a multiple of %d)", s, end, last ? 8 : 64);
    }
    for (int i = 0; i < 3; ++i)
        if (cfg->reserved[i] != 0)
            return fail(MSA_ERR_INVALID_ARGUMENT, "cfg reserved fields must be 0");
    if (T < 0)
        return fail(MSA_ERR_INVALID_ARGUMENT, "num_tokens %lld", (long long)T);
    if (T > kMaxTokens)
        return fail(MSA_ERR_UNSUPPORTED, "num_tokens %lld (at most 2^24)", (long long)T);
    return MSA_OK;
}

int width_of(const msa_adapter_cfg *cfg) { return cfg->slice_end[cfg->num_slices - 1]; }

int64_t workspace_needed(const msa_adapter_cfg *cfg, int64_t T)
{
    return T * cfg->num_slices * cfg->rank * 4;
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// a * b * c as non-negative int64
bool fits(int64_t a, int64_t b, int64_t c)
{
    int64_t m;
    return !__builtin_mul_overflow(a, b, &m) && !__builtin_mul_overflow(m, c, &m);
}

msa_status check_args(const msa_adapter_cfg *cfg, int64_t T, const Params &p, const void *workspace,
                      int64_t workspace_bytes, int32_t flags)
{
    const msa_status s = check_cfg(cfg, T);
    if (s != MSA_OK)
        return s;
    if (flags & ~MSA_LAUNCH_PDL)
        return fail(MSA_ERR_INVALID_ARGUMENT, "unknown launch flag bits 0x%x", flags);
    if (T == 0)
        return MSA_OK;
    const int64_t K = cfg->hidden_size, W = width_of(cfg), es = cfg->hidden_dtype == MSA_DTYPE_BF16 ? 2 : 1;
    if (!p.hidden || !p.down || !p.up || !p.ids || !p.rows || !p.out)
        return fail(MSA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (p.hidden_stride < K || p.down_stride < K || p.rows_stride < W || p.out_stride < W)
        return fail(MSA_ERR_INVALID_ARGUMENT, "a row stride is less than the row's elements");
    if (p.out == p.rows && p.out_stride != p.rows_stride)
        return fail(MSA_ERR_INVALID_ARGUMENT, "out in the place of rows has another row stride");
    if (p.hidden_stride * es % 16 || p.down_stride % 8 || p.rows_stride % 8 || p.out_stride % 8)
        return fail(MSA_ERR_MISALIGNED, "row strides must be multiples of 16 bytes");
    if (!aligned(p.hidden, 16) || !aligned(p.down, 16) || !aligned(p.up, 16) || !aligned(p.rows, 16) ||
        !aligned(p.out, 16))
        return fail(MSA_ERR_MISALIGNED, "hidden, down, up, rows and out must be 16-byte aligned");
    if (!aligned(p.ids, 4) || !aligned(p.hidden_scales, 4) || !aligned(p.adapter_scales, 4))
        return fail(MSA_ERR_MISALIGNED, "adapter_ids or scales misaligned");
    if (!fits(T, p.hidden_stride, 2) || !fits(T, p.rows_stride, 2) || !fits(T, p.out_stride, 2) ||
        !fits((int64_t)cfg->num_adapters * cfg->num_slices * cfg->rank, p.down_stride, 2))
        return fail(MSA_ERR_OFFSET_OVERFLOW, "an extent overflows int64");
    if (!workspace || workspace_bytes < workspace_needed(cfg, T))
        return fail(MSA_ERR_INVALID_ARGUMENT, "workspace: %lld bytes, %lld needed",
                    (long long)(workspace ? workspace_bytes : 0), (long long)workspace_needed(cfg, T));
    if (!aligned(workspace, 256))
        return fail(MSA_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    return MSA_OK;
}

msa_status launch(void (*kernel)(Params), dim3 grid, int threads, int smem, bool pdl, cudaStream_t stream, Params &p)
{
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    lc.gridDim = grid;
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = (size_t)smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 1 : 0;
    void *args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(&lc, reinterpret_cast<const void *>(kernel), args);
    if (e != cudaSuccess)
        return fail(MSA_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
    return MSA_OK;
}

}  // namespace

extern "C" {

msa_status msa_adapter_workspace_bytes(const msa_adapter_cfg *cfg, int64_t num_tokens, int64_t *bytes)
{
    const msa_status s = check_cfg(cfg, num_tokens);
    if (s != MSA_OK)
        return s;
    if (!bytes)
        return fail(MSA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    *bytes = workspace_needed(cfg, num_tokens);
    return MSA_OK;
}

msa_status msa_adapter_forward(const msa_adapter_cfg *cfg, int64_t num_tokens, const void *hidden,
                               int64_t hidden_stride, const float *hidden_scales, const void *down,
                               int64_t down_stride, const void *up, const int32_t *adapter_ids,
                               const float *adapter_scales, const void *rows, int64_t rows_stride, void *out,
                               int64_t out_stride, void *workspace, int64_t workspace_bytes,
                               int32_t launch_flags, cudaStream_t stream)
{
    Params p;
    memset(&p, 0, sizeof p);
    p.hidden = static_cast<const uint8_t *>(hidden);
    p.hidden_scales = hidden_scales;
    p.down = static_cast<const uint16_t *>(down);
    p.up = static_cast<const uint16_t *>(up);
    p.ids = adapter_ids;
    p.adapter_scales = adapter_scales;
    p.rows = static_cast<const uint16_t *>(rows);
    p.out = static_cast<uint16_t *>(out);
    p.u = static_cast<float *>(workspace);
    p.hidden_stride = hidden_stride;
    p.down_stride = down_stride;
    p.rows_stride = rows_stride;
    p.out_stride = out_stride;
    const msa_status s = check_args(cfg, num_tokens, p, workspace, workspace_bytes, launch_flags);
    if (s != MSA_OK || num_tokens == 0)
        return s;
    p.num_tokens = num_tokens;
    p.hidden_size = cfg->hidden_size;
    p.width = width_of(cfg);
    p.rank = cfg->rank;
    p.num_adapters = cfg->num_adapters;
    p.num_slices = cfg->num_slices;
    p.fp8 = cfg->hidden_dtype == MSA_DTYPE_FP8_E4M3;
    memcpy(p.slice_end, cfg->slice_end, sizeof p.slice_end);
    const msa_status d = launch(msa_adapter_down_kernel, dim3((unsigned)num_tokens), 256, 0,
                                launch_flags & MSA_LAUNCH_PDL, stream, p);
    return d != MSA_OK ? d : launch(msa_adapter_up_kernel, dim3((unsigned)num_tokens), 256, 0, true, stream, p);
}

}  // extern "C"
