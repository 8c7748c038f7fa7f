// RMSNorm of the hidden states with the residual's addition, and an E4M3 output with one
// scale for each token (include/msa_norm.h).
//
// The work is streaming: 7 bytes an element are moved (x, residual, residual_out, codes)
// for about ten operations, so HBM bandwidth bounds it, and at a few tokens the chain of
// one load, one reduction over the row and one store.
//   * A row is read once, into the registers of `threads_per_row` threads: vectors of 8
//     elements, up to seven a thread, all their loads issued before the first is used.
//   * The largest |y| needs no second pass: y = fl(fl(h w) r) with r > 0, and rounding is
//     monotone, so max |y| = fl(max |fl(h w)| r), and the sum of squares and the maximum of
//     |h w| go through one reduction with one barrier (none for rows of one warp).  The maximum
//     is taken of the bit patterns, which order as the magnitudes do, NaN above infinity.
//   * A row's partial sums are added in the order of the warps by every thread: the result
//     does not depend on the schedule.

#include "msa_norm.h"
#include "msa_internal.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

namespace {

constexpr int kMaxHidden = 16384;
constexpr int kMaxVecs = 7;                 // vectors of 8 elements a thread
// Registers of a thread that has V vectors, and the warps of it that an SM holds.  (Six vectors, of 112
// registers, never have most in flight: no row takes them.)
constexpr int kRegs[kMaxVecs + 1] = {0, 64, 64, 64, 80, 96, 0, 128};
constexpr int warps_of(int v) { return 16384 / (32 * kRegs[v]) * 4; }
constexpr int kWarpRows = 8;                // rows of one warp each share a CTA
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100
constexpr float kHuge = 3.0e38f;

struct Params {
    const uint16_t *x;
    const uint16_t *residual;               // nullptr: none
    const uint16_t *weight;
    uint16_t *residual_out;                 // nullptr: not written
    uint16_t *out;                          // nullptr: not written
    uint8_t *codes;                         // nullptr: not written
    float *scales;
    int64_t x_stride, residual_stride, residual_out_stride, out_stride, codes_stride;
    int64_t num_tokens;
    int32_t hidden;
    int32_t vecs;                           // ceil(hidden / 8)
    int32_t threads_per_row;                // a multiple of 32
    float eps;
    float inv_hidden;
};

__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float2 v)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v.y), "f"(v.x));
    return d;
}

__device__ __forceinline__ uint4 pack_bf16x8(const float2 *y)
{
    return make_uint4(pack_bf16x2(y[0]), pack_bf16x2(y[1]), pack_bf16x2(y[2]), pack_bf16x2(y[3]));
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float2 a, float2 b)
{
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Vector i of a row of bf16 values; the last one may be short (n < 8), zeros behind it.
__device__ __forceinline__ uint4 load_vec(const uint16_t *row, int i, int n)
{
    if (n >= 8)
        return *reinterpret_cast<const uint4 *>(row + 8 * i);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < n)
            w[j / 2] |= (uint32_t)row[8 * i + j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_vec(uint16_t *row, int i, int n, uint4 v)
{
    if (n >= 8) {
        *reinterpret_cast<uint4 *>(row + 8 * i) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < n)
            row[8 * i + j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
}

__device__ __forceinline__ void store_codes(uint8_t *row, int i, int n, uint2 v)
{
    if (n >= 8) {
        *reinterpret_cast<uint2 *>(row + 8 * i) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < n)
            row[8 * i + j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
}

// The sum of squares of a row and the largest |h w| as a bit pattern.  A row is one warp's, or
// the whole CTA's.
struct RowSums {
    float ss;
    uint32_t top;
};

__device__ __forceinline__ RowSums row_sums(float ss, uint32_t top, int warps)
{
    __shared__ float s_ss[32];
    __shared__ uint32_t s_top[32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    top = __reduce_max_sync(0xffffffffu, top);
    if (warps == 1)
        return {ss, top};
    if ((threadIdx.x & 31) == 0) {
        s_ss[threadIdx.x >> 5] = ss;
        s_top[threadIdx.x >> 5] = top;
    }
    __syncthreads();
    ss = 0.0f;
    top = 0;
    for (int w = 0; w < warps; ++w) {
        ss += s_ss[w];
        top = max(top, s_top[w]);
    }
    return {ss, top};
}

// A thread's part of both sums: of h^2, and the largest |h w| as a bit pattern.
template <int V>
__device__ __forceinline__ void partial_sums(const float2 (&h)[V][4], const uint4 (&rw)[V], float *ss, uint32_t *top)
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t ws[4] = {rw[v].x, rw[v].y, rw[v].z, rw[v].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 a = h[v][j], w = unpack2(ws[j]);
            *ss = fmaf(a.x, a.x, fmaf(a.y, a.y, *ss));
            *top = max(*top, max(__float_as_uint(a.x * w.x) & 0x7fffffffu, __float_as_uint(a.y * w.y) & 0x7fffffffu));
        }
    }
}

template <int V>
__global__ void __maxnreg__(kRegs[V])
msa_norm_kernel(const __grid_constant__ Params p)
{
    const int tpr = p.threads_per_row, warps = tpr >> 5;
    const int lane = threadIdx.x % tpr;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = t < p.num_tokens;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);

    uint4 rx[V], rr[V], rw[V];
    int n[V];                               // elements of this thread's vectors
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = lane + v * tpr;
        n[v] = live && i < p.vecs ? min(8, p.hidden - 8 * i) : 0;
        rx[v] = rr[v] = rw[v] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (n[v] > 0)
            rx[v] = load_vec(p.x + t * p.x_stride, lane + v * tpr, n[v]);
    if (p.residual)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (n[v] > 0)
                rr[v] = load_vec(p.residual + t * p.residual_stride, lane + v * tpr, n[v]);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (n[v] > 0)
            rw[v] = load_vec(p.weight, lane + v * tpr, n[v]);

    float2 h[V][4];
    float ss = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t xs[4] = {rx[v].x, rx[v].y, rx[v].z, rx[v].w};
        const uint32_t rs[4] = {rr[v].x, rr[v].y, rr[v].z, rr[v].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 x = unpack2(xs[j]), r = unpack2(rs[j]);
            h[v][j] = p.residual ? make_float2(x.x + r.x, x.y + r.y) : x;
        }
        if (p.residual_out && n[v] > 0)
            store_vec(p.residual_out + t * p.residual_out_stride, lane + v * tpr, n[v], pack_bf16x8(h[v]));
    }
    partial_sums<V>(h, rw, &ss, &top);
    RowSums s = row_sums(ss, top, warps);
    float mean = fmaf(s.ss, p.inv_hidden, p.eps);
    // Squares that leave the range of fp32: once more with h scaled by a power of two.
    if (!(mean >= kTiny && mean <= kHuge)) {
        const float f = mean < kTiny ? 0x1p80f : 0x1p-80f;
        if (warps > 1)
            __syncthreads();                // the first sums are read
        ss = 0.0f;
        top = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[v][j] = make_float2(h[v][j].x * f, h[v][j].y * f);
        partial_sums<V>(h, rw, &ss, &top);
        s = row_sums(ss, top, warps);
        mean = fmaf(s.ss, p.inv_hidden, p.eps * f * f);
    }
    const float r = rsqrtf(mean);
    const float amax = __uint_as_float(s.top) * r;
    const float scale = (amax < kTiny ? kTiny : amax) * (1.0f / 448.0f);   // NaN stays
    // (a division for each code takes 68.4 us for 55.4 at 8,192 x 6,144; one code in 100,000 is another
    // one then, and their rms error against 64 bits the same to four digits)
    const float inv = 1.0f / scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (n[v] <= 0)
            continue;
        const int i = lane + v * tpr;
        const uint32_t ws[4] = {rw[v].x, rw[v].y, rw[v].z, rw[v].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 w = unpack2(ws[j]);
            h[v][j] = make_float2(h[v][j].x * w.x * r, h[v][j].y * w.y * r);   // y
        }
        if (p.out)
            store_vec(p.out + t * p.out_stride, i, n[v], pack_bf16x8(h[v]));
        if (p.codes) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[v][j] = make_float2(h[v][j].x * inv, h[v][j].y * inv);
            store_codes(p.codes + t * p.codes_stride, i, n[v],
                        make_uint2(pack_e4m3x4(h[v][0], h[v][1]), pack_e4m3x4(h[v][2], h[v][3])));
        }
    }
    if (p.codes && live && lane == 0)
        p.scales[t] = scale;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

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

// An array of rows: aligned, its stride at least the row's K elements and a multiple of
// `step`, its extent within int64.
msa_status check_rows(const char *name, const void *ptr, int64_t stride, int64_t T, int32_t K, int step)
{
    if (stride < K)
        return fail(MSA_ERR_INVALID_ARGUMENT, "%s: row stride %lld < hidden_size %d", name, (long long)stride, K);
    if (reinterpret_cast<uintptr_t>(ptr) % 16 || stride % step)
        return fail(MSA_ERR_MISALIGNED, "%s: 16-byte aligned rows, a stride that is a multiple of %d elements", name,
                    step);
    int64_t bytes;
    if (__builtin_mul_overflow(T, stride, &bytes) || __builtin_mul_overflow(bytes, (int64_t)2, &bytes))
        return fail(MSA_ERR_OFFSET_OVERFLOW, "%s: extent overflows int64", name);
    return MSA_OK;
}

msa_status validate(const msa_norm_cfg *cfg, int64_t T, const Params &p, int32_t flags)
{
    msa_internal_set_detail("");
    if (!cfg)
        return fail(MSA_ERR_INVALID_ARGUMENT, "cfg is NULL");
    const int32_t K = cfg->hidden_size;
    if (K < 1)
        return fail(MSA_ERR_INVALID_ARGUMENT, "hidden_size %d", K);
    if (K > kMaxHidden)
        return fail(MSA_ERR_UNSUPPORTED, "hidden_size %d (at most %d)", K, kMaxHidden);
    if (!(cfg->rms_eps >= 0.0f && std::isfinite(cfg->rms_eps)))
        return fail(MSA_ERR_INVALID_ARGUMENT, "rms_eps must be non-negative and finite");
    if (cfg->reserved[0] != 0 || cfg->reserved[1] != 0)
        return fail(MSA_ERR_INVALID_ARGUMENT, "cfg reserved fields must be 0");
    if (flags & ~MSA_LAUNCH_PDL)
        return fail(MSA_ERR_INVALID_ARGUMENT, "unknown launch flag bits 0x%x", flags);
    if (T < 0)
        return fail(MSA_ERR_INVALID_ARGUMENT, "num_tokens %lld", (long long)T);
    if (T > 0x7fffffff)
        return fail(MSA_ERR_UNSUPPORTED, "num_tokens %lld (at most 2^31 - 1)", (long long)T);
    if (T == 0)
        return MSA_OK;
    if (!p.x || !p.weight)
        return fail(MSA_ERR_INVALID_ARGUMENT, "x and weight are required");
    if (p.residual_out && !p.residual)
        return fail(MSA_ERR_INVALID_ARGUMENT, "residual_out without a residual");
    if (!p.out && !p.codes)
        return fail(MSA_ERR_INVALID_ARGUMENT, "no output: out or codes is required");
    if (!p.codes != !p.scales)
        return fail(MSA_ERR_INVALID_ARGUMENT, "codes and scales are given together");
    if (reinterpret_cast<uintptr_t>(p.weight) % 16 || reinterpret_cast<uintptr_t>(p.scales) % 4)
        return fail(MSA_ERR_MISALIGNED, "weight (16 bytes) or scales (4 bytes) misaligned");
    const struct { const char *name; const void *ptr; int64_t stride; int step; } rows[5] = {
        {"x", p.x, p.x_stride, 8}, {"residual", p.residual, p.residual_stride, 8},
        {"residual_out", p.residual_out, p.residual_out_stride, 8}, {"out", p.out, p.out_stride, 8},
        {"codes", p.codes, p.codes_stride, 16}};
    for (const auto &a : rows) {
        const msa_status s = a.ptr ? check_rows(a.name, a.ptr, a.stride, T, K, a.step) : MSA_OK;
        if (s != MSA_OK)
            return s;
    }
    const bool in_place[4] = {p.residual_out && p.residual_out == p.residual && p.residual_out_stride != p.residual_stride,
                              p.residual_out && p.residual_out == p.x && p.residual_out_stride != p.x_stride,
                              p.out && p.out == p.x && p.out_stride != p.x_stride,
                              p.out && p.out == p.residual && p.out_stride != p.residual_stride};
    for (bool bad : in_place)
        if (bad)
            return fail(MSA_ERR_INVALID_ARGUMENT, "an output in the place of an input has another row stride");
    return MSA_OK;
}

}  // namespace

extern "C" msa_status msa_norm_forward(const msa_norm_cfg *cfg, int64_t num_tokens, const void *x, int64_t x_stride,
                                       const void *residual, int64_t residual_stride, const void *weight,
                                       void *residual_out, int64_t residual_out_stride, void *out,
                                       int64_t out_stride, void *codes, int64_t codes_stride, float *scales,
                                       int32_t launch_flags, cudaStream_t stream)
{
    Params p;
    memset(&p, 0, sizeof p);
    p.x = static_cast<const uint16_t *>(x);
    p.residual = static_cast<const uint16_t *>(residual);
    p.weight = static_cast<const uint16_t *>(weight);
    p.residual_out = static_cast<uint16_t *>(residual_out);
    p.out = static_cast<uint16_t *>(out);
    p.codes = static_cast<uint8_t *>(codes);
    p.scales = scales;
    p.x_stride = x_stride;
    p.residual_stride = residual_stride;
    p.residual_out_stride = residual_out_stride;
    p.out_stride = out_stride;
    p.codes_stride = codes_stride;
    const msa_status s = validate(cfg, num_tokens, p, launch_flags);
    if (s != MSA_OK || num_tokens == 0)
        return s;
    p.num_tokens = num_tokens;
    p.hidden = cfg->hidden_size;
    p.vecs = (p.hidden + 7) / 8;
    p.eps = cfg->rms_eps;
    p.inv_hidden = 1.0f / (float)p.hidden;

    // Vectors of a thread.  Rows whose warps fit onto the GPU twice with one vector each: one, since
    // the chain of a row is what takes time (one token of 6,144 2.4 us; 777 of 1,001 2.45 us, 2.95 with
    // four).  Otherwise those with which an SM has most vectors in flight, whole rows of its resident
    // warps: 8,192 x 6,144 takes 55.5 us with three, 58.6 with four, of 80 registers (as many in flight),
    // 60.4 with three of 73 registers (three quarters as many); rows of 1,536 run at 0.99 of the copy
    // rate with three each and at 0.59 with one.
    using Kernel = void (*)(Params);
    struct Choice { int vecs; Kernel kernel; };
    static const Choice choices[] = {{1, msa_norm_kernel<1>}, {2, msa_norm_kernel<2>}, {3, msa_norm_kernel<3>},
                                     {4, msa_norm_kernel<4>}, {5, msa_norm_kernel<5>}, {7, msa_norm_kernel<7>}};
    Choice chosen = choices[0];
    if (p.vecs > 1024 || num_tokens * ((p.vecs + 31) / 32) > 2 * 152 * warps_of(1)) {
        int best = 0;
        for (const Choice &c : choices) {
            const int wpr = (p.vecs + 32 * c.vecs - 1) / (32 * c.vecs), flying = warps_of(c.vecs) / wpr * p.vecs;
            if (flying > best) {
                best = flying;
                chosen = c;
            }
        }
    }
    const int v = chosen.vecs;
    p.threads_per_row = ((p.vecs + v - 1) / v + 31) / 32 * 32;
    const int rows = p.threads_per_row == 32 ? kWarpRows : 1;
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    lc.gridDim = dim3((unsigned)((num_tokens + rows - 1) / rows));
    lc.blockDim = dim3((unsigned)(p.threads_per_row * rows));
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    void *args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(&lc, reinterpret_cast<const void *>(chosen.kernel), args);
    if (e != cudaSuccess)
        return fail(MSA_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
    return MSA_OK;
}
