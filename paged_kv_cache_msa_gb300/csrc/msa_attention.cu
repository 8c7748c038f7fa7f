// Attention over the paged K/V caches: argument checks, dispatch, and the kernel for
// every layout.
//
// What is computed is stated in include/msa_attention.h.

#include "msa_attention_internal.h"

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

namespace {

// ---------------------------------------------------------------------------
// the kernel for every layout: one CTA per (query, up to eight heads of a K/V head)
// ---------------------------------------------------------------------------
//
// 128 threads walk the visible tokens 128 at a time with the running maximum and sum
// of an online softmax.  Scores: a thread holds one token and multiplies its key row
// with the CTA's (at most eight) query rows, kept as fp32 in shared memory.  Output: a
// thread holds one dim (of 64 dims, one dim of every other token) of the eight rows
// and adds the tokens' values times their weights.  Rows are read 8 elements (FP8) or
// 8 elements of 16 bits at a time, the alignment that every accepted layout has.  It
// is bound by its fp32 multiply-adds and serves the layouts that the tensor-core
// kernels do not take: 64 queries of 16 blocks (64 heads on 8 of 128 dims, E4M3) take it
// 473 us (the decode kernel 52), 8,192 prefill queries 30.2 ms (1.00).
constexpr int kRowThreads = 128;
constexpr int kRowHeads = 8;

__device__ __forceinline__ void load8(const uint8_t *base, bool fp8, int64_t elem, float (&x)[8])
{
    if (fp8) {
        const uint2 w = *reinterpret_cast<const uint2 *>(base + elem);
        const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = attn_e4m3x2_to_f2((ww[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(base + 2 * elem);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(ww[i] << 16);
            x[2 * i + 1] = __uint_as_float(ww[i] & 0xFFFF0000u);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) msa_attention_rows_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float s_q[kRowHeads][D];
    __shared__ float s_p[kRowThreads][kRowHeads];
    __shared__ int64_t s_v[kRowThreads];        // element offset of the token's value row, -1: not visible
    __shared__ float s_red[2][4][kRowHeads];
    __shared__ int32_t s_ids[64];
    __shared__ int s_n, s_group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunks = (p.group + kRowHeads - 1) / kRowHeads;
    const int64_t bid = blockIdx.x;
    const int hc = (int)(bid % chunks);
    const int c = (int)((bid / chunks) % p.hkv);
    const int64_t t = bid / ((int64_t)chunks * p.hkv);
    const int h0 = c * p.group + hc * kRowHeads;
    const int nh = min(kRowHeads, p.group - hc * kRowHeads);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const int32_t own = attn_len(p, p.kv_len[t], p.table_offset[t]);
    if (tid == 0) {
        s_group = 0x7fffffff;
        s_n = 0;
        if (p.topk_ids) {   // the ids of this query that name a block, each once
            const int64_t nb = ((int64_t)own + p.block_tokens - 1) / p.block_tokens;
            int n = 0;
            for (int i = 0; i < p.topk; ++i) {
                const int32_t id = p.topk_ids[t * p.topk + i];
                bool keep = id >= 0 && id < nb;
                for (int j = 0; j < n && keep; ++j)
                    keep = s_ids[j] != id;
                if (keep)
                    s_ids[n++] = id;
            }
            s_n = n;
        }
    }
    const float qs = p.scale_log2 * attn_k_scale(p, c);
    for (int i = tid; i < kRowHeads * D; i += kRowThreads) {
        const int h = i / D;
        const float x = h < nh ? __uint_as_float((uint32_t)p.q[(t * p.hq + h0 + h) * D + i % D] << 16) : 0.0f;
        // over E4M3 keys no score of an infinite query is a number, as on the tensor cores
        s_q[h][i % D] = p.k.fp8 && fabsf(x) == INFINITY ? __int_as_float(0x7fc00000) : x;
    }
    __syncthreads();
    for (int i = tid; i <= p.num_groups && p.num_groups > 0; i += kRowThreads)
        if (p.group_start[i] > t)
            atomicMin(&s_group, i);
    __syncthreads();

    constexpr int kSlices = kRowThreads / D;     // threads per dim
    const int dim = tid % D, slice = tid / D;
    float acc[kRowHeads] = {}, m[kRowHeads], l[kRowHeads] = {};
#pragma unroll
    for (int h = 0; h < kRowHeads; ++h)
        m[h] = -INFINITY;

    // the prefix of the query's group, then its own history
    const int g = s_group - 1;
    const bool has_prefix = g >= 0 && g < p.num_groups;
    for (int part = has_prefix ? 0 : 1; part < 2; ++part) {
        const int64_t off = part == 0 ? p.prefix_offset[g] : p.table_offset[t];
        const int64_t len = part == 0 ? attn_len(p, p.prefix_len[g], off) : own;
        const bool sparse = p.topk_ids != nullptr;
        const int64_t total = sparse ? (int64_t)s_n * p.block_tokens : len;
        for (int64_t v0 = 0; v0 < total; v0 += kRowThreads) {
            const int64_t v = v0 + tid;
            int64_t j = v;
            if (sparse && v < total)
                j = (int64_t)s_ids[v / p.block_tokens] * p.block_tokens + v % p.block_tokens;
            const int32_t pg = (v < total && j < len) ? attn_page(p, off, j) : -1;
            float s[kRowHeads];
#pragma unroll
            for (int h = 0; h < kRowHeads; ++h)
                s[h] = 0.0f;
            int64_t voff = -1;
            if (pg >= 0) {
                const int64_t row = attn_page_row(p, j);
                const int64_t koff = (int64_t)pg * p.k.stride_page + (int64_t)c * p.k.stride_head + row * p.k.stride_token;
                voff = (int64_t)pg * p.v.stride_page + (int64_t)c * p.v.stride_head + row * p.v.stride_token;
                for (int d = 0; d < D; d += 8) {
                    float x[8];
                    load8(p.k.data, p.k.fp8, koff + d, x);
#pragma unroll
                    for (int h = 0; h < kRowHeads; ++h)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            s[h] = fmaf(s_q[h][d + e], x[e], s[h]);
                }
            }
            float mx[kRowHeads];
#pragma unroll
            for (int h = 0; h < kRowHeads; ++h) {
                s[h] = pg >= 0 ? s[h] * qs : -INFINITY;
                mx[h] = s[h];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], o));
                if (lane == 0)
                    s_red[0][warp][h] = mx[h];
            }
            s_v[tid] = voff;
            __syncthreads();
#pragma unroll
            for (int h = 0; h < kRowHeads; ++h) {
                const float mn = fmaxf(fmaxf(fmaxf(s_red[0][0][h], s_red[0][1][h]),
                                             fmaxf(s_red[0][2][h], s_red[0][3][h])), m[h]);
                const float alpha = mn == -INFINITY ? 1.0f : exp2f(m[h] - mn);
                const float e = s[h] == -INFINITY ? 0.0f : exp2f(s[h] - mn);
                s_p[tid][h] = e;
                float sum = e;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0)
                    s_red[1][warp][h] = sum;
                m[h] = mn;
                l[h] *= alpha;
                acc[h] *= alpha;
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < kRowHeads; ++h)
                l[h] += s_red[1][0][h] + s_red[1][1][h] + s_red[1][2][h] + s_red[1][3][h];
            const int last = (int)min((int64_t)kRowThreads, total - v0);
            for (int i = slice; i < last; i += kSlices) {
                const int64_t vo = s_v[i];
                if (vo < 0)
                    continue;
                const float x = p.v.fp8 ? attn_e4m3x2_to_f2(p.v.data[vo + dim]).x
                                        : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p.v.data)[vo + dim] << 16);
#pragma unroll
                for (int h = 0; h < kRowHeads; ++h)
                    acc[h] = fmaf(s_p[i][h], x, acc[h]);
            }
            __syncthreads();
        }
    }
    if (kSlices > 1) {   // the dims of the other tokens
#pragma unroll
        for (int h = 0; h < kRowHeads; ++h)
            if (slice > 0)
                s_p[tid][h] = acc[h];
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kRowHeads; ++h)
            if (slice == 0)
                for (int i = 1; i < kSlices; ++i)
                    acc[h] += s_p[i * D + dim][h];
    }
    const float vs = attn_v_scale(p, c);
    if (slice == 0) {
#pragma unroll
        for (int h = 0; h < kRowHeads; ++h)
            if (h < nh) {
                const int64_t row = t * p.hq + h0 + h;
                p.out[row * D + dim] = attn_bf16(l[h] == 0.0f ? 0.0f : acc[h] * (vs / l[h]));
                if (dim == 0 && p.lse)
                    p.lse[row] = attn_lse(m[h], l[h]);
            }
    }
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

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

msa_status check_cfg(const msa_attention_cfg *cfg, int64_t T, bool sparse)
{
    msa_internal_set_detail("");
    if (!cfg)
        return fail(MSA_ERR_INVALID_ARGUMENT, "cfg is NULL");
    if (cfg->num_kv_heads < 1 || cfg->num_q_heads < 1)
        return fail(MSA_ERR_INVALID_ARGUMENT, "%d query heads, %d K/V heads", cfg->num_q_heads, cfg->num_kv_heads);
    if (cfg->num_q_heads % cfg->num_kv_heads)
        return fail(MSA_ERR_INVALID_ARGUMENT, "num_q_heads %d is not a multiple of num_kv_heads %d",
                    cfg->num_q_heads, cfg->num_kv_heads);
    if (cfg->num_kv_heads > 1024 || cfg->num_q_heads / cfg->num_kv_heads > 128)
        return fail(MSA_ERR_UNSUPPORTED, "%d K/V heads (1..1024), %d query heads on each (1..128)",
                    cfg->num_kv_heads, cfg->num_q_heads / cfg->num_kv_heads);
    if (cfg->head_dim != 64 && cfg->head_dim != 128)
        return fail(MSA_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", cfg->head_dim);
    if (cfg->page_size <= 0)
        return fail(MSA_ERR_INVALID_ARGUMENT, "page_size %d", cfg->page_size);
    if (sparse && (cfg->block_tokens < 32 || cfg->block_tokens > 1024 || cfg->block_tokens % 32))
        return fail(MSA_ERR_UNSUPPORTED, "block_tokens %d (multiple of 32, 32..1024)", cfg->block_tokens);
    if (sparse && (cfg->topk < 1 || cfg->topk > 64))
        return fail(MSA_ERR_UNSUPPORTED, "topk %d (1..64)", cfg->topk);
    if (!(cfg->softmax_scale > 0.0f) || !std::isfinite(cfg->softmax_scale))
        return fail(MSA_ERR_INVALID_ARGUMENT, "softmax_scale %g", (double)cfg->softmax_scale);
    if (cfg->scale_mode != MSA_SCALE_PER_TENSOR && cfg->scale_mode != MSA_SCALE_PER_HEAD)
        return fail(MSA_ERR_UNSUPPORTED, "scale_mode %d", cfg->scale_mode);
    if (cfg->reserved[0] || cfg->reserved[1])
        return fail(MSA_ERR_INVALID_ARGUMENT, "reserved fields must be 0");
    if (T < 0)
        return fail(MSA_ERR_INVALID_ARGUMENT, "num_queries %lld", (long long)T);
    // the kernels' grids: one CTA per query and (a piece of) a K/V head at most
    const int64_t per = (int64_t)cfg->num_kv_heads * ((cfg->num_q_heads / cfg->num_kv_heads + kRowHeads - 1) / kRowHeads);
    if (T > (int64_t)0x7fffffff / per)
        return fail(MSA_ERR_UNSUPPORTED, "num_queries %lld x heads exceeds the grid", (long long)T);
    return MSA_OK;
}

// The arguments that both operators have (after check_cfg, num_queries > 0).
msa_status check_common(const msa_attention_cfg *cfg, const void *q, const int32_t *kv_len,
                        const int64_t *table_offset, const int32_t *page_table, int64_t page_table_len,
                        const msa_cache_desc *kc, const msa_cache_desc *vc, const float *scales, const void *out,
                        const float *lse, const void *workspace, int64_t workspace_bytes, int64_t needed)
{
    if (!q || !kv_len || !table_offset || !page_table || !kc || !vc || !out)
        return fail(MSA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (page_table_len <= 0)
        return fail(MSA_ERR_INVALID_ARGUMENT, "page_table_len %lld", (long long)page_table_len);
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(kv_len, 4) || !aligned(table_offset, 8) ||
        !aligned(page_table, 4) || !aligned(lse, 4))
        return fail(MSA_ERR_MISALIGNED, "a buffer is misaligned");
    msa_status s = msa_internal_check_cache("k_cache", kc, cfg->num_kv_heads, cfg->head_dim, cfg->page_size);
    if (s == MSA_OK)
        s = msa_internal_check_cache("v_cache", vc, cfg->num_kv_heads, cfg->head_dim, cfg->page_size);
    if (s != MSA_OK)
        return s;
    if (kc->dtype == MSA_DTYPE_FP8_E4M3 || vc->dtype == MSA_DTYPE_FP8_E4M3) {
        if (!scales)
            return fail(MSA_ERR_INVALID_ARGUMENT, "an FP8 cache needs scales");
        if (!aligned(scales, 4))
            return fail(MSA_ERR_MISALIGNED, "scales is misaligned");
    }
    if (workspace_bytes < needed || (needed > 0 && !workspace))
        return fail(MSA_ERR_INVALID_ARGUMENT, "workspace of %lld bytes, %lld needed",
                    workspace ? (long long)workspace_bytes : 0LL, (long long)needed);
    if (!aligned(workspace, 16))
        return fail(MSA_ERR_MISALIGNED, "workspace is misaligned");
    return MSA_OK;
}

AttnCache cache_of(const msa_cache_desc *c)
{
    AttnCache a;
    a.data = static_cast<const uint8_t *>(c->data);
    a.num_pages = c->num_pages;
    a.stride_page = c->stride_page;
    a.stride_head = c->stride_head;
    a.stride_token = c->stride_token;
    a.fp8 = c->dtype == MSA_DTYPE_FP8_E4M3;
    return a;
}

AttnParams params_of(const msa_attention_cfg *cfg, int64_t T, const void *q, const int32_t *kv_len,
                     const int64_t *table_offset, const int32_t *page_table, int64_t page_table_len,
                     const msa_cache_desc *kc, const msa_cache_desc *vc, const float *scales, void *out, float *lse)
{
    AttnParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(q);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.kv_len = kv_len;
    p.table_offset = table_offset;
    p.page_table = page_table;
    p.page_table_len = page_table_len;
    p.scales = scales;
    p.k = cache_of(kc);
    p.v = cache_of(vc);
    p.num_queries = T;
    p.hq = cfg->num_q_heads;
    p.hkv = cfg->num_kv_heads;
    p.group = cfg->num_q_heads / cfg->num_kv_heads;
    p.page_size = cfg->page_size;
    p.page_shift = p.block_shift = -1;
    for (int sh = 0; sh < 31; ++sh) {
        if ((1 << sh) == cfg->page_size)
            p.page_shift = sh;
        if ((1 << sh) == cfg->block_tokens)
            p.block_shift = sh;
    }
    p.block_tokens = cfg->block_tokens;
    p.topk = cfg->topk;
    p.per_head_scales = cfg->scale_mode == MSA_SCALE_PER_HEAD;
    p.scale_log2 = cfg->softmax_scale * 1.4426950408889634f;
    return p;
}

msa_status launched(cudaError_t e)
{
    return e == cudaSuccess ? MSA_OK : fail(MSA_ERR_CUDA, "attention launch failed: %s", cudaGetErrorString(e));
}

msa_status launch_rows(const AttnParams &p, int head_dim, cudaStream_t stream)
{
    const int64_t grid = p.num_queries * p.hkv * ((p.group + kRowHeads - 1) / kRowHeads);
    void *args[] = {const_cast<AttnParams *>(&p)};
    return launched(attn_launch(head_dim == 128 ? reinterpret_cast<const void *>(&msa_attention_rows_kernel<128>)
                                                : reinterpret_cast<const void *>(&msa_attention_rows_kernel<64>),
                                grid, kRowThreads, 0, stream, args));
}

int group_shift(int group)
{
    int s = 0;
    while ((1 << s) < group)
        ++s;
    return s;
}

// Runs of queries: log2 of a query's rows in a tile (at most 32 queries and kAttnTileList
// ids), tiles x K/V heads, and the CTAs that share a tile's blocks where the machine holds
// `ctas`: a CTA for each, or, where it holds twice as many or more at once, several and a
// join (8 K/V heads: 40 queries 26 us, 64 with a CTA each; 100: 33, 58; 160: 45, 63; 200, the
// border: 57.6, 62.6 with one, 57.5 with two).  More than it holds at once would cost: 333
// queries 78 us, 88 in two pieces, 81 in three.
struct Runs {
    int shift;
    int64_t units;
    int32_t splits;
};

Runs runs_of(int group, int hkv, int topk, int64_t T, int ctas)
{
    Runs r;
    r.shift = group_shift(group);
    while ((128 >> r.shift) > 32 || (128 >> r.shift) * topk > kAttnTileList)
        ++r.shift;
    const int64_t qt = 128 >> r.shift;
    r.units = (T + qt - 1) / qt * hkv;
    const int64_t fit = ctas / r.units;
    r.splits = fit > 1 ? (int32_t)(fit < 16 ? fit : 16) : 1;
    return r;
}

// Rows of a tile that T queries can fill, an even number so that slots stay 16-byte aligned.
int32_t slot_rows_of(int64_t T, int shift)
{
    const int64_t rows = T << shift;
    return rows >= 128 ? 128 : (int32_t)((rows + 1) & ~(int64_t)1);
}

// Queries of a window behind prefixes, whose rows go to the workspace.
int64_t prefix_window(int64_t hq)
{
    const int64_t n = kAttnWindowRows / hq;
    return n < 1 ? 1 : n < kAttnWindow ? n : kAttnWindow;
}

// The workspace: cuts, prefix sums and groups of a window, the decode kernel's slots, the
// tile kernel's slots, and with groups the whole units' rows of both.  Sizes are those of
// the largest grids, so that they do not depend on the device.  Without groups the slots
// are those of a sparse call with runs of queries, where its tiles are split.
struct Layout {
    int64_t pre, groups, pieces, tile_pieces, rows, tile_rows, bytes;
};

constexpr int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

Layout layout_of(const msa_attention_cfg *cfg, int64_t T, int64_t num_groups)
{
    const int group = cfg->num_q_heads / cfg->num_kv_heads;
    const int64_t nh = attn_decode_heads(group, false), D = cfg->head_dim;
    const int64_t window = T < prefix_window(cfg->num_q_heads) ? T : prefix_window(cfg->num_q_heads);
    const int64_t rows = num_groups > 0 ? align256(window * cfg->num_q_heads * (D + 4) * 4) : 0;
    int64_t slots = 0, slot_rows = 0;
    if (num_groups > 0) {
        slots = 2 * (2 * kAttnMaxCtas);
        slot_rows = slot_rows_of(T, group_shift(group));
    } else if (T > 0 && cfg->topk >= 1 && cfg->topk <= 64 && cfg->block_tokens % kAttnTokens == 0) {
        const Runs r = runs_of(group, cfg->num_kv_heads, cfg->topk, T, 2 * kAttnMaxCtas);
        slots = r.splits > 1 ? r.units * r.splits : 0;
        slot_rows = slot_rows_of(T, r.shift);
    }
    Layout l;
    l.pre = align256(kAttnMaxCtas * 16);
    l.groups = l.pre + align256((kAttnWindow + 1) * 8);
    l.pieces = l.groups + align256(sizeof(AttnGroups));
    l.tile_pieces = l.pieces + align256(2 * (int64_t)kAttnMaxCtas * nh * (D + 2) * 4);
    l.rows = l.tile_pieces + align256(slots * slot_rows * (D + 2) * 4);
    l.tile_rows = l.rows + rows;
    l.bytes = T == 0 ? 0 : l.tile_rows + rows;
    return l;
}

int64_t workspace_needed(const msa_attention_cfg *cfg, int64_t T, int64_t num_groups)
{
    return layout_of(cfg, T, num_groups).bytes;
}

// Rows of the widest TMA box that never crosses a page or a selected block: a power of two.
int box_rows(const AttnParams &p)
{
    int br = kAttnTokens;
    while (br > 1 && (p.page_size % br || (p.topk_ids && p.block_tokens % br)))
        br /= 2;
    return br;
}

// A cache as a map of (dims, rows of a page, heads, pages), boxes of `rows` rows and at
// most 128 bytes.  False when TMA cannot take the layout.
bool encode_cache(CUtensorMap *m, const AttnCache &c, int head_dim, int heads, int page_size, int rows)
{
    const int es = c.fp8 ? 1 : 2;
    const int width = head_dim * es < 128 ? head_dim * es : 128;
    int64_t st = c.stride_token * es, sh = c.stride_head * es, sp = c.stride_page * es;
    // the stride of a dimension of one entry is never used
    if (heads == 1)
        sh = 16;
    if (c.num_pages == 1)
        sp = 16;
    const int64_t limit = (int64_t)1 << 40;
    if (st % 16 || sh % 16 || sp % 16 || st <= 0 || sh <= 0 || sp <= 0 || st >= limit || sh >= limit || sp >= limit ||
        c.num_pages < 1 || c.num_pages >= 0x7fffffff)
        return false;
    const int64_t dims[4] = {head_dim, page_size, heads, c.num_pages};
    const int64_t strides[3] = {st, sh, sp};
    const int32_t box[4] = {width / es, rows, 1, 1};
    return msa_internal_encode_tiled(m, c.data, es, 4, dims, strides, box, width);
}

// The current device's SMs, 0 when it has no tcgen05 tensor cores or cannot be asked.
int tensor_sms()
{
    static std::atomic<int> known[64];     // SMs + 1 of each device, once asked
    int dev = 0, major = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    if (dev < 64 && known[dev].load(std::memory_order_relaxed))
        return known[dev].load(std::memory_order_relaxed) - 1;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    sms = major == 10 ? sms : 0;
    if (dev < 64)
        known[dev].store(sms + 1, std::memory_order_relaxed);
    return sms;
}

// What the tensor-core kernels need to know of the caches; box_rows 0 when they do not
// take the layout: caches of one dtype whose strides are multiples of 16 bytes, pages
// (and blocks) a multiple of 8 tokens.  Fewer rows a box would mean more than 16 copies
// a tile.
struct Maps {
    CUtensorMap k, v;
    int box_rows, sms;
    int32_t oob_page;
};

void make_maps(Maps *m, const AttnParams &p, int head_dim)
{
    memset(m, 0, sizeof *m);
    m->sms = tensor_sms();
    const int br = box_rows(p);
    if (m->sms == 0 || br < 8 || p.k.fp8 != p.v.fp8 || !encode_cache(&m->k, p.k, head_dim, p.hkv, p.page_size, br) ||
        !encode_cache(&m->v, p.v, head_dim, p.hkv, p.page_size, br))
        return;
    m->box_rows = br;
    m->oob_page = (int32_t)(p.k.num_pages > p.v.num_pages ? p.k.num_pages : p.v.num_pages);
}

AttnPieces pieces_of(const AttnParams &p, const Maps &maps, const Layout &l, int head_dim, void *workspace)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    AttnPieces w;
    memset(&w, 0, sizeof w);
    w.cut = reinterpret_cast<int4 *>(ws);
    w.pre = reinterpret_cast<int64_t *>(ws + l.pre);
    w.pieces = reinterpret_cast<float *>(ws + l.pieces);
    w.rows = reinterpret_cast<float *>(ws + l.rows);
    w.heads = attn_decode_heads(p.group, p.k.fp8);
    w.head_chunks = p.hkv * ((p.group + w.heads - 1) / w.heads);
    w.ctas = maps.sms < kAttnMaxCtas ? maps.sms : kAttnMaxCtas;
    // Beside its tiles a (query, head chunk) of 8 heads costs about what 256 bytes a token do
    // (list, softmax, output): 256 short lists of 64-byte rows 19.6 us (20.4 with two items,
    // 26.4 without), 64 of 128-byte rows 52 (53.4 with one, 55 without).  Chunks of 16 heads,
    // whose tiles take longer, do better without: 37 lists of 256-byte rows 25.2 us (27.7 with
    // one item).
    w.segment = w.heads == 8 ? 256 / (head_dim * (p.k.fp8 ? 1 : 2)) : 0;
    w.box_rows = maps.box_rows;
    w.oob_page = maps.oob_page;
    return w;
}

int tile_ctas(const Maps &maps) { return 2 * (maps.sms < kAttnMaxCtas ? maps.sms : kAttnMaxCtas); }   // two a SM

// gp_shift: rows of a query, a power of two that holds the heads on a K/V head.
AttnTiles tiles_of(const AttnParams &p, const Maps &maps, const Layout &l, void *workspace, int gp_shift)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    AttnTiles t;
    memset(&t, 0, sizeof t);
    t.groups = reinterpret_cast<AttnGroups *>(ws + l.groups);
    t.pieces = reinterpret_cast<float *>(ws + l.tile_pieces);
    t.rows = reinterpret_cast<float *>(ws + l.tile_rows);
    t.nq = p.num_queries;
    t.gp_shift = gp_shift;
    t.splits = 1;
    t.ctas = tile_ctas(maps);
    t.slot_rows = slot_rows_of(p.num_queries, gp_shift);
    t.box_rows = maps.box_rows;
    t.oob_page = maps.oob_page;
    return t;
}

// Single queries: windows of kAttnWindow queries, each the decode kernel and the join of
// what was cut between its CTAs.
msa_status run_decode(const AttnParams &p, const Maps &maps, const Layout &l, int head_dim, void *workspace,
                      cudaStream_t stream)
{
    AttnPieces w = pieces_of(p, maps, l, head_dim, workspace);
    for (w.q0 = 0; w.q0 < p.num_queries; w.q0 += kAttnWindow) {
        w.nq = p.num_queries - w.q0 < kAttnWindow ? p.num_queries - w.q0 : kAttnWindow;
        msa_status s = launched(attn_decode(p, w, head_dim, maps.k, maps.v, stream));
        if (s == MSA_OK)
            s = launched(attn_join_cut(p, w, head_dim, stream));
        if (s != MSA_OK)
            return s;
    }
    return MSA_OK;
}

msa_status run_query_runs(const AttnParams &p, const Maps &maps, const Layout &l, int head_dim, void *workspace,
                          cudaStream_t stream)
{
    const Runs r = runs_of(p.group, p.hkv, p.topk, p.num_queries, tile_ctas(maps));
    AttnTiles t = tiles_of(p, maps, l, workspace, r.shift);
    t.splits = r.splits;
    t.ctas = (int32_t)(r.units * r.splits);
    msa_status s = launched(attn_tiles(p, t, head_dim, maps.k, maps.v, stream));
    if (s == MSA_OK && t.splits > 1)
        s = launched(attn_join_splits(p, pieces_of(p, maps, l, head_dim, workspace), t, head_dim, stream));
    return s;
}

// Prefixes: windows of queries, each the tile kernel over the prefixes, the decode kernel
// over the queries' own tokens, and the join of both.
msa_status run_prefix(const AttnParams &p, const Maps &maps, const Layout &l, int head_dim, void *workspace,
                      cudaStream_t stream)
{
    AttnPieces w = pieces_of(p, maps, l, head_dim, workspace);
    AttnTiles t = tiles_of(p, maps, l, workspace, group_shift(p.group));
    w.joined = 1;
    const int64_t window = prefix_window(p.hq);
    for (w.q0 = 0; w.q0 < p.num_queries; w.q0 += window) {
        w.nq = p.num_queries - w.q0 < window ? p.num_queries - w.q0 : window;
        t.q0 = w.q0;
        t.nq = w.nq;
        msa_status s = launched(attn_tiles(p, t, head_dim, maps.k, maps.v, stream));
        if (s == MSA_OK)
            s = launched(attn_decode(p, w, head_dim, maps.k, maps.v, stream));
        if (s == MSA_OK)
            s = launched(attn_join_rows(p, w, t, head_dim, stream));
        if (s != MSA_OK)
            return s;
    }
    return MSA_OK;
}

}  // namespace

cudaError_t attn_launch(const void *fn, int64_t grid, int block, int smem, cudaStream_t stream, void **args)
{
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    lc.gridDim = dim3((unsigned)grid);
    lc.blockDim = dim3((unsigned)block);
    lc.dynamicSmemBytes = (size_t)smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelExC(&lc, fn, args);
}

extern "C" msa_status msa_attention_workspace_bytes(const msa_attention_cfg *cfg, int64_t num_queries,
                                                    int64_t num_groups, int64_t *bytes)
{
    msa_status s = check_cfg(cfg, num_queries, false);
    if (s != MSA_OK)
        return s;
    if (!bytes)
        return fail(MSA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    if (num_groups < 0 || num_groups > kAttnMaxGroups)
        return fail(MSA_ERR_UNSUPPORTED, "num_groups %lld (0..%d)", (long long)num_groups, kAttnMaxGroups);
    *bytes = workspace_needed(cfg, num_queries, num_groups);
    return MSA_OK;
}

extern "C" msa_status msa_sparse_attention_forward(const msa_attention_cfg *cfg, int64_t num_queries, const void *q,
                                                   const int32_t *kv_len, const int64_t *table_offset,
                                                   const int32_t *page_table, int64_t page_table_len,
                                                   const int32_t *topk_ids, const msa_cache_desc *k_cache,
                                                   const msa_cache_desc *v_cache, const float *scales, void *out,
                                                   float *lse, void *workspace, int64_t workspace_bytes,
                                                   int32_t launch_flags, cudaStream_t stream)
{
    msa_status s = check_cfg(cfg, num_queries, true);
    if (s != MSA_OK)
        return s;
    if (launch_flags & ~(MSA_LAUNCH_PDL | MSA_LAUNCH_QUERY_RUNS))
        return fail(MSA_ERR_INVALID_ARGUMENT, "launch flags 0x%x (MSA_LAUNCH_PDL, MSA_LAUNCH_QUERY_RUNS)", launch_flags);
    if (num_queries == 0)
        return MSA_OK;
    if (!topk_ids)
        return fail(MSA_ERR_INVALID_ARGUMENT, "topk_ids is NULL");
    if (!aligned(topk_ids, 4))
        return fail(MSA_ERR_MISALIGNED, "topk_ids is misaligned");
    s = check_common(cfg, q, kv_len, table_offset, page_table, page_table_len, k_cache, v_cache, scales, out, lse,
                     workspace, workspace_bytes, workspace_needed(cfg, num_queries, 0));
    if (s != MSA_OK)
        return s;
    AttnParams p = params_of(cfg, num_queries, q, kv_len, table_offset, page_table, page_table_len, k_cache, v_cache,
                             scales, out, lse);
    p.topk_ids = topk_ids;
    Maps maps;
    make_maps(&maps, p, cfg->head_dim);
    if (maps.box_rows == 0)
        return launch_rows(p, cfg->head_dim, stream);
    const Layout l = layout_of(cfg, num_queries, 0);
    // A tile of the tile kernel lies in one block.  The hint is the caller's, who knows
    // the queries: 8,192 prefill queries 1.00 ms (4.9 as single queries), 333 78 us (211);
    // 64 unrelated ones 82 us (52 as single queries).
    if ((launch_flags & MSA_LAUNCH_QUERY_RUNS) && cfg->block_tokens % kAttnTokens == 0)
        return run_query_runs(p, maps, l, cfg->head_dim, workspace, stream);
    return run_decode(p, maps, l, cfg->head_dim, workspace, stream);
}

extern "C" msa_status msa_prefix_attention_forward(const msa_attention_cfg *cfg, int64_t num_queries, const void *q,
                                                   int64_t num_groups, const int32_t *group_start,
                                                   const int32_t *prefix_len, const int64_t *prefix_offset,
                                                   const int32_t *kv_len, const int64_t *table_offset,
                                                   const int32_t *page_table, int64_t page_table_len,
                                                   const msa_cache_desc *k_cache, const msa_cache_desc *v_cache,
                                                   const float *scales, void *out, float *lse, void *workspace,
                                                   int64_t workspace_bytes, int32_t launch_flags, cudaStream_t stream)
{
    msa_status s = check_cfg(cfg, num_queries, false);
    if (s != MSA_OK)
        return s;
    if (launch_flags & ~MSA_LAUNCH_PDL)
        return fail(MSA_ERR_INVALID_ARGUMENT, "launch flags 0x%x (MSA_LAUNCH_PDL)", launch_flags);
    if (num_groups < 0 || num_groups > kAttnMaxGroups)
        return fail(MSA_ERR_UNSUPPORTED, "num_groups %lld (0..%d)", (long long)num_groups, kAttnMaxGroups);
    if (num_queries == 0)
        return MSA_OK;
    if (num_groups > 0 && (!group_start || !prefix_len || !prefix_offset))
        return fail(MSA_ERR_INVALID_ARGUMENT, "a group array is NULL");
    if (!aligned(group_start, 4) || !aligned(prefix_len, 4) || !aligned(prefix_offset, 8))
        return fail(MSA_ERR_MISALIGNED, "a group array is misaligned");
    s = check_common(cfg, q, kv_len, table_offset, page_table, page_table_len, k_cache, v_cache, scales, out, lse,
                     workspace, workspace_bytes, workspace_needed(cfg, num_queries, num_groups));
    if (s != MSA_OK)
        return s;
    AttnParams p = params_of(cfg, num_queries, q, kv_len, table_offset, page_table, page_table_len, k_cache, v_cache,
                             scales, out, lse);
    p.group_start = group_start;
    p.prefix_len = prefix_len;
    p.prefix_offset = prefix_offset;
    p.num_groups = (int32_t)num_groups;
    Maps maps;
    make_maps(&maps, p, cfg->head_dim);
    if (maps.box_rows == 0)
        return launch_rows(p, cfg->head_dim, stream);
    const Layout l = layout_of(cfg, num_queries, num_groups);
    return num_groups > 0 ? run_prefix(p, maps, l, cfg->head_dim, workspace, stream)
                          : run_decode(p, maps, l, cfg->head_dim, workspace, stream);
}
