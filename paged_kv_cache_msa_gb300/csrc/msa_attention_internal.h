// Shared by the translation units of the attention operators (not exported).
#pragma once

#include "msa_attention.h"
#include "msa_internal.h"

#include <cuda_runtime.h>

#include <cstdint>

constexpr int kAttnMaxGroups = 512;
constexpr int kAttnWindow = 384;     // queries a launch of the tensor-core decode kernel takes
constexpr int kAttnWindowRows = 65536;       // rows of a window of queries behind prefixes
constexpr int kAttnMaxCtas = 192;    // its CTAs (one per SM) at most
constexpr int kAttnTokens = 128;     // tokens of a tile of keys and values
// What a tile of queries costs over a prefix beside its tokens (queries, output), in tiles
// of tokens: a CTA's share of the tile kernel counts it.  64 queries behind 8,192 tokens
// 69.0 us (73.1 without, 70.3 with three), six behind 65,536 72.7 (74.1, 73.0).
constexpr int kAttnUnit = 2;
constexpr int kAttnTileList = 1024;  // (query, id) pairs of a sparse tile

// One cache as the kernels see it; strides in elements.
struct AttnCache {
    const uint8_t *data;
    int64_t num_pages;
    int64_t stride_page, stride_head, stride_token;
    int32_t fp8;
};

struct AttnParams {
    const uint16_t *q;               // [T, Hq, D] bf16
    uint16_t *out;                   // [T, Hq, D] bf16
    float *lse;                      // [T, Hq] or nullptr
    const int32_t *kv_len;
    const int64_t *table_offset;
    const int32_t *page_table;
    int64_t page_table_len;
    const int32_t *topk_ids;         // [T, topk]; nullptr: dense (prefix attention)
    const int32_t *group_start;      // [num_groups + 1]
    const int32_t *prefix_len;
    const int64_t *prefix_offset;
    const float *scales;
    AttnCache k, v;
    int64_t num_queries;
    int32_t num_groups;
    int32_t hq, hkv, group;          // heads; group = hq / hkv
    int32_t page_size;
    int32_t page_shift;              // log2(page_size) when a power of two, else -1
    int32_t block_tokens, topk;
    int32_t block_shift;             // as page_shift
    int32_t per_head_scales;
    float scale_log2;                // softmax_scale * log2(e): scores are kept as powers of two
};

// A piece of a row's attention: its output relative to the maximum, the maximum (of the
// scores times log2 e) and the sum.  Pieces of whole units are rows of D + 4 floats
// [output | maximum | sum | unused], indexed by (query of the window, query head).
//
// What the decode kernel needs beside AttnParams: a window of queries and its part of the
// workspace.  CTA i holds the items [share * i, share * (i + 1)) of the list over (query,
// head chunk, tile), in which `segment` items without a tile come before the tiles of each
// (query, head chunk); share = ceil(items / ctas).  The piece of a (query, head chunk) that
// began in another CTA is in slot i, of one that goes on in the next in slot ctas + i: a
// slot is [heads][D] of output, then the maxima, then the sums.
struct AttnPieces {
    int4 *cut;                       // [ctas]: query, head chunk and last CTA of the one that
                                     // began in a CTA and goes on in the next; query -1: none
    int64_t *pre;                    // [nq + 1]: items before each query of the window (joined)
    float *pieces;                   // slots
    float *rows;                     // whole units (joined)
    int64_t q0, nq;                  // the window
    int32_t heads;                   // query heads of a head chunk: 8 or 16 (attn_decode_heads)
    int32_t head_chunks;             // of all K/V heads
    int32_t ctas;
    int32_t segment;                 // items that a (query, head chunk) has before its tiles
    int32_t box_rows;                // rows of a TMA box
    int32_t oob_page;                // a page past both caches
    int32_t joined;                  // every piece goes to the workspace
};

// The groups of a window, made by the tile kernel: queries start[g] .. start[g + 1] - 1 of
// the window have a prefix of len[g] tokens; item[g] items come before theirs.
struct AttnGroups {
    int64_t item[kAttnMaxGroups + 1];
    int64_t share;                   // items of a CTA
    int32_t start[kAttnMaxGroups + 1];
    int32_t len[kAttnMaxGroups];
};

// What the tile kernel needs beside AttnParams.  Sparse: CTA = (tile, K/V head, split), a
// split tile's piece in slot CTA.  Prefix: items over (group, tile, K/V head, 128 tokens),
// slots as in AttnPieces.  A slot is [slot_rows][D], then [slot_rows][maximum, sum].
struct AttnTiles {
    AttnGroups *groups;              // prefix
    float *pieces;                   // slots
    float *rows;                     // prefix: whole units
    int64_t q0, nq;                  // the window (sparse: every query)
    int32_t gp_shift;                // log2 of the rows of a query
    int32_t slot_rows;               // rows that a tile can have, an even number
    int32_t splits;                  // sparse: CTAs that share a tile's blocks
    int32_t ctas;
    int32_t box_rows, oob_page;
};

// One launch, with programmatic dependent launch: the first kernel of a call waits for the
// kernels ahead of it before it touches memory, and what follows starts after that, so
// each may always start early.
cudaError_t attn_launch(const void *fn, int64_t grid, int block, int smem, cudaStream_t stream, void **args);

int attn_decode_heads(int group, bool fp8);
cudaError_t attn_decode(const AttnParams &p, const AttnPieces &w, int head_dim, const CUtensorMap &kmap,
                        const CUtensorMap &vmap, cudaStream_t stream);
cudaError_t attn_tiles(const AttnParams &p, const AttnTiles &w, int head_dim, const CUtensorMap &kmap,
                       const CUtensorMap &vmap, cudaStream_t stream);
// Joins the pieces of: (query, head chunk)s cut between CTAs; a window's own tokens and
// prefixes; split sparse tiles.
cudaError_t attn_join_rows(const AttnParams &p, const AttnPieces &w, const AttnTiles &tiles, int head_dim,
                           cudaStream_t stream);
cudaError_t attn_join_splits(const AttnParams &p, const AttnPieces &w, const AttnTiles &tiles, int head_dim,
                             cudaStream_t stream);
cudaError_t attn_join_cut(const AttnParams &p, const AttnPieces &w, int head_dim, cudaStream_t stream);

#ifdef __CUDACC__

// Dequantisation scales of K/V head c (1 for bf16 caches).
__device__ __forceinline__ float attn_k_scale(const AttnParams &p, int c)
{
    return p.k.fp8 ? __ldg(p.scales + (p.per_head_scales ? c : 0)) : 1.0f;
}

__device__ __forceinline__ float attn_v_scale(const AttnParams &p, int c)
{
    return p.v.fp8 ? __ldg(p.scales + (p.per_head_scales ? p.hkv + c : 1)) : 1.0f;
}

// The tokens of a history of `len` whose table row starts at `off`, without those past the
// table's end, which no query sees: no length makes a kernel walk further.
__device__ __forceinline__ int32_t attn_len(const AttnParams &p, int32_t len, int64_t off)
{
    constexpr int64_t kFar = (int64_t)1 << 31;       // past any length
    if (len <= 0 || off >= p.page_table_len || off <= -kFar)
        return 0;
    const int64_t pages = p.page_table_len - off;
    return pages >= kFar ? len : (int32_t)min((int64_t)len, pages * p.page_size);
}

// The page of token j of the history whose table row starts at `off`, or -1.
__device__ __forceinline__ int32_t attn_page(const AttnParams &p, int64_t off, int64_t j)
{
    const uint32_t tok = (uint32_t)j;      // below 2^31
    const int64_t i = off + (p.page_shift >= 0 ? tok >> p.page_shift : tok / (uint32_t)p.page_size);
    if (i < 0 || i >= p.page_table_len)
        return -1;
    const int32_t pg = __ldg(p.page_table + i);
    return (pg >= 0 && (int64_t)pg < p.k.num_pages && (int64_t)pg < p.v.num_pages) ? pg : -1;
}

__device__ __forceinline__ int32_t attn_page_row(const AttnParams &p, int64_t j)
{
    const uint32_t tok = (uint32_t)j;
    return (int32_t)(p.page_shift >= 0 ? tok & (uint32_t)(p.page_size - 1) : tok % (uint32_t)p.page_size);
}

// two E4M3 codes -> (low code, high code)
__device__ __forceinline__ float2 attn_e4m3x2_to_f2(uint32_t codes)
{
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((unsigned short)codes));
    float lo, hi;
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h; }"
        : "=f"(lo), "=f"(hi)
        : "r"(h2));
    return make_float2(lo, hi);
}

// One element of a cache, not scaled.
__device__ __forceinline__ float attn_value(const AttnCache &c, int64_t elem)
{
    return c.fp8 ? attn_e4m3x2_to_f2(c.data[elem]).x
                 : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(c.data)[elem] << 16);
}

__device__ __forceinline__ uint16_t attn_bf16(float x)
{
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
    return r;
}

// ln of the sum, from the maximum (of the scores times log2 e) and the sum relative to it
__device__ __forceinline__ float attn_lse(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

#endif
