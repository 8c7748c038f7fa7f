// Shared by the adapter operator's translation units (not exported).
#pragma once

#include "msa_adapter.h"
#include "msa_internal.h"

#include <cuda_runtime.h>

#include <cstdint>

// What the sort says of a call's tiles of tokens.
struct AdapterHead {
    int32_t with_adapter;    // tiles of tokens of one adapter
    int32_t tiles;           // and, behind them, those of tokens without one
    int32_t splits;          // pieces of K of the down-projection
};

struct AdapterParams {
    const uint8_t *hidden;
    const float *hidden_scales;
    const uint16_t *down, *up;
    const int32_t *ids;
    const float *adapter_scales;
    const uint16_t *rows;
    uint16_t *out;
    AdapterHead *head;
    int32_t *adapters;               // of each tile, -1: none
    int32_t *tokens;                 // [tiles, tile_tokens], -1: none; nullptr: at most 128 tokens, not sorted
    float *u;                        // [splits, T, S * r]: sums over pieces of K
    int64_t hidden_stride, down_stride, rows_stride, out_stride;   // elements
    int64_t num_tokens;
    int32_t hidden_size, width, rank, num_adapters, num_slices, fp8;
    int32_t tile_tokens;             // 16 or 128
    int32_t max_splits;              // pieces of K at most
    int32_t n_blocks, n_tiles;       // blocks of down rows, tiles of 8 rows in a block
    int32_t chunk;                   // columns of a CTA's share of the up-projection
    int32_t slice_end[MSA_ADAPTER_MAX_SLICES];
};

// The down-projection of tiles of 128 tokens (msa_adapter_tile.cu) into p.u: what it is launched
// with, made ahead of the call's first launch, and its launch for at most `tiles`.
struct AdapterTileShape {
    int32_t n;           // rows of down an MMA pair takes: a multiple of 16 (32 where two boxes)
    int32_t boxes;       // 1 or 2 of at most 256 rows
    int32_t stages;
    int32_t tmem;        // columns allocated
    uint32_t stage_bytes;
};

struct AdapterTilePlan {
    AdapterTileShape shape;
    CUtensorMap down;
};

cudaError_t adapter_tile_allow();        // its shared memory, on the current device
bool adapter_tile_plan(const AdapterParams &p, AdapterTilePlan *plan);
cudaError_t adapter_tile_launch(const AdapterParams &p, const AdapterTilePlan &plan, int64_t tiles, cudaStream_t stream);

#ifdef __CUDACC__
namespace {

// (x0, x1) -> a bf16 pair, x0 in the low half
__device__ __forceinline__ uint32_t adapter_bf16x2(float x0, float x1)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x1), "f"(x0));
    return d;
}

// (x0, x1) as three bf16 pairs whose sum is (x0, x1), all 24 bits of them (down to bf16's smallest,
// 2^-133): 8 bits cut off at a time, what is left of an infinity being nothing.
__device__ __forceinline__ void adapter_split(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const auto top = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };
    const auto pair = [](float x, float y) { return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632); };
    hi = pair(x0, x1);
    x0 = isinf(x0) ? 0.0f : x0 - top(x0);
    x1 = isinf(x1) ? 0.0f : x1 - top(x1);
    mid = pair(x0, x1);
    lo = pair(x0 - top(x0), x1 - top(x1));
}

// Two E4M3 codes (the low half of c) -> a bf16 pair: exact, since bf16 holds every E4M3 value.
__device__ __forceinline__ uint32_t adapter_e4m3x2(uint32_t c)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)c));
    float lo, hi;
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return adapter_bf16x2(lo, hi);
}

}  // namespace
#endif
