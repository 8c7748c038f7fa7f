// Low-rank adapters of many requests beside a shared projection (include/msa_adapter.h).
//
// Up to three kernels:
//   sort   the tokens by adapter, in tiles of 16 or 128 of one adapter each (up to 128 tokens are
//          put into tiles by every CTA of the next kernels: 64 tokens over 48 adapters took 18.1 us,
//          1.1 more with the sort, 64 over 3 adapters 8.5 and 1.7 more, 128 over 3 10.1 and 0.5).  Reading
//          an adapter costs more than anything else in a decode batch, and in no order of the tokens
//          is it read more often than once a tile: 512 tokens over 16 adapters, mixed, took 100 us
//          in tiles of consecutive tokens that go through their distinct adapters.
//   down   every token's hidden state through its adapter's down-projection, into a workspace
//          (partial sums over pieces of K)
//   up     the up-projection of their sum, added to the rows
// A tile's tokens share the MMA's B operand, its adapter; each has a row of its own, so nothing
// passes from one request to another.  Reading the adapters bounds a decode batch (65 MB for 64
// tokens over 48 adapters of rank 16), reading and writing the rows a prefill: both HBM.  One
// kernel in the place of two, clusters of 8 or 16 CTAs that share a tile's K and join its sums
// through distributed shared memory, took 9.5 us for one token and 31.7 for those 64 (5.6 and
// 18.7): fewer warps read a tile, in rounds of loads that wait 2 us each.

#include "msa_adapter_internal.h"

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

namespace {

constexpr int kTile = 16;            // tokens of a tile: the MMA's M
constexpr int kDownWarps = 8;        // warps of a CTA of the down-projection, each a piece of its K
constexpr int kUnitK = 64;           // K elements a warp takes at a time: 128 bytes of bf16
constexpr int kUpWarps = 16 * 152;   // warps that fill the GPU in the up-projection
constexpr int kFill = 2 * 152;       // CTAs that fill the GPU at two an SM
constexpr int kListed = 128;         // tokens that a CTA puts into tiles by itself
constexpr int kSortKept = 8;         // tokens of a thread of the sort that it loads once
constexpr int kMaxAdapters = 16384;  // the sort counts them in shared memory

// CTAs that a down-projection's pieces of K are to fill.  Wide tiles have fewer and longer pieces: a CTA
// an SM, although two fit (8,192 tokens of rank 32 105.7 us for 109.6, of rank 16 96.3 for 101.5; 5,000
// bf16 ones of rank 48 108 for 129; 4,000 of rank 8 53.0 for 52.3): each has a start, an
// epilogue and its partial sums to write and to read.
__host__ __device__ constexpr int fill_of(bool narrow) { return narrow ? kFill : kFill / 2; }

__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The next kernel may start once this one has waited for those ahead: they are complete then, and
// what they wrote has been performed, before any CTA of the next kernel begins.  So the up-projection
// reads what kernels ahead of this call, and the sort, wrote before its own wait; what the
// down-projection writes, after it.  PTX promises a grid only what is visible after its own wait, so
// nothing but this order of events stands behind those reads: they go to L2 (`early`, cp.async.cg),
// where completed writes are, and past the L1, which might hold older lines.  With the wait first, one
// token takes 7.0 us for 5.6, 64 tokens over 48 adapters 20.2 for 18.7, 8,192 tokens 1 % more.
__device__ __forceinline__ void wait_for_kernels_ahead()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
}

template <class T>
__device__ __forceinline__ T early(const T *p)
{
    return __ldcg(p);
}

// ---------------------------------------------------------------------------
// the tokens by adapter
// ---------------------------------------------------------------------------

// One CTA: counts, the adapters' first tiles, then each token's place.  Tokens of one warp with the
// same adapter (a prefill's chunk) take their places with one atomic.  Which of an adapter's tokens
// share a tile depends on the order of the warps; no token's result depends on that.
__global__ void __launch_bounds__(1024) msa_adapter_sort_kernel(const __grid_constant__ AdapterParams p)
{
    extern __shared__ int s_place[];                 // a count, then the next place, of each adapter; the last: none
    __shared__ int s_sum[32];
    wait_for_kernels_ahead();
    const int tid = threadIdx.x, lane = tid & 31, nt = blockDim.x, n = p.num_adapters + 1;
    const int64_t T = p.num_tokens;
    // this thread's first tokens' adapters, loaded at once and kept for the second pass
    int mine[kSortKept];
#pragma unroll
    for (int i = 0; i < kSortKept; ++i)
        mine[i] = (int64_t)i * nt + tid < T ? __ldg(p.ids + (int64_t)i * nt + tid) : -1;
    for (int a = tid; a < n; a += nt)
        s_place[a] = 0;
    __syncthreads();
    // f(token, adapter, n - 1 without one; -1 behind the last token), a warp's tokens at once
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kSortKept; ++i) {
            const int64_t t = (int64_t)i * nt + tid;
            if (t - lane >= T)
                break;
            f(t, t >= T ? -1 : mine[i] < 0 || mine[i] >= p.num_adapters ? n - 1 : mine[i]);
        }
        for (int64_t t = (int64_t)kSortKept * nt + tid; t - lane < T; t += nt) {
            const int a = t < T ? __ldg(p.ids + t) : -1;
            f(t, t >= T ? -1 : a < 0 || a >= p.num_adapters ? n - 1 : a);
        }
    };
    each([&](int64_t, int a) {
        const uint32_t same = __match_any_sync(0xffffffffu, a);
        if (a >= 0 && lane == __ffs(same) - 1)
            atomicAdd(&s_place[a], __popc(same));
    });
    __syncthreads();
    // tiles before each adapter's: a run of adapters a thread
    const int ts = p.tile_tokens, per = (n + nt - 1) / nt, a0 = min(n, tid * per), a1 = min(n, a0 + per);
    int sum = 0;
    for (int a = a0; a < a1; ++a)
        sum += (s_place[a] + ts - 1) / ts;
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o)
            before += x;
    }
    if (lane == 31)
        s_sum[tid >> 5] = before;
    __syncthreads();
    if (tid < 32) {
        int x = tid < nt / 32 ? s_sum[tid] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (tid >= o)
                x += y;
        }
        s_sum[tid] = x;
    }
    __syncthreads();
    int tile = before - sum + (tid >= 32 ? s_sum[(tid >> 5) - 1] : 0);
    for (int a = a0; a < a1; ++a) {
        const int count = s_place[a], tiles = (count + ts - 1) / ts;
        if (a == n - 1) {
            p.head->with_adapter = tile;
            p.head->tiles = tile + tiles;
            // so many pieces of K that the down-projection fills the GPU once
            const int units = max(1, tile * p.n_blocks);
            p.head->splits = max(1, min(p.max_splits, fill_of(ts == kTile) / units));
        }
        s_place[a] = tile * ts;
        for (int i = count; i < tiles * ts; ++i)
            p.tokens[tile * ts + i] = -1;
        tile += tiles;
    }
    __syncthreads();
    each([&](int64_t t, int a) {
        const uint32_t same = __match_any_sync(0xffffffffu, a);
        const int leader = __ffs(same) - 1;
        int at = 0;
        if (a >= 0 && lane == leader)
            at = atomicAdd(&s_place[a], __popc(same));
        at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1u));
        if (a >= 0) {
            p.tokens[at] = (int)t;
            if (at % ts == 0)
                p.adapters[at / ts] = a == n - 1 ? -1 : a;
        }
    });
}

// The tiles of up to kListed tokens, which every CTA makes for itself: a thread has a token, whose
// place is the number of tokens before it with the same adapter.
struct TileList {
    int id[kListed];                 // -1: none, -2: behind the last token
    int adapter[kListed];            // of a tile
    int heads[2][kListed / 32];      // of each warp, with an adapter and without
    uint8_t tile[kListed][kListed / kTile];   // of an adapter's first token: its tiles
    uint8_t token[kListed][kTile];   // 255: none
};

// The tiles of 16 tokens of one adapter: from the sort (p.tokens), from a list in shared memory, or
// (at most 16 tokens) found by each warp.  Those without an adapter come last.
struct Tiles {
    int with_adapter, all, splits;
    int id;              // at most 16 tokens: this lane's token's adapter, and
    uint32_t same;       // the tokens with the same one
    uint32_t leaders;    // the first token of each distinct adapter

    // by all threads of a CTA, kListed or more
    __device__ __forceinline__ void load(const AdapterParams &p, TileList &s)
    {
        if (p.tokens) {
            with_adapter = early(&p.head->with_adapter);
            all = early(&p.head->tiles);
            splits = early(&p.head->splits);
            return;
        }
        const int lane = threadIdx.x & 31;
        if (p.num_tokens <= kTile) {
            const int t = lane & 15;
            id = t < p.num_tokens ? early(p.ids + t) : -1;
            if (id < 0 || id >= p.num_adapters)
                id = -1;
            same = __match_any_sync(0xffffffffu, id) & 0xffffu;
            leaders = __ballot_sync(0xffffffffu, id >= 0 && lane == __ffs(same) - 1);
            with_adapter = __popc(leaders);
            all = with_adapter + (__any_sync(0xffffffffu, id < 0 && t < p.num_tokens) ? 1 : 0);
        } else {
            make(p, s);
        }
        splits = max(1, min(p.max_splits, kFill / max(1, with_adapter * p.n_blocks)));
    }
    __device__ __forceinline__ void make(const AdapterParams &p, TileList &s)
    {
        const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
        const bool there = t < p.num_tokens;         // at most kListed
        int a = -2;
        if (there) {
            a = early(p.ids + t);
            a = a < 0 || a >= p.num_adapters ? -1 : a;
        }
        if (t < kListed) {
            s.id[t] = a;
            reinterpret_cast<uint4 *>(s.token)[t] = make_uint4(~0u, ~0u, ~0u, ~0u);
        }
        __syncthreads();
        // the tokens before this one with the same adapter, and the first of all
        const uint32_t below = (1u << lane) - 1u, mine = __match_any_sync(0xffffffffu, a);
        int before = __popc(mine & below), root = 32 * warp + __ffs(mine) - 1;
#pragma unroll
        for (int v = kListed / 32 - 2; v >= 0; --v)
            if (v < warp && 32 * warp < kListed) {
                uint32_t same = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int4 x = reinterpret_cast<const int4 *>(s.id + 32 * v)[j];
                    same |= (x.x == a ? 1u << 4 * j : 0u) | (x.y == a ? 2u << 4 * j : 0u) |
                            (x.z == a ? 4u << 4 * j : 0u) | (x.w == a ? 8u << 4 * j : 0u);
                }
                before += __popc(same);
                if (same)
                    root = 32 * v + __ffs(same) - 1;
            }
        const bool first = there && before % kTile == 0;
        const uint32_t some = __ballot_sync(0xffffffffu, first && a >= 0), none = __ballot_sync(0xffffffffu, first && a < 0);
        if (lane == 0 && t < kListed) {
            s.heads[0][warp] = __popc(some);
            s.heads[1][warp] = __popc(none);
        }
        __syncthreads();
        int at[2] = {0, 0}, total[2] = {0, 0};
#pragma unroll
        for (int v = 0; v < kListed / 32; ++v)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                at[i] += v < warp ? s.heads[i][v] : 0;
                total[i] += s.heads[i][v];
            }
        with_adapter = total[0];
        all = total[0] + total[1];
        if (first) {
            const int tile = a >= 0 ? at[0] + __popc(some & below) : total[0] + at[1] + __popc(none & below);
            s.tile[root][before / kTile] = (uint8_t)tile;
            s.adapter[tile] = a;
        }
        __syncthreads();
        if (there)
            s.token[s.tile[root][before / kTile]][before % kTile] = (uint8_t)t;
        __syncthreads();
    }
    // The adapter of a tile, and this lane's token (of slot lane % 16), -1 without one.
    __device__ __forceinline__ void get(const AdapterParams &p, const TileList &s, int tile, int &adapter, int &token) const
    {
        const int slot = threadIdx.x & 15;
        if (p.tokens) {
            adapter = early(p.adapters + tile);
            token = early(p.tokens + tile * kTile + slot);
            return;
        }
        if (p.num_tokens > kTile) {
            adapter = s.adapter[tile];
            token = s.token[tile][slot] == 255 ? -1 : s.token[tile][slot];
            return;
        }
        uint32_t left = leaders;
        for (int j = 0; j < tile; ++j)
            left &= left - 1;
        if (left) {
            const int leader = __ffs(left) - 1;
            adapter = __shfl_sync(0xffffffffu, id, leader);
            token = __shfl_sync(0xffffffffu, same, leader) >> slot & 1u ? slot : -1;
        } else {
            adapter = -1;
            token = id < 0 && slot < p.num_tokens ? slot : -1;
        }
    }
};

// 8 elements of a row from k on as bf16 pairs, zeros from K on; k is a multiple of 8.  WHOLE: all
// of them are there.
template <bool FP8, bool WHOLE>
__device__ __forceinline__ uint4 load_hidden(const AdapterParams &p, int64_t row, int k)
{
    const int n = WHOLE ? 8 : p.hidden_size - k;
    if (n <= 0)
        return make_uint4(0, 0, 0, 0);
    if (FP8) {
        const uint8_t *src = p.hidden + row * p.hidden_stride + k;
        uint2 c = make_uint2(0, 0);
        if (n >= 8)
            c = __ldg(reinterpret_cast<const uint2 *>(src));
        else
            for (int j = 0; j < n; ++j)
                (j < 4 ? c.x : c.y) |= (uint32_t)src[j] << (8 * (j & 3));
        return make_uint4(adapter_e4m3x2(c.x & 0xffffu), adapter_e4m3x2(c.x >> 16),
                          adapter_e4m3x2(c.y & 0xffffu), adapter_e4m3x2(c.y >> 16));
    }
    const uint16_t *src = reinterpret_cast<const uint16_t *>(p.hidden) + row * p.hidden_stride + k;
    if (n >= 8)
        return __ldg(reinterpret_cast<const uint4 *>(src));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < n)
            w[j / 2] |= (uint32_t)src[j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 load_down(const AdapterParams &p, const uint16_t *row, int k)
{
    const int n = p.hidden_size - k;
    if (n >= 8)
        return __ldg(reinterpret_cast<const uint4 *>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < n)
            w[j / 2] |= (uint32_t)row[k + j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// the down-projection of tiles of 16 tokens
// ---------------------------------------------------------------------------
//
// A CTA takes a tile, a block of up to 8 * NT (48) of its adapter's rows and a piece of K, which its
// warps share; their sums meet in shared memory.  A lane holds 8 neighbouring elements of K of a
// token's row and of an adapter's row: the MMA's order of K is free as long as both operands
// agree, so 16-byte loads are its fragments as they come.
template <bool FP8, int NT>
__global__ void __launch_bounds__(32 * kDownWarps, 2) msa_adapter_down_kernel(const __grid_constant__ AdapterParams p)
{
    __shared__ float s_sum[kDownWarps][kTile][8 * NT];
    __shared__ __align__(16) TileList s_tiles;
    wait_for_kernels_ahead();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int n = p.num_slices * p.rank;
    Tiles tiles;
    tiles.load(p, s_tiles);
    const int work = tiles.with_adapter * p.n_blocks * tiles.splits;
    for (int item = blockIdx.x; item < work; item += gridDim.x) {
        const int block = item % p.n_blocks, split = item / p.n_blocks % tiles.splits;
        int a, token;
        tiles.get(p, s_tiles, item / p.n_blocks / tiles.splits, a, token);
        // (a slot without a token takes slot 0's along, and so do the rows of a short block's last tiles:
        // loads without branches between them, of lines that are there already)
        const int some = __shfl_sync(0xffffffffu, token, __ffs(__ballot_sync(0xffffffffu, token >= 0)) - 1);
        const int filled = token >= 0 ? token : some;
        const int tok[2] = {__shfl_sync(0xffffffffu, filled, g), __shfl_sync(0xffffffffu, filled, g + 8)};
        const int n0 = block * p.n_tiles * 8, nt = min(p.n_tiles, (n - n0) / 8);     // the rank is a multiple of 8
        const uint16_t *down = p.down + ((int64_t)a * n + n0 + g) * p.down_stride;
        int64_t at[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            at[i] = i < nt ? i * 8 * p.down_stride : 0;
        const int units = (p.hidden_size + kUnitK - 1) / kUnitK;
        const int piece = split * kDownWarps + warp, pieces = tiles.splits * kDownWarps;
        const int first = (int)((int64_t)units * piece / pieces), last = (int)((int64_t)units * (piece + 1) / pieces);

        float acc[NT][4] = {};
        uint4 x[2][2], w[NT][2];
        auto multiply = [&]() {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t lo[4] = {x[0][h].x, x[1][h].x, x[0][h].y, x[1][h].y};
                const uint32_t hi[4] = {x[0][h].z, x[1][h].z, x[0][h].w, x[1][h].w};
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    mma(acc[i], lo, w[i][h].x, w[i][h].y);
                    mma(acc[i], hi, w[i][h].z, w[i][h].w);
                }
            }
        };
        const int whole = min(last, p.hidden_size / kUnitK);       // units without a tail
        const uint16_t *wp = down + first * kUnitK + 8 * q;
        for (int u = first; u < whole; ++u, wp += kUnitK) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[i][h] = __ldg(reinterpret_cast<const uint4 *>(wp + at[i] + 32 * h));
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    x[r][h] = load_hidden<FP8, true>(p, tok[r], u * kUnitK + 32 * h + 8 * q);
            multiply();
        }
        for (int u = max(first, whole); u < last; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = u * kUnitK + 32 * h + 8 * q;
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    w[i][h] = load_down(p, down + at[i], k);
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    x[r][h] = load_hidden<FP8, false>(p, tok[r], k);
            }
            multiply();
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            *reinterpret_cast<float2 *>(&s_sum[warp][g][8 * i + 2 * q]) = make_float2(acc[i][0], acc[i][1]);
            *reinterpret_cast<float2 *>(&s_sum[warp][g + 8][8 * i + 2 * q]) = make_float2(acc[i][2], acc[i][3]);
        }
        __syncthreads();
        const float c = p.adapter_scales ? p.adapter_scales[a] : 1.0f;
        // a warp writes the rows of tokens 2 warp and 2 warp + 1
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 2 * warp + h, t = __shfl_sync(0xffffffffu, token, r);
            if (t < 0)
                continue;
            const float scale = c * (p.hidden_scales ? p.hidden_scales[t] : 1.0f);
            for (int i = lane; i < 8 * nt; i += 32) {
                float sum = 0.0f;
#pragma unroll
                for (int v = 0; v < kDownWarps; ++v)
                    sum += s_sum[v][r][i];
                p.u[((int64_t)split * p.num_tokens + t) * n + n0 + i] = sum * scale;
            }
        }
        __syncthreads();                 // the sums are read
    }
}

// ---------------------------------------------------------------------------
// the up-projection, added to the rows
// ---------------------------------------------------------------------------
//
// Columns are taken 32 at a time (a slice ends at a multiple of 64).  Column 8 (n / 2) + 2 i +
// n % 2 of the 32 is column n of the MMA's i-th tile, so that a lane's four accumulators of a row
// are 8 neighbouring columns: 16-byte loads and stores of the rows, which the accumulators begin
// with.  u is summed over the pieces of K, in their order, and split into three bf16 parts, which hold
// all 24 bits of it: with two, 17 bits, one output in 500 falls to another bf16 value than fp32 sums give
// (three: one in 800 to 3,000, the sums' order), 8,192 tokens of rank 64 take 137 us for 152, of rank 32
// 103 for 107, 64 tokens over 48 adapters of rank 16 18.1 for 18.7.
//   RC      ceil(rank / 16), rounded up to a power of two
//   EXACT   the rank is 16 RC: offsets into up are constants, and no lane is beyond it

// What a warp has of its tile of tokens and of u.
template <int RC, bool EXACT>
struct UpTile {
    int rank, n, g, q;
    bool live[2];                    // rows g and g + 8 are read and written
    const uint16_t *src[2];
    uint16_t *dst[2];
    const float *u[2];               // nullptr: no adapter
    uint32_t hi[RC][4], mid[RC][4], lo[RC][4];
    int slice, slice_end;

    // `token`: of slot lane % 16, -1 without one
    __device__ __forceinline__ void init(const AdapterParams &p, int token, bool adapter)
    {
        rank = EXACT ? 16 * RC : p.rank;
        n = p.num_slices * rank;
        g = (threadIdx.x & 31) >> 2;
        q = threadIdx.x & 3;
        slice = -1;
        slice_end = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t t = __shfl_sync(0xffffffffu, token, g + 8 * h);
            live[h] = t >= 0;
            src[h] = p.rows + t * p.rows_stride + 8 * q;
            dst[h] = p.out + t * p.out_stride + 8 * q;
            u[h] = live[h] && adapter ? p.u + t * n : nullptr;
        }
    }
    // the parts of u for the slice of column c, when that is another one
    __device__ __forceinline__ void slice_of(const AdapterParams &p, int c, int splits)
    {
        if (c < slice_end)
            return;
        do
            ++slice;
        while (c >= p.slice_end[slice]);
        slice_end = p.slice_end[slice];
        // Parts that are loaded at once: the loop over them is a chain of reads from L2 (one part and
        // piece after another: 16 tokens over 16 adapters of rank 64 26.4 us for 20.9, 5,000 tokens of rank 48
        // 106 for 98).  With ranks up to 16 a row's parts come before the other row's, which a tile
        // of a few tokens does not have: one token 5.6 us, and 6.2 with both rows' at once.
        constexpr int U = RC == 1 ? 4 : RC == 2 ? 2 : 1, H = RC == 1 ? 1 : 2;
        float4 v[RC][2] = {};
#pragma unroll
        for (int h0 = 0; h0 < 2; h0 += H) {
            if (H == 1 && !__any_sync(0xffffffffu, u[h0] != nullptr))
                continue;
            for (int s0 = 0; s0 < splits; s0 += U) {
                float4 x[U][RC][H] = {};
#pragma unroll
                for (int s = 0; s < U; ++s)
#pragma unroll
                    for (int k = 0; k < RC; ++k)
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            if (s0 + s < splits && u[h0 + h] && (EXACT || 16 * k + 4 * q < rank))
                                x[s][k][h] = *reinterpret_cast<const float4 *>(
                                    u[h0 + h] + (int64_t)(s0 + s) * p.num_tokens * n + slice * rank + 16 * k + 4 * q);
#pragma unroll
                for (int s = 0; s < U; ++s)
#pragma unroll
                    for (int k = 0; k < RC; ++k)
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            float4 &y = v[k][h0 + h];
                            y = make_float4(y.x + x[s][k][h].x, y.y + x[s][k][h].y, y.z + x[s][k][h].z, y.w + x[s][k][h].w);
                        }
            }
        }
#pragma unroll
        for (int k = 0; k < RC; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                adapter_split(v[k][h].x, v[k][h].y, hi[k][h], mid[k][h], lo[k][h]);
                adapter_split(v[k][h].z, v[k][h].w, hi[k][h + 2], mid[k][h + 2], lo[k][h + 2]);
            }
    }
    // a word of the rows g and g + 8, of the MMA's tile i, with what an adapter's rows w add
    __device__ __forceinline__ void add(uint32_t r0, uint32_t r1, const uint2 (&w)[RC], uint32_t &o0, uint32_t &o1) const
    {
        const float2 a = unpack2(r0), b = unpack2(r1);
        float acc[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int k = 0; k < RC; ++k) {
            mma(acc, hi[k], w[k].x, w[k].y);
            mma(acc, mid[k], w[k].x, w[k].y);
            mma(acc, lo[k], w[k].x, w[k].y);
        }
        o0 = adapter_bf16x2(acc[0], acc[1]);
        o1 = adapter_bf16x2(acc[2], acc[3]);
    }
};

// A warp takes a tile and `chunk` columns, 32 * PC at a time, whose rows of up and of the tokens
// are loaded at once; the first of them before it waits for u.
template <int RC, bool EXACT>
__global__ void __launch_bounds__(128, RC <= 2 ? 4 : 2) msa_adapter_up_kernel(const __grid_constant__ AdapterParams p)
{
    constexpr int PC = RC == 1 ? 4 : RC == 2 ? 2 : 1;
    __shared__ __align__(16) TileList s_tiles;
    Tiles tiles;
    tiles.load(p, s_tiles);
    const int count = p.out != p.rows ? tiles.all : tiles.with_adapter;
    const int chunks = (p.width + p.chunk - 1) / p.chunk;
    const int64_t work = (int64_t)count * chunks;
    bool waited = false;
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); item < work; item += (int64_t)gridDim.x * 4) {
        const int from = (int)(item % chunks) * p.chunk, end = min(p.width, from + p.chunk);
        int a, token;
        tiles.get(p, s_tiles, (int)(item / chunks), a, token);
        UpTile<RC, EXACT> t;
        t.init(p, token, a >= 0);
        const int up_row = 8 * (t.g >> 1) + (t.g & 1);
        for (int c0 = from; c0 < end; c0 += 32 * PC) {
            uint32_t in[PC][2][4];
            uint2 w[PC][4][RC];
#pragma unroll
            for (int b = 0; b < PC; ++b) {
                const int c = c0 + 32 * b;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (t.live[h] && c + 8 * t.q < end) {
                        const uint4 r = early(reinterpret_cast<const uint4 *>(t.src[h] + c));
                        in[b][h][0] = r.x, in[b][h][1] = r.y, in[b][h][2] = r.z, in[b][h][3] = r.w;
                    }
                if (a < 0)
                    continue;
                const uint16_t *up = p.up + ((int64_t)a * p.width + c + up_row) * t.rank + 4 * t.q;
                const bool whole = EXACT && c + 32 <= end;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < RC; ++k)
                        if (whole || (c + up_row + 2 * i < end && (EXACT || 16 * k + 4 * t.q < t.rank)))
                            w[b][i][k] = early(reinterpret_cast<const uint2 *>(up + 2 * i * t.rank + 16 * k));
                        else
                            w[b][i][k] = make_uint2(0, 0);
            }
            if (!waited)
                wait_for_kernels_ahead();
            waited = true;
#pragma unroll
            for (int b = 0; b < PC; ++b) {
                const int c = c0 + 32 * b;
                if (c >= end)
                    break;
                if (a >= 0) {
                    t.slice_of(p, c, tiles.splits);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        t.add(in[b][0][i], in[b][1][i], w[b][i], in[b][0][i], in[b][1][i]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (t.live[h] && c + 8 * t.q < end)
                        *reinterpret_cast<uint4 *>(t.dst[h] + c) = make_uint4(in[b][h][0], in[b][h][1], in[b][h][2], in[b][h][3]);
            }
        }
    }
    if (!waited)                         // no CTA finishes before its wait
        wait_for_kernels_ahead();
}

// The same for tiles of 128 tokens, whose rows are what costs (8,192 of 11,392 are 373 MB, 56 us
// at the copy rate).  A CTA takes a tile and `chunk` columns, a warp 16 of its tokens.  The
// adapter's rows of up and the tokens' rows go through shared memory, kUpStage columns ahead of
// those that are computed: a lane copies the pieces of rows that it uses, 8 KB a warp, 128 KB an
// SM in flight (with two blocks of 32 columns in registers, 32 KB an SM, 80 us and not 70; from rank 33
// on, whose registers leave one CTA an SM, 64 KB).  The
// 32-byte pieces of a row of up are placed so that the rows 0, 1, 8 and 9 (16, 17, 24 and 25), of
// which a half warp loads a piece each, lie on different banks: the two rows 2 apart go elsewhere
// (ranks up to 16), or the piece's number is changed.
constexpr int kUpStage = 128;        // columns of a stage of up

template <int RC>
__device__ __forceinline__ uint32_t up_piece(int row, int k)       // byte offset of piece k of a row of a stage
{
    const uint32_t r = (uint32_t)row, far = r >> 3 & 1u;
    if (RC == 1)
        return 32u * ((r & ~10u) | far << 1 | (r >> 1 & 1u) << 3);
    return 32u * ((r * RC + (uint32_t)k) ^ (RC == 2 ? far : (r & 1u) | far << 1));
}

// From row 8 a + b to row 8 a + b + 2 i (b 0 or 1) of a stage.
template <int RC>
__device__ constexpr uint32_t up_step(int i)
{
    return RC == 1 ? 32u * ((i & 1) * 8 + (i >> 1) * 4) : 32u * RC * 2 * i;
}

template <int RC, bool EXACT>
__global__ void __launch_bounds__(256, RC <= 2 ? 2 : 1) msa_adapter_up_stream_kernel(const __grid_constant__ AdapterParams p)
{
    extern __shared__ __align__(128) uint8_t s_up[];                 // two stages of up, two of each warp's rows
    constexpr uint32_t kStageBytes = 32u * RC * kUpStage, kRowBytes = 16u * 32u * 2u * (kUpStage / 32);
    const int tid = threadIdx.x, warp = tid >> 5, splits = early(&p.head->splits);
    const int count = early(p.out != p.rows ? &p.head->tiles : &p.head->with_adapter);
    const int chunks = (p.width + p.chunk - 1) / p.chunk;
    const int64_t work = (int64_t)count * chunks;
    const uint32_t s0 = (uint32_t)__cvta_generic_to_shared(s_up);
    const uint32_t s_rows = s0 + 2u * kStageBytes + (uint32_t)warp * (2u * kRowBytes) + 16u * (uint32_t)(tid & 31);
    bool waited = false;
    for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
        const int tile = (int)(item % count), from = (int)(item / count) * p.chunk, end = min(p.width, from + p.chunk);
        const int a = early(p.adapters + tile);
        UpTile<RC, EXACT> t;
        t.init(p, early(p.tokens + tile * 128 + warp * kTile + (tid & 15)), a >= 0);
        // 16 bytes, zeros where there is nothing
        auto copy16 = [](uint32_t to, const uint16_t *from, bool there) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
        };
        auto stage = [&](int c, uint32_t buf) {
#pragma unroll
            for (int b = 0; b < kUpStage / 32; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool there = t.live[h] && c + 32 * b + 8 * t.q < end;
                    copy16(s_rows + buf * kRowBytes + (uint32_t)(2 * b + h) * 512u, there ? t.src[h] + c + 32 * b : p.rows, there);
                }
            // halves of pieces of up
            if (a >= 0) {
                const uint16_t *up = p.up + ((int64_t)a * p.width + c) * t.rank;
#pragma unroll
                for (int e0 = 0; e0 < kUpStage * 2 * RC; e0 += 256) {
                    const int e = e0 + tid, row = e / (2 * RC), h = e % (2 * RC);
                    const bool there = c + row < end && (EXACT || 8 * h < t.rank);
                    copy16(s0 + buf * kStageBytes + up_piece<RC>(row, h >> 1) + 16u * (h & 1),
                           there ? up + row * t.rank + 8 * h : p.up, there);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        stage(from, 0);
        if (from + kUpStage < end)
            stage(from + kUpStage, 1);
        if (!waited)
            wait_for_kernels_ahead();
        waited = true;
        const int up_row = 8 * (t.g >> 1) + (t.g & 1);
        uint32_t at[RC];                 // of this lane's piece k of row up_row
#pragma unroll
        for (int k = 0; k < RC; ++k)
            at[k] = s0 + up_piece<RC>(up_row, k) + 8u * t.q;
        for (int c0 = from, it = 0; c0 < end; c0 += kUpStage, ++it) {
            if (c0 + kUpStage < end)
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            else
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            const uint32_t buf = (uint32_t)(it & 1);
#pragma unroll 2
            for (int b = 0; b < kUpStage / 32; ++b) {
                const int c = c0 + 32 * b;
                if (c >= end)
                    break;
                uint32_t r[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(r[h][0]), "=r"(r[h][1]), "=r"(r[h][2]), "=r"(r[h][3])
                                 : "r"(s_rows + buf * kRowBytes + (uint32_t)(2 * b + h) * 512u));
                if (a >= 0) {
                    t.slice_of(p, c, splits);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint2 w[RC];
#pragma unroll
                        for (int k = 0; k < RC; ++k)
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                         : "=r"(w[k].x), "=r"(w[k].y)
                                         : "r"(at[k] + buf * kStageBytes + (uint32_t)b * (1024u * RC) + up_step<RC>(i)));
                        t.add(r[0][i], r[1][i], w, r[0][i], r[1][i]);
                    }
                }
                if (c + 8 * t.q < end)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (t.live[h])
                            *reinterpret_cast<uint4 *>(t.dst[h] + c) = make_uint4(r[h][0], r[h][1], r[h][2], r[h][3]);
            }
            __syncthreads();
            if (c0 + 2 * kUpStage < end)
                stage(c0 + 2 * kUpStage, buf);
        }
    }
    if (!waited)
        wait_for_kernels_ahead();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr int64_t kMaxTokens = 1 << 24;
constexpr int32_t kMaxSize = 1 << 30;    // of K and W: a tile or a chunk more is an int32 too

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
    if (cfg->hidden_size > kMaxSize)
        return fail(MSA_ERR_UNSUPPORTED, "hidden_size %d (at most 2^30)", cfg->hidden_size);
    if (cfg->rank < 1)
        return fail(MSA_ERR_INVALID_ARGUMENT, "rank %d", cfg->rank);
    if (cfg->rank % 8 || cfg->rank > 128)
        return fail(MSA_ERR_UNSUPPORTED, "rank %d (multiples of 8, at most 128)", cfg->rank);
    if (cfg->num_adapters < 1)
        return fail(MSA_ERR_INVALID_ARGUMENT, "num_adapters %d", cfg->num_adapters);
    if (cfg->num_adapters > kMaxAdapters)
        return fail(MSA_ERR_UNSUPPORTED, "num_adapters %d (at most %d)", cfg->num_adapters, kMaxAdapters);
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
        if (end > kMaxSize)
            return fail(MSA_ERR_UNSUPPORTED, "slice_end[%d] is %d (at most 2^30)", s, end);
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

// How a call's work is cut, and what its workspace holds.
struct Plan {
    bool wide;               // tiles of 128 tokens (msa_adapter_tile.cu); else of 16
    bool sorted;             // by a kernel: more than 128 tokens, or wide tiles
    int n_blocks, n_tiles;   // tiles of 16: blocks of at most 48 rows of down (two CTAs an SM), tiles of 8 rows in each
    int max_splits;          // pieces of K
    int64_t tiles;           // at most
    int64_t adapters, tokens, u, bytes;      // offsets into the workspace
};

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// The tokens from which on a call takes wide tiles.
//
// Narrow tiles read the hidden states once for each block of 48 rows of down and an adapter once for 16
// tokens, wide ones start later and have fewer CTAs.  Where the sides meet, T^2 * rows * K is 2.5e11 to
// 9e11, of bf16 and E4M3 (6,144 wide hidden states and 11,392 wide rows, three adapters' chunks, narrow
// and wide us: 80 rows 27.1 and 27.3 at 1,000 tokens, 160 rows 21.6 and 22.2 at 500, 37.1 and 31.6 at
// 1,000, 320 rows 20.1 and 30.7 at 300, 31.6 and 29.8 at 500, 54.2 and 38.9 at 1,000; 1,000 and 960 wide,
// 160 rows 13.4 and 15.0 at 1,500, 17.0 and 15.8 at 2,000).  Adapters in no order fill wide
// tiles badly below 56 tokens each (16 of them, 320 rows: 37.4 and 60.6 at 500 tokens, 60.2 and 61.0 at
// 1,000); a batch of 900 tokens or more is taken for a prefill's chunks.  That is a guess: the rule sees
// the table, not how many of its adapters a batch has.  One request's 600 tokens beside a table of 16
// or more take narrow tiles, 900 requests of one token each wide ones.
int64_t wide_from(const msa_adapter_cfg *cfg)
{
    const double rows = (double)cfg->num_slices * cfg->rank;
    const int64_t tokens = (int64_t)std::ceil(std::sqrt(5e11 / (rows * cfg->hidden_size)));
    const int64_t mixed = 56 * (int64_t)(cfg->num_adapters < 16 ? cfg->num_adapters : 16);
    const int64_t from = tokens > mixed ? tokens : mixed;
    return from > kTile + 1 ? from : kTile + 1;
}

Plan plan_of(const msa_adapter_cfg *cfg, int64_t T)
{
    Plan c;
    const int64_t rows = (int64_t)cfg->num_slices * cfg->rank, units = (cfg->hidden_size + kUnitK - 1) / kUnitK;
    c.wide = T >= wide_from(cfg);
    c.sorted = c.wide || T > kListed;
    const int ts = c.wide ? 128 : kTile;
    c.tiles = T / ts + (T < cfg->num_adapters + 1 ? T : cfg->num_adapters + 1);
    c.n_blocks = c.wide ? 1 : (int)((rows / 8 + 5) / 6);
    c.n_tiles = (int)((rows / 8 + c.n_blocks - 1) / c.n_blocks);
    // no fewer than a unit of K for each warp of 8, four for a wide tile; and what the fewest tiles
    // that T tokens can make would take to fill the GPU
    const int64_t most = c.wide ? (units / 4 < 8 ? units / 4 : 8) : (units + kDownWarps - 1) / kDownWarps;
    const int64_t want = fill_of(!c.wide) / (((T + ts - 1) / ts > 0 ? (T + ts - 1) / ts : 1) * c.n_blocks);
    c.max_splits = (int)(want < most ? want : most);
    if (c.max_splits < 1)
        c.max_splits = 1;
    c.adapters = c.sorted ? 256 : 0;
    c.tokens = c.adapters + (c.sorted ? align256(c.tiles * 4) : 0);
    c.u = c.tokens + (c.sorted ? align256(c.tiles * ts * 4) : 0);
    c.bytes = T == 0 ? 0 : c.u + c.max_splits * T * rows * 4;
    return c;
}

int64_t workspace_needed(const msa_adapter_cfg *cfg, int64_t T) { return plan_of(cfg, T).bytes; }

// The most that any call of up to T tokens needs.  What a call needs grows with its tokens but where
// a tile more leaves fewer pieces of K, or where wide tiles begin.
int64_t workspace_for(const msa_adapter_cfg *cfg, int64_t T)
{
    int64_t most = workspace_needed(cfg, T);
    const auto at = [&](int64_t t) {
        const int64_t n = t < T ? workspace_needed(cfg, t) : 0;
        most = n > most ? n : most;
    };
    for (const int ts : {kTile, 128})
        for (int64_t t = ts; t < T && t <= (int64_t)kFill * ts; t += ts)
            at(t);
    at(wide_from(cfg) - 1);
    return most;
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// a * b * c as non-negative int64
bool fits(int64_t a, int64_t b, int64_t c)
{
    int64_t m;
    return !__builtin_mul_overflow(a, b, &m) && !__builtin_mul_overflow(m, c, &m);
}

msa_status check_args(const msa_adapter_cfg *cfg, int64_t T, const AdapterParams &p, const void *workspace,
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
    if (p.down_stride >= (int64_t)1 << 39)           // TMA's limit is 2^40 bytes
        return fail(MSA_ERR_UNSUPPORTED, "down_stride %lld (below 2^39)", (long long)p.down_stride);
    if (!workspace || workspace_bytes < workspace_needed(cfg, T))
        return fail(MSA_ERR_INVALID_ARGUMENT, "workspace: %lld bytes, %lld needed",
                    (long long)(workspace ? workspace_bytes : 0), (long long)workspace_needed(cfg, T));
    if (!aligned(workspace, 256))
        return fail(MSA_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    return MSA_OK;
}

using Kernel = void (*)(AdapterParams);

// by rank: 16, 32, 64, 128 exactly, or up to them
const Kernel kUpKernels[2][4] = {{msa_adapter_up_kernel<1, false>, msa_adapter_up_kernel<2, false>,
                                  msa_adapter_up_kernel<4, false>, msa_adapter_up_kernel<8, false>},
                                 {msa_adapter_up_kernel<1, true>, msa_adapter_up_kernel<2, true>,
                                  msa_adapter_up_kernel<4, true>, msa_adapter_up_kernel<8, true>}};
const Kernel kUpStreamKernels[2][4] = {{msa_adapter_up_stream_kernel<1, false>, msa_adapter_up_stream_kernel<2, false>,
                                        msa_adapter_up_stream_kernel<4, false>, msa_adapter_up_stream_kernel<8, false>},
                                       {msa_adapter_up_stream_kernel<1, true>, msa_adapter_up_stream_kernel<2, true>,
                                        msa_adapter_up_stream_kernel<4, true>, msa_adapter_up_stream_kernel<8, true>}};

// Dynamic shared memory of the streaming up-projection.
constexpr int up_stream_smem(int rc) { return 2 * (32 << rc) * kUpStage + 8 * 2 * (16 * 32 * 2 * (kUpStage / 32)); }

// Lets the kernels have as much shared memory as any call of theirs takes, once on each device.  (A
// limit is a kernel's, for all threads: one set for each call could fall below what another
// thread's call is about to launch with.)
cudaError_t allow_shared_memory(bool wide)
{
    static std::atomic<uint64_t> done[2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done[wide].load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    auto allow = [&](Kernel k, int smem) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    };
    allow(msa_adapter_sort_kernel, (kMaxAdapters + 1) * 4);
    for (int rc = 0; wide && rc < 4; ++rc) {
        allow(kUpStreamKernels[0][rc], up_stream_smem(rc));
        allow(kUpStreamKernels[1][rc], up_stream_smem(rc));
    }
    if (wide && e == cudaSuccess)
        e = adapter_tile_allow();
    if (e == cudaSuccess)
        done[wide].fetch_or(bit, std::memory_order_release);
    return e;
}

msa_status launch(Kernel kernel, dim3 grid, int threads, int smem, cudaStream_t stream, AdapterParams &p)
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
    lc.numAttrs = 1;
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
    *bytes = workspace_for(cfg, num_tokens);
    return MSA_OK;
}

msa_status msa_adapter_forward(const msa_adapter_cfg *cfg, int64_t num_tokens, const void *hidden,
                               int64_t hidden_stride, const float *hidden_scales, const void *down,
                               int64_t down_stride, const void *up, const int32_t *adapter_ids,
                               const float *adapter_scales, const void *rows, int64_t rows_stride, void *out,
                               int64_t out_stride, void *workspace, int64_t workspace_bytes,
                               int32_t launch_flags, cudaStream_t stream)
{
    AdapterParams p;
    memset(&p, 0, sizeof p);
    p.hidden = static_cast<const uint8_t *>(hidden);
    p.hidden_scales = hidden_scales;
    p.down = static_cast<const uint16_t *>(down);
    p.up = static_cast<const uint16_t *>(up);
    p.ids = adapter_ids;
    p.adapter_scales = adapter_scales;
    p.rows = static_cast<const uint16_t *>(rows);
    p.out = static_cast<uint16_t *>(out);
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
    const Plan c = plan_of(cfg, num_tokens);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.head = reinterpret_cast<AdapterHead *>(ws);
    p.adapters = reinterpret_cast<int32_t *>(ws + c.adapters);
    p.tokens = c.sorted ? reinterpret_cast<int32_t *>(ws + c.tokens) : nullptr;
    p.u = reinterpret_cast<float *>(ws + c.u);
    p.tile_tokens = c.wide ? 128 : kTile;
    p.max_splits = c.max_splits;
    p.n_blocks = c.n_blocks;
    p.n_tiles = c.n_tiles;
    // all that can fail ahead of the first launch
    AdapterTilePlan tile_plan;
    if (c.sorted) {
        const cudaError_t e = allow_shared_memory(c.wide);
        if (e != cudaSuccess)
            return fail(MSA_ERR_CUDA, "cudaFuncSetAttribute failed: %s", cudaGetErrorString(e));
    }
    if (c.wide && !adapter_tile_plan(p, &tile_plan))
        return fail(MSA_ERR_CUDA, "down: no tensor map");
    if (c.sorted) {
        const int smem = (p.num_adapters + 1) * 4;
        // as many threads as have something to do: barriers of 1,024 take 1 us more
        const int64_t most = num_tokens > p.num_adapters + 1 ? num_tokens : p.num_adapters + 1;
        const int threads = most >= 1024 ? 1024 : (int)((most + 31) / 32 * 32);
        const msa_status d = launch(msa_adapter_sort_kernel, dim3(1), threads, smem, stream, p);
        if (d != MSA_OK)
            return d;
    }
    if (c.wide) {
        const cudaError_t e = adapter_tile_launch(p, tile_plan, c.tiles, stream);
        if (e != cudaSuccess)
            return fail(MSA_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
    } else {
        static const Kernel downs[2][3] = {
            {msa_adapter_down_kernel<false, 2>, msa_adapter_down_kernel<false, 4>, msa_adapter_down_kernel<false, 6>},
            {msa_adapter_down_kernel<true, 2>, msa_adapter_down_kernel<true, 4>, msa_adapter_down_kernel<true, 6>}};
        const int64_t work = c.tiles * c.n_blocks * c.max_splits;
        const msa_status d = launch(downs[p.fp8][(c.n_tiles - 1) / 2], dim3((unsigned)(work < kFill ? work : kFill)),
                                    32 * kDownWarps, 0, stream, p);
        if (d != MSA_OK)
            return d;
    }

    const int k16 = (p.rank + 15) / 16, rc = k16 <= 1 ? 0 : k16 <= 2 ? 1 : k16 <= 4 ? 2 : 3;
    const bool exact = p.rank == 16 << rc;
    if (!c.wide) {
        // columns of a warp: what it loads at once, or more where the warps are enough all the same
        p.chunk = rc == 0 ? 128 : rc == 1 ? 64 : 32;
        while (p.chunk < 512 && c.tiles * ((p.width + p.chunk - 1) / p.chunk) > kUpWarps)
            p.chunk *= 2;
        const int64_t ctas = (c.tiles * ((p.width + p.chunk - 1) / p.chunk) + 3) / 4;
        return launch(kUpKernels[exact][rc], dim3((unsigned)(ctas < 8 * 152 ? ctas : 8 * 152)), 128, 0, stream, p);
    }
    const int64_t groups = (num_tokens + 127) / 128;
    // Each chunk reads all parts of u again, max_splits * rank * 4 bytes a token and slice beside its own
    // 4 a column: chunks grow until that is a quarter, while there are two CTAs for each SM (2,048 tokens
    // of rank 64 64.2 us without and 55.4 with, 1,024 of rank 32 33.8 and 30.0, 512 of rank 96 47.1 and 40.7;
    // for 4,000 of rank 8, whose u is small, as large chunks take 57.2 for 54.8).
    p.chunk = kUpStage;
    while (p.chunk < 1024) {
        const int64_t items = groups * ((p.width + p.chunk - 1) / p.chunk);
        if (items <= 2 * 152 || (items <= 8 * 152 && p.chunk >= 4 * p.max_splits * p.rank))
            break;
        p.chunk *= 2;
    }
    const int64_t ctas = c.tiles * ((p.width + p.chunk - 1) / p.chunk);
    return launch(kUpStreamKernels[exact][rc], dim3((unsigned)(ctas < 8 * 152 ? ctas : 8 * 152)), 256, up_stream_smem(rc),
                  stream, p);
}

}  // extern "C"
