// The adapters of large batches: tiles of 128 tokens on the tcgen05 tensor cores
// (include/msa_adapter.h).
//
// Down-projection.  A CTA takes 128 consecutive tokens, a piece of K, and every second distinct adapter of the tile
// (a prefill chunk has one, two at its border); all of an adapter's num_slices * rank rows are
// the MMA's N, so that the hidden states are read once, which is what bounds the kernel: 8,192
// tokens of 6,144 E4M3 values are 50 MB, 7.5 us at the copy rate.
//   warp 0      copies: 64-element K blocks of the adapter's rows (and of bf16 hidden states) by
//               TMA into a ring of stages, 128-byte rows in the 128-byte swizzle
//   warp 1      tensor-memory owner; issues the MMAs (M 128, N up to 2 x 256, K 16)
//   warps 2..9  E4M3 hidden states: loaded a few K blocks ahead into registers, made bf16 (exact)
//               and stored in the swizzle; then the accumulator, scaled, to the partial sums
// A token of another adapter has a row of its own in the MMA, which is not written.
//
// Up-projection.  Reading and writing the rows bounds it: 8,192 rows of 11,392 are 373 MB, 56 us
// at the copy rate.  A persistent CTA takes an equal share of the (tile, block of 64 columns)s, a
// tile's one after another, so that u is made once for most of them:
//   warp 0       copies: row blocks (128 tokens x 64 columns) and, for each distinct adapter of
//                the tile, its 64 rows of up, by TMA into rings
//   warps 1..3   one for each group of adding warps: MMAs of u's two bf16 parts, hi and lo, against
//                the same 64 rows (M 128, N 64), into the next of the group's two accumulators
//   warps 4..7   u of the next (tile, slice): the pieces of K added in their order, in two parts
//   warps 8..19  three groups, a row block each by turns: add the accumulator to the rows of its
//                adapter's tokens, in the row block
//   warp 20      stores finished row blocks by TMA
// Blocks go by turns because a block's waits and instructions, one after another, take longer
// than its share of the copies (0.75 us): with one MMA warp and eight adding warps that took each
// block together 167 us, with three groups 120, counting ring places on in place of divisions 108.
// A stage or accumulator belongs to one group, so that no wait can come a phase too early.
// (A version on mma.sync with the rows in registers took 125 us for that, at 309 instructions a
// warp for 16 tokens x 32 columns; this one has a sixth of them.)
// Every wait is bounded; rows that a CTA could not finish are NaN.

#include "msa_adapter_internal.h"
#include "msa_tcgen05.cuh"

#include <cstring>

namespace {

constexpr int kM = 128;                       // tokens of a tile
constexpr int kBlockK = 64;                   // K elements of a stage: 128 bytes of bf16
constexpr int kMaxStages = 8;
constexpr int kWorkers = 8;                   // conversion and epilogue warps
constexpr int kThreads = 64 + 32 * kWorkers;
constexpr int kAhead = 4;                     // K blocks of E4M3 values loaded ahead
constexpr int kMaxSplits = kAdapterWideSplits;
constexpr uint32_t kTileX = kM * 128;

struct TileShape {
    int32_t n;           // rows of down an MMA pair takes: a multiple of 16 (32 where two boxes)
    int32_t boxes;       // 1 or 2 of at most 256 rows
    int32_t stages;
    int32_t tmem;        // columns allocated
    uint32_t stage_bytes;
};

// A place in a ring of n stages or buffers, and the parity of its phase.  (Counted on: divisions
// by a number that is not known to the compiler cost every role 0.1 us each.)
struct Ring {
    uint32_t at = 0, phase = 0, n;

    __device__ __forceinline__ explicit Ring(uint32_t stages) : n(stages) {}
    __device__ __forceinline__ void next()
    {
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
};

// warp_wait, whose limit begins with a first sleep that reads no timer: a read takes longer than
// most waits here.
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (__all_sync(0xffffffffu, mbar_try(bar, parity)))
        return true;
    if (__all_sync(0xffffffffu, mbar_try_asleep(bar, parity)))
        return true;
    return warp_wait(bar, parity, abort_flag);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// An MMA, and an arrival when all of this thread's are complete, by one thread: made once for
// all, descriptors are moved on by adding to them.  (Issued by a whole warp with descriptors made
// anew, four MMAs and two commits took 1 us; as here ... .)
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void commit_one(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 codes of a row from k on, zeros from K on
__device__ __forceinline__ uint4 load_codes(const uint8_t *row, int k, int hidden)
{
    const int n = hidden - k;
    if (n >= 16)
        return __ldg(reinterpret_cast<const uint4 *>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (j < n)
            w[j / 4] |= (uint32_t)row[k + j] << (8 * (j & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads)
msa_adapter_down_tile_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ TileShape s,
                             const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kMaxStages], bar_empty[kMaxStages], bar_acc, bar_free, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_count[4], s_id[kM], s_list[kM];
    volatile int *abort_flag = &s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;

    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the tile's distinct adapters, in the order of their first tokens
    const int64_t t0 = (int64_t)blockIdx.x * kM;
    int id = -1;
    uint32_t leaders = 0;
    if (warp < 4) {
        if (t0 + tid < p.num_tokens)
            id = p.ids[t0 + tid];
        if (id >= p.num_adapters || id < 0)
            id = -1;
        s_id[tid] = id;
    }
    __syncthreads();
    if (warp < 4) {
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        leaders = __ballot_sync(0xffffffffu, id >= 0 && lane == __ffs(same) - 1);
        for (uint32_t left = leaders; left; left &= left - 1) {      // those that an earlier warp has
            const int who = __ffs(left) - 1, a = __shfl_sync(0xffffffffu, id, who);
            bool seen = false;
            for (int v = 0; v < warp; ++v)
                seen |= s_id[32 * v + lane] == a;
            if (__any_sync(0xffffffffu, seen))
                leaders &= ~(1u << who);
        }
        if (lane == 0)
            s_count[warp] = __popc(leaders);
    }
    __syncthreads();
    const int count = s_count[0] + s_count[1] + s_count[2] + s_count[3];
    const int pass0 = blockIdx.z, pass_step = gridDim.z;
    if (pass0 >= count)
        return;
    if (warp < 4 && (leaders >> lane & 1)) {
        int at = __popc(leaders & ((1u << lane) - 1u));
        for (int v = 0; v < warp; ++v)
            at += s_count[v];
        s_list[at] = id;
    }
    if (tid == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(smem_u32(&bar_full[i]), FP8 ? 1 + kWorkers : 1);
            mbar_init(smem_u32(&bar_empty[i]), 1);
        }
        mbar_init(smem_u32(&bar_acc), 1);
        mbar_init(smem_u32(&bar_free), kWorkers);
        mbar_init(smem_u32(&bar_drain), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&s_tmem), (uint32_t)s.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (not before: the next kernel must not take tensor memory that this one still waits for)
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const uint32_t tmem = s_tmem;

    const int rows = p.num_slices * p.rank;
    const int blocks = (p.hidden_size + kBlockK - 1) / kBlockK;
    const int k0 = (int)((int64_t)blocks * blockIdx.y / gridDim.y), k1 = (int)((int64_t)blocks * (blockIdx.y + 1) / gridDim.y);
    const uint32_t ST = (uint32_t)s.stages;

    if (warp == 0) {
        // ---------------- copies ----------------
        Ring st(ST);
        uint32_t it = 0;
        bool ok = true;
        for (int pass = pass0; ok && pass < count; pass += pass_step) {
            const int y = s_list[pass] * rows;
            for (int kb = k0; kb < k1; ++kb, ++it, st.next()) {
                const uint32_t full = smem_u32(&bar_full[st.at]);
                ok = tile_wait(smem_u32(&bar_empty[st.at]), st.phase ^ 1u, abort_flag);
                if (!ok)
                    break;
#ifndef MSA_STARVE
                const uint32_t x = ring + st.at * s.stage_bytes;
                if (lane == 0) {
                    mbar_expect_tx(full, (uint32_t)s.n * 128u + (FP8 ? 0u : kTileX));
                    for (int b = 0; b < s.boxes; ++b)
                        tma_load_2d(x + kTileX + (uint32_t)(b * (s.n / s.boxes)) * 128u, &wmap, kb * kBlockK,
                                    y + b * (s.n / s.boxes), full);
                    if (!FP8)
                        tma_load_2d(x, &xmap, kb * kBlockK, (int32_t)t0, full);
                }
                __syncwarp();
#else
                (void)full;
                (void)y;
#endif
            }
        }
        if (!ok)
            *abort_flag = 1;
#ifndef MSA_STARVE
        // every copy has landed before the CTA finishes
        for (uint32_t i = 0; i < ST && i < it; ++i)
            (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_full[i]), ((it - 1u - i) / ST) & 1u));
#endif
    } else if (warp == 1) {
        // ---------------- MMAs ----------------
        const int half = s.n / s.boxes;
        const uint32_t idesc = mma_idesc(1, 1, kM, half, false, false);
        const uint64_t desc = smem_desc(ring, 128, 16u, 1024u);
        Ring st(ST);
        uint32_t done = 0;
        bool ok = true;
        for (int pass = pass0; ok && pass < count; pass += pass_step, ++done) {
            if (done > 0)
                ok = tile_wait(smem_u32(&bar_free), (done - 1u) & 1u, abort_flag);
            for (int kb = k0; ok && kb < k1; ++kb, st.next()) {
                ok = tile_wait(smem_u32(&bar_full[st.at]), st.phase, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t a = desc + st.at * (s.stage_bytes >> 4);
                    for (int b = 0; b < s.boxes; ++b)
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k)
                            mma_one(tmem + (uint32_t)(b * half), a + 2 * k, a + (kTileX >> 4) + (uint32_t)(b * half) * 8u + 2 * k,
                                    idesc, kb > k0 || k > 0);
                    commit_one(smem_u32(&bar_empty[st.at]));
                    if (kb == k1 - 1)
                        commit_one(smem_u32(&bar_acc));
                }
                __syncwarp();
            }
        }
        if (!ok)
            *abort_flag = 1;
        if (lane == 0)
            commit_one(smem_u32(&bar_drain));   // every MMA has completed before tensor memory is released
        __syncwarp();
        (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_drain), 0));
    } else {
        // ---------------- conversion and epilogue ----------------
        const int w = tid - 64, quarter = warp & 3, row = quarter * 32 + lane, part = (warp - 2) >> 2;
        const int64_t t = t0 + row;
        const float hs = p.hidden_scales && t < p.num_tokens ? p.hidden_scales[t] : 1.0f;
        Ring st(ST);
        uint32_t done = 0;
        bool ok = true;
        for (int pass = pass0; pass < count; pass += pass_step, ++done) {
            const int a = s_list[pass];
            if (FP8) {
                // this thread's pieces of 16 codes: of rows w / 4 and 64 + w / 4
                const int col = 16 * (w & 3);
                const uint8_t *src[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = (w >> 2) + 64 * h;
                    src[h] = s_id[r] == a ? p.hidden + (t0 + r) * p.hidden_stride : nullptr;
                }
                uint4 next[kAhead][2];
#pragma unroll
                for (int d = 0; d < kAhead; ++d)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        next[d][h] = src[h] && k0 + d < k1 ? load_codes(src[h], (k0 + d) * kBlockK + col, p.hidden_size)
                                                           : make_uint4(0, 0, 0, 0);
                for (int kb = k0; ok && kb < k1; kb += kAhead) {
#pragma unroll
                    for (int d = 0; d < kAhead; ++d) {
                        if (!ok || kb + d >= k1)
                            break;
                        ok = tile_wait(smem_u32(&bar_empty[st.at]), st.phase ^ 1u, abort_flag);
                        if (!ok)
                            break;
                        const uint32_t x = ring + st.at * s.stage_bytes;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 c = next[d][h];
                            const uint32_t off = (uint32_t)((w >> 2) + 64 * h) * 128u + 2u * (uint32_t)col;
                            sts128(x + swizzle<128>(off), adapter_e4m3x2(c.x & 0xffffu), adapter_e4m3x2(c.x >> 16),
                                   adapter_e4m3x2(c.y & 0xffffu), adapter_e4m3x2(c.y >> 16));
                            sts128(x + swizzle<128>(off + 16u), adapter_e4m3x2(c.z & 0xffffu), adapter_e4m3x2(c.z >> 16),
                                   adapter_e4m3x2(c.w & 0xffffu), adapter_e4m3x2(c.w >> 16));
                            if (src[h] && kb + d + kAhead < k1)
                                next[d][h] = load_codes(src[h], (kb + d + kAhead) * kBlockK + col, p.hidden_size);
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_u32(&bar_full[st.at]));
                        st.next();
                    }
                }
            }
            ok = ok && tile_wait(smem_u32(&bar_acc), done & 1u, abort_flag);
            const float c = hs * (p.adapter_scales ? p.adapter_scales[a] : 1.0f);
            const bool mine = s_id[row] == a;
            float *dst = p.u + ((int64_t)blockIdx.y * p.num_tokens + t) * rows;
            if (ok)
                tc_fence_after();
            for (int col = 16 * part; col < rows; col += 32) {
                uint32_t v[16];
                if (ok) {
                    tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)col, v);
                    tc_wait_ld();
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (mine && col + 4 * j < rows) {
                        float f[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            f[e] = ok ? c * __uint_as_float(v[4 * j + e]) : __int_as_float(0x7fc00000);
                        *reinterpret_cast<float4 *>(dst + col + 4 * j) = make_float4(f[0], f[1], f[2], f[3]);
                    }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_free));
        }
        if (!ok)
            *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, (uint32_t)s.tmem);
    }
}

// ---------------------------------------------------------------------------
// the up-projection, added to the rows
// ---------------------------------------------------------------------------

constexpr int kBlockN = 64;                   // columns of a row block: 128 bytes
constexpr uint32_t kRowBlock = kM * 128;      // bytes of one
constexpr uint32_t kUpSlab = kBlockN * 128;   // 64 rows of up, 64 elements of the rank
constexpr int kUpGroups = 3;                  // of four warps
constexpr int kAccs = 2;                      // accumulators of a group
constexpr uint32_t kUpTmem = 512;             // columns, of which the groups use 3 x 2 x 64
constexpr int kUpStore = 8 + 4 * kUpGroups;   // the storing warp
constexpr int kUpThreads = 32 * (kUpStore + 1);
constexpr int kRing = 2 * kUpGroups;          // stages of the rows at most, and of up: two of a group

struct UpShape {
    int32_t row_stages;      // 6 or 3: a multiple of the groups
    int32_t u_buffers;       // 1 or 2
    int32_t slabs;           // of 64 elements of the rank: 1 or 2
    int32_t blocks;          // of 64 columns
    int32_t ctas;
    int32_t share, more;     // (tile, block)s of a CTA; the first `more` have one more
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int32_t x, int32_t y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(src)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// The adapters of 128 tokens, held by a warp: token 32 w + lane in id[w], -1 without one.
struct TileIds {
    int id[4];
    uint32_t lead[4];        // the first token of each distinct adapter
    int count;               // distinct adapters

    __device__ __forceinline__ void load(const AdapterParams &p, int64_t t0)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int64_t t = t0 + 32 * w + lane;
            id[w] = t < p.num_tokens ? __ldg(p.ids + t) : -1;
            if (id[w] < 0 || id[w] >= p.num_adapters)
                id[w] = -1;
        }
        count = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t same = __match_any_sync(0xffffffffu, id[w]);
            lead[w] = __ballot_sync(0xffffffffu, id[w] >= 0 && lane == __ffs(same) - 1);
            for (uint32_t left = w > 0 ? lead[w] : 0; left; left &= left - 1) {
                const int who = __ffs(left) - 1, a = __shfl_sync(0xffffffffu, id[w], who);
                bool seen = false;
#pragma unroll
                for (int v = 0; v < 3; ++v)
                    seen |= v < w && id[v] == a;
                if (__any_sync(0xffffffffu, seen))
                    lead[w] &= ~(1u << who);
            }
            count += __popc(lead[w]);
        }
    }
    // f(adapter) for each distinct adapter until it gives false
    template <class F>
    __device__ __forceinline__ bool each(F f) const
    {
        bool ok = true;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            for (uint32_t left = lead[w]; ok && left; left &= left - 1)
                ok = f(__shfl_sync(0xffffffffu, id[w], __ffs(left) - 1));
        return ok;
    }
};

// A CTA's share of the (tile, column block)s, which every role walks in the same order.
struct UpWalk {
    int left, tile;          // left: blocks after this one
    int block, slice, slice_end;
    TileIds ids;
    bool fresh;              // another tile or slice than the last block with adapters had

    __device__ __forceinline__ void start(const AdapterParams &p, const UpShape &s)
    {
        const int at = (int)blockIdx.x * s.share + min((int)blockIdx.x, s.more);
        left = s.share + ((int)blockIdx.x < s.more);
        tile = at / s.blocks;
        block = at - tile * s.blocks - 1;
        slice_end = 0;
        ids.load(p, (int64_t)tile * kM);
    }
    // the next block that has anything to do; `copy`: rows without an adapter are stored too
    __device__ __forceinline__ bool next(const AdapterParams &p, const UpShape &s, bool copy)
    {
        while (left > 0) {
            if (++block == s.blocks) {
                ++tile;
                block = 0;
                slice_end = 0;
                ids.load(p, (int64_t)tile * kM);
            }
            if (ids.count == 0 && !copy) {
                left -= s.blocks - block;
                block = s.blocks - 1;
                continue;
            }
            --left;
            fresh = ids.count > 0 && block * kBlockN >= slice_end;
            if (fresh) {
                slice = 0;
                while (block * kBlockN >= p.slice_end[slice])
                    ++slice;
                slice_end = p.slice_end[slice];
            }
            return true;
        }
        return false;
    }
};

// A pair of stages for each group, as the loading warp goes through them.
struct GroupPairs {
    uint32_t times[kUpGroups] = {};      // uses of each group's pair

    __device__ __forceinline__ uint32_t used(uint32_t g) const { return g == 0 ? times[0] : g == 1 ? times[1] : times[2]; }
    __device__ __forceinline__ uint32_t at(uint32_t g) const { return 2u * g + (used(g) & 1u); }
    __device__ __forceinline__ uint32_t phase(uint32_t g) const { return used(g) >> 1 & 1u; }
    __device__ __forceinline__ void next(uint32_t g)
    {
#pragma unroll
        for (uint32_t i = 0; i < kUpGroups; ++i)
            times[i] += i == g;
    }
};
static_assert(kUpGroups == 3, "GroupPairs");

__global__ void __launch_bounds__(kUpThreads)
msa_adapter_up_tile_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ UpShape s,
                           const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap omap,
                           const __grid_constant__ CUtensorMap umap)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_row[kRing], bar_row_empty[kRing], bar_row_done[kRing];
    __shared__ __align__(8) uint64_t bar_up[kRing], bar_up_empty[kRing], bar_acc[kUpGroups * kAccs], bar_acc_empty[kUpGroups * kAccs];
    __shared__ __align__(8) uint64_t bar_u[2], bar_u_empty[2], bar_drain[kUpGroups];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    volatile int *abort_flag = &s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rows = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t ups = rows + (uint32_t)s.row_stages * kRowBlock;
    const uint32_t us = ups + (uint32_t)(kRing * s.slabs) * kUpSlab;     // [buffer][part][slab] of [128][64] bf16
    const uint32_t u_bytes = 2u * (uint32_t)s.slabs * kRowBlock;
    const uint32_t RS = (uint32_t)s.row_stages, UB = (uint32_t)s.u_buffers;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&bar_row[i]), 1);
            mbar_init(smem_u32(&bar_row_empty[i]), 1);
            mbar_init(smem_u32(&bar_row_done[i]), 4);
            mbar_init(smem_u32(&bar_up[i]), 1);
            mbar_init(smem_u32(&bar_up_empty[i]), 1);
        }
        for (int i = 0; i < kUpGroups * kAccs; ++i) {
            mbar_init(smem_u32(&bar_acc[i]), 1);
            mbar_init(smem_u32(&bar_acc_empty[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar_u[i]), 4);
            mbar_init(smem_u32(&bar_u_empty[i]), kUpGroups);
        }
        for (int i = 0; i < kUpGroups; ++i)
            mbar_init(smem_u32(&bar_drain[i]), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // Tensor memory is taken after the wait, so that the kernels ahead never wait for what this one
    // holds, and before the next kernel may start, so that this one never waits for what that holds.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 1)
        tmem_alloc(smem_u32(&s_tmem), kUpTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const uint32_t tmem = s_tmem;
    const bool copy = p.out != p.rows;
    UpWalk walk;
    walk.start(p, s);

    if (warp == 0) {
        // ---------------- copies ----------------
        Ring row(RS);
        GroupPairs up;
        uint32_t ri = 0, group = 0;
        bool ok = true;
        for (; ok && walk.next(p, s, copy); group = group == kUpGroups - 1 ? 0 : group + 1) {
            ok = tile_wait(smem_u32(&bar_row_empty[row.at]), row.phase ^ 1u, abort_flag);
            if (!ok)
                break;
#ifndef MSA_STARVE
            if (lane == 0) {
                mbar_expect_tx(smem_u32(&bar_row[row.at]), kRowBlock);
                tma_load_2d(rows + row.at * kRowBlock, &rmap, walk.block * kBlockN, walk.tile * kM, smem_u32(&bar_row[row.at]));
            }
            __syncwarp();
#endif
            ++ri;
            row.next();
            ok = walk.ids.each([&](int a) {
                const uint32_t at = up.at(group), full = smem_u32(&bar_up[at]);
                if (!tile_wait(smem_u32(&bar_up_empty[at]), up.phase(group) ^ 1u, abort_flag))
                    return false;
#ifndef MSA_STARVE
                if (lane == 0) {
                    mbar_expect_tx(full, (uint32_t)s.slabs * kUpSlab);
                    for (int b = 0; b < s.slabs; ++b)
                        tma_load_2d(ups + (at * (uint32_t)s.slabs + (uint32_t)b) * kUpSlab, &umap, 64 * b,
                                    a * p.width + walk.block * kBlockN, full);
                }
                __syncwarp();
#else
                (void)a;
                (void)full;
#endif
                up.next(group);
                return true;
            });
        }
        if (!ok)
            *abort_flag = 1;
#ifndef MSA_STARVE
        // every copy has landed before the CTA finishes
        for (uint32_t i = 0; i < RS && i < ri; ++i)
            (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_row[i]), ((ri - 1u - i) / RS) & 1u));
        for (uint32_t i = 0; i < kRing; ++i)
            if (up.times[i / 2] > i % 2)
                (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_up[i]), ((up.times[i / 2] - 1u - i % 2) / 2) & 1u));
#endif
    } else if (warp <= kUpGroups) {
        // ---------------- MMAs ----------------
        constexpr uint32_t idesc = mma_idesc(1, 1, kM, kBlockN, false, false);
        const uint64_t u_desc = smem_desc(us, 128, 16u, 1024u), up_desc = smem_desc(ups, 128, 16u, 1024u);
        const uint32_t part = (uint32_t)s.slabs * (kRowBlock >> 4);      // from u's first part to its second
        const int steps = (p.rank + 15) / 16;
        const uint32_t group = (uint32_t)warp - 1u;
        Ring pair(2), u(UB);             // the group's stages of up and its accumulators go together
        uint32_t turn = 0;
        bool ok = true, first = true;
        for (; ok && walk.next(p, s, copy); turn = turn == kUpGroups - 1 ? 0 : turn + 1) {
            if (walk.fresh) {            // of whichever group: the buffer before is free when all have passed
                if (!first) {
                    if (lane == 0)
                        commit_one(smem_u32(&bar_u_empty[u.at]));
                    __syncwarp();
                    u.next();
                }
                first = false;
                ok = tile_wait(smem_u32(&bar_u[u.at]), u.phase, abort_flag);
            }
            if (turn != group)
                continue;
            const uint64_t ud = u_desc + u.at * (u_bytes >> 4);
            for (int i = 0; ok && i < walk.ids.count; ++i, pair.next()) {
                const uint32_t at = 2u * group + pair.at;
                ok = tile_wait(smem_u32(&bar_up[at]), pair.phase, abort_flag) &&
                     tile_wait(smem_u32(&bar_acc_empty[at]), pair.phase ^ 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t w = up_desc + at * (uint32_t)s.slabs * (kUpSlab >> 4);
                    const uint32_t d = tmem + at * kBlockN;
#pragma unroll 2
                    for (int k = 0; k < steps; ++k) {
                        const uint32_t slab = (uint32_t)k >> 2, in = ((uint32_t)k & 3u) * 2u;
                        const uint64_t a = ud + slab * (kRowBlock >> 4) + in, b = w + slab * (kUpSlab >> 4) + in;
                        mma_one(d, a, b, idesc, k > 0);
                        mma_one(d, a + part, b, idesc, true);
                    }
                    commit_one(smem_u32(&bar_up_empty[at]));
                    commit_one(smem_u32(&bar_acc[at]));
                }
                __syncwarp();
            }
        }
        if (!ok)
            *abort_flag = 1;
        if (lane == 0)
            commit_one(smem_u32(&bar_drain[group]));   // every MMA has completed before tensor memory is released
        __syncwarp();
        (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_drain[group]), 0));
    } else if (warp == kUpStore) {
        // ---------------- stores ----------------
        Ring row(RS);
        uint32_t before = RS;            // the stage of the block before
        bool ok = true;
        while (ok && walk.next(p, s, copy)) {
            ok = tile_wait(smem_u32(&bar_row_done[row.at]), row.phase, abort_flag);
            if (!ok)
                break;
            if (lane == 0) {
                tma_store_2d(&omap, walk.block * kBlockN, walk.tile * kM, rows + row.at * kRowBlock);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                // the block before has been read
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                if (before < RS)
                    mbar_arrive(smem_u32(&bar_row_empty[before]));
            }
            __syncwarp();
            before = row.at;
            row.next();
        }
        if (!ok) {
            // what was not stored: NaN for the rows with an adapter, the others as they are
            *abort_flag = 1;
            do
                for (int w = 0; w < 4; ++w) {
                    const int id = w == 0 ? walk.ids.id[0] : w == 1 ? walk.ids.id[1] : w == 2 ? walk.ids.id[2] : walk.ids.id[3];
                    const int64_t t = (int64_t)walk.tile * kM + 32 * w + lane;
                    if (t < p.num_tokens && (copy || id >= 0))
                        for (int c = walk.block * kBlockN; c < min((walk.block + 1) * kBlockN, p.width); ++c)
                            p.out[t * p.out_stride + c] = id >= 0 ? (uint16_t)0x7fc0 : p.rows[t * p.rows_stride + c];
                    __syncwarp();
                }
            while (walk.next(p, s, copy));
        }
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ---------------- u ----------------
        const int r = tid - 128, n = p.num_slices * p.rank, chunks = (p.rank + 15) / 16 * 2;
        Ring u(UB);
        bool ok = true;
        while (ok && walk.next(p, s, copy)) {
            if (walk.ids.count == 0 || !walk.fresh)
                continue;
            ok = tile_wait(smem_u32(&bar_u_empty[u.at]), u.phase ^ 1u, abort_flag);
            if (!ok)
                break;
            const int64_t t = (int64_t)walk.tile * kM + r;
            const bool on = (warp == 4 ? walk.ids.id[0] : warp == 5 ? walk.ids.id[1] : warp == 6 ? walk.ids.id[2]
                                                                                               : walk.ids.id[3]) >= 0;
            const float *src = p.u + t * n + walk.slice * p.rank;
            for (int c = 0; c < chunks; ++c) {      // 8 elements of the rank, zeros from it on
                float4 x[kMaxSplits][2];
#pragma unroll
                for (int k = 0; k < kMaxSplits; ++k) {       // all loads before the first sum
                    x[k][0] = x[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (on && k < p.splits && 8 * c < p.rank) {
                        const float4 *q = reinterpret_cast<const float4 *>(src + (int64_t)k * p.num_tokens * n + 8 * c);
                        x[k][0] = q[0];
                        x[k][1] = q[1];
                    }
                }
                float v[8] = {};
#pragma unroll
                for (int k = 0; k < kMaxSplits; ++k) {
                    v[0] += x[k][0].x, v[1] += x[k][0].y, v[2] += x[k][0].z, v[3] += x[k][0].w;
                    v[4] += x[k][1].x, v[5] += x[k][1].y, v[6] += x[k][1].z, v[7] += x[k][1].w;
                }
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    adapter_split(v[2 * e], v[2 * e + 1], hi[e], lo[e]);
                const uint32_t off = swizzle<128>((uint32_t)r * 128u + (uint32_t)(c & 7) * 16u);
                const uint32_t dst = us + u.at * u_bytes + (uint32_t)(c >> 3) * kRowBlock + off;
                sts128(dst, hi[0], hi[1], hi[2], hi[3]);
                sts128(dst + (uint32_t)s.slabs * kRowBlock, lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_u[u.at]));
            u.next();
        }
        if (!ok)
            *abort_flag = 1;
    } else {
        // ---------------- the sums ----------------
        const int quarter = warp & 3, mine_row = quarter * 32 + lane;
        const uint32_t group = (uint32_t)(warp - 8) >> 2, acc0 = tmem + ((uint32_t)(quarter * 32) << 16);
        Ring row(RS), pair(kAccs);
        uint32_t turn = 0;
        bool ok = true;
        for (; ok && walk.next(p, s, copy); row.next(), turn = turn == kUpGroups - 1 ? 0 : turn + 1) {
            if (turn != group)
                continue;
            const int mine = quarter == 0   ? walk.ids.id[0]
                             : quarter == 1 ? walk.ids.id[1]
                             : quarter == 2 ? walk.ids.id[2]
                                            : walk.ids.id[3];
            const uint32_t at = rows + row.at * kRowBlock;
            ok = tile_wait(smem_u32(&bar_row[row.at]), row.phase, abort_flag) && walk.ids.each([&](int a) {
                const uint32_t acc = group * kAccs + pair.at;
                if (!tile_wait(smem_u32(&bar_acc[acc]), pair.phase, abort_flag))
                    return false;
                pair.next();
                const bool any = __any_sync(0xffffffffu, mine == a);
                if (any)
                    tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t v[32];
                    if (any) {
                        tmem_ld32(acc0 + acc * kBlockN + 32u * half, v);
                        tc_wait_ld();
                    }
                    if (half == 1) {
                        if (any)
                            tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_u32(&bar_acc_empty[acc]));
                    }
                    if (any && mine == a) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t cell = at + swizzle<128>((uint32_t)mine_row * 128u + (uint32_t)(64 * half + 16 * c));
                            const uint4 x = lds128(cell);
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                            uint32_t o[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[e] = adapter_bf16x2(__uint_as_float(w[e] << 16) + __uint_as_float(v[8 * c + 2 * e]),
                                                      __uint_as_float(w[e] & 0xFFFF0000u) + __uint_as_float(v[8 * c + 2 * e + 1]));
                            sts128(cell, o[0], o[1], o[2], o[3]);
                        }
                    }
                    __syncwarp();
                }
                return true;
            });
            if (!ok)
                break;
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_row_done[row.at]));
        }
        if (!ok)
            *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, kUpTmem);
    }
}

}  // namespace

bool adapter_down_tiles(const AdapterParams &p, bool pdl, cudaStream_t stream, cudaError_t *error)
{
    *error = cudaSuccess;
    const int rows = p.num_slices * p.rank;
    TileShape s;
    s.boxes = rows > 256 ? 2 : 1;
    s.n = (rows + 16 * s.boxes - 1) / (16 * s.boxes) * (16 * s.boxes);
    s.tmem = 32;
    while (s.tmem < s.n)
        s.tmem *= 2;
    s.stage_bytes = kTileX + (uint32_t)s.n * 128u;
    // two CTAs on an SM where at least three stages fit into half of its shared memory
    const uint32_t halfsm = 108 * 1024;
    s.stages = (int)((3 * s.stage_bytes <= halfsm ? halfsm : 2 * halfsm) / s.stage_bytes);
    if (s.stages > kMaxStages)
        s.stages = kMaxStages;
    const int64_t all = (int64_t)p.num_adapters * rows;
    const int64_t wdims[2] = {p.hidden_size, all}, wstride[1] = {2 * p.down_stride};
    const int64_t xdims[2] = {p.hidden_size, p.num_tokens}, xstride[1] = {2 * p.hidden_stride};
    const int32_t wbox[2] = {kBlockK, s.n / s.boxes}, xbox[2] = {kBlockK, kM};
    const int64_t limit = (int64_t)1 << 40;
    CUtensorMap xmap, wmap;
    memset(&xmap, 0, sizeof xmap);
    if (all >= 0x7fffffff || wstride[0] >= limit || (!p.fp8 && xstride[0] >= limit) ||
        !msa_internal_encode_tiled(&wmap, p.down, 2, 2, wdims, wstride, wbox, 128) ||
        (!p.fp8 && !msa_internal_encode_tiled(&xmap, p.hidden, 2, 2, xdims, xstride, xbox, 128)))
        return false;
    const void *fn = p.fp8 ? reinterpret_cast<const void *>(&msa_adapter_down_tile_kernel<true>)
                           : reinterpret_cast<const void *>(&msa_adapter_down_tile_kernel<false>);
    const int smem = s.stages * (int)s.stage_bytes + 1024;
    *error = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (*error != cudaSuccess)
        return true;
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    lc.gridDim = dim3((unsigned)((p.num_tokens + kM - 1) / kM), (unsigned)p.splits, 2);
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = (size_t)smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = pdl ? 1 : 0;
    AdapterParams params = p;
    void *args[] = {&params, &s, &xmap, &wmap};
    *error = cudaLaunchKernelExC(&lc, fn, args);
    return true;
}

bool adapter_up_tiles(const AdapterParams &p, cudaStream_t stream, cudaError_t *error)
{
    *error = cudaSuccess;
    UpShape s;
    s.slabs = p.rank > 64 ? 2 : 1;
    s.u_buffers = s.slabs == 1 ? 2 : 1;
    // a multiple of the groups, so that a stage is one group's and no wait on it comes a phase early
    s.row_stages = s.slabs == 1 ? kRing : kUpGroups;
    s.blocks = (p.width + kBlockN - 1) / kBlockN;
    const int64_t limit = (int64_t)1 << 40, all = (int64_t)p.num_adapters * p.width;
    const int64_t total = (p.num_tokens + kM - 1) / kM * s.blocks;
    const int64_t dims[2] = {p.width, p.num_tokens}, rstride[1] = {2 * p.rows_stride}, ostride[1] = {2 * p.out_stride};
    const int64_t udims[2] = {p.rank, all}, ustride[1] = {2 * p.rank};
    const int32_t box[2] = {kBlockN, kM}, ubox[2] = {64, kBlockN};
    CUtensorMap rmap, omap, umap;
    if (rstride[0] >= limit || ostride[0] >= limit || all >= 0x7fffffff || total >= 0x7fffffff ||
        !msa_internal_encode_tiled(&rmap, p.rows, 2, 2, dims, rstride, box, 128) ||
        !msa_internal_encode_tiled(&omap, p.out, 2, 2, dims, ostride, box, 128) ||
        !msa_internal_encode_tiled(&umap, p.up, 2, 2, udims, ustride, ubox, 128))
        return false;
    int dev = 0, sms = 0;
    if ((*error = cudaGetDevice(&dev)) != cudaSuccess ||
        (*error = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return true;
    s.ctas = (int)(total < sms ? total : sms);
    s.share = (int)(total / s.ctas);
    s.more = (int)(total % s.ctas);
    const int smem = s.row_stages * (int)kRowBlock + kRing * s.slabs * (int)kUpSlab +
                     s.u_buffers * 2 * s.slabs * (int)kRowBlock + 1024;
    const void *fn = reinterpret_cast<const void *>(&msa_adapter_up_tile_kernel);
    *error = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (*error != cudaSuccess)
        return true;
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    lc.gridDim = dim3((unsigned)s.ctas);
    lc.blockDim = dim3(kUpThreads);
    lc.dynamicSmemBytes = (size_t)smem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    AdapterParams params = p;
    void *args[] = {&params, &s, &rmap, &omap, &umap};
    *error = cudaLaunchKernelExC(&lc, fn, args);
    return true;
}
