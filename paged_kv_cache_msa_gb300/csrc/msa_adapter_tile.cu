// The adapters' down-projection for large batches: tiles of 128 tokens on the tcgen05 tensor
// cores (include/msa_adapter.h).
//
// A CTA takes a tile of tokens of one adapter and a piece of K (and another, where there are more
// than CTAs); all of the adapter's num_slices * rank rows are the MMA's N, so that the hidden
// states are read once: 8,192 tokens of 6,144 E4M3 values are 50 MB, 7.5 us at the copy rate.
//   warp 0      copies: 64-element K blocks of the adapter's rows by TMA into a ring of stages,
//               128-byte rows in the 128-byte swizzle
//   warp 1      tensor-memory owner; issues the MMAs (M 128, N up to 2 x 256, K 16)
//   warps 2..9  hidden states (their tokens are in no order): loaded a few K blocks ahead into
//               registers, made bf16 where they are E4M3 (exact), stored in the swizzle; then the
//               accumulator, scaled, to the partial sums
// What bounds it: of 27 us for 8,192 E4M3 tokens of 160 rows (96 CTAs of 48 K blocks) 14 are starts and
// epilogues and 13.5 the K blocks, 0.28 us each, which stay with the hidden states' loads, their
// conversion or three quarters of the MMAs left out: by what is left over, the reads from L2, 94 MB
// of the adapter's rows for its tiles and 38 of hidden states, 9.8 TB/s.
// Every wait is bounded; rows that a CTA could not finish are NaN.  (MSA_GIVE_UP, a test build: the
// workers give up before their first wait, while copies land.)

#include "msa_adapter_internal.h"
#include "msa_tcgen05.cuh"

#include <cstring>

namespace {

constexpr int kM = 128;                       // tokens of a tile
constexpr int kBlockK = 64;                   // K elements of a stage: 128 bytes of bf16
constexpr int kMaxStages = 8;
constexpr int kWorkers = 8;                   // conversion and epilogue warps
constexpr int kThreads = 64 + 32 * kWorkers;
constexpr uint32_t kTileX = kM * 128;
constexpr uint32_t kHalfSm = 108 * 1024;      // shared memory of a CTA's ring, two on an SM; one has twice that
constexpr int kMaxSmem = 2 * kHalfSm + 1024;

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

// An MMA, and an arrival when all of this thread's are complete, by one thread; descriptors are
// made once and moved on by adding to them.
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

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// 16 bytes of a row from element k on, zeros from K on.
template <bool FP8>
__device__ __forceinline__ uint4 load_piece(const uint8_t *row, int k, int hidden)
{
    constexpr int es = FP8 ? 1 : 2;
    const int n = (hidden - k) * es;             // bytes
    if (n >= 16)
        return __ldg(reinterpret_cast<const uint4 *>(row + (int64_t)k * es));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (j < n)
            w[j / 4] |= (uint32_t)row[(int64_t)k * es + j] << (8 * (j & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads)
msa_adapter_down_tile_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ AdapterTileShape s,
                             const __grid_constant__ CUtensorMap wmap)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[kMaxStages], bar_empty[kMaxStages], bar_acc, bar_free, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    volatile int *abort_flag = &s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;

    if (tid == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(smem_u32(&bar_full[i]), 1 + kWorkers);
            mbar_init(smem_u32(&bar_empty[i]), 1);
        }
        mbar_init(smem_u32(&bar_acc), 1);
        mbar_init(smem_u32(&bar_free), kWorkers);
        mbar_init(smem_u32(&bar_drain), 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // Tensor memory is taken after the wait, so that the kernels ahead never wait for what this one
    // holds, and before the next kernel may start, so that this one never waits for what that holds.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int splits = p.head->splits, work = p.head->with_adapter * splits;
    if ((int)blockIdx.x >= work)
        return;
    if (warp == 1)
        tmem_alloc(smem_u32(&s_tmem), (uint32_t)s.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const uint32_t tmem = s_tmem;

    const int rows = p.num_slices * p.rank;
    const int blocks = (p.hidden_size + kBlockK - 1) / kBlockK;
    const uint32_t ST = (uint32_t)s.stages;
    // the K blocks of an item's piece
    auto first_block = [&](int split) { return (int)((int64_t)blocks * split / splits); };

    if (warp == 0) {
        // ---------------- copies ----------------
        Ring st(ST);
        uint32_t it = 0;
        bool ok = true;
        for (int item = blockIdx.x; ok && item < work; item += gridDim.x) {
            const int y = p.adapters[item / splits] * rows, k1 = first_block(item % splits + 1);
            for (int kb = first_block(item % splits); kb < k1; ++kb, ++it, st.next()) {
                const uint32_t full = smem_u32(&bar_full[st.at]);
                ok = tile_wait(smem_u32(&bar_empty[st.at]), st.phase ^ 1u, abort_flag);
                if (!ok)
                    break;
#ifndef MSA_STARVE
                if (lane == 0) {
                    const uint32_t w = ring + st.at * s.stage_bytes + kTileX;
                    mbar_expect_tx(full, (uint32_t)s.n * 128u);
                    for (int b = 0; b < s.boxes; ++b)
                        tma_load_2d(w + (uint32_t)(b * (s.n / s.boxes)) * 128u, &wmap, kb * kBlockK,
                                    y + b * (s.n / s.boxes), full);
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
        for (int item = blockIdx.x; ok && item < work; item += gridDim.x, ++done) {
            const int k0 = first_block(item % splits), k1 = first_block(item % splits + 1);
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
        // ---------------- hidden states and epilogue ----------------
        // A K block's pieces of 16 bytes: of E4M3 four a row, of bf16 eight; this thread's are those at
        // `col`, of row r0 and of rows kStep further.
        constexpr int kPerRow = FP8 ? 4 : 8, kStep = 32 * kWorkers / kPerRow, kPieces = kM / kStep, kAhead = FP8 ? 4 : 2;
        const int w = tid - 64, quarter = warp & 3, part = (warp - 2) >> 2;
        const int r0 = w / kPerRow, col = (w % kPerRow) * (kBlockK / kPerRow);
        Ring st(ST);
        uint32_t done = 0;
#ifdef MSA_GIVE_UP
        bool ok = false;
#else
        bool ok = true;
#endif
        for (int item = blockIdx.x; item < work; item += gridDim.x, ++done) {
            const int tile = item / splits, split = item % splits, k0 = first_block(split), k1 = first_block(split + 1);
            const int a = p.adapters[tile];
            const int32_t *tokens = p.tokens + (int64_t)tile * kM;
            const uint8_t *src[kPieces];
#pragma unroll
            for (int h = 0; h < kPieces; ++h) {
                const int t = tokens[r0 + kStep * h];
                src[h] = t >= 0 ? p.hidden + (int64_t)t * p.hidden_stride * (FP8 ? 1 : 2) : nullptr;
            }
            uint4 next[kAhead][kPieces];
#pragma unroll
            for (int d = 0; d < kAhead; ++d)
#pragma unroll
                for (int h = 0; h < kPieces; ++h)
                    next[d][h] = src[h] && k0 + d < k1 ? load_piece<FP8>(src[h], (k0 + d) * kBlockK + col, p.hidden_size)
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
                    for (int h = 0; h < kPieces; ++h) {
                        const uint4 c = next[d][h];
                        const uint32_t off = (uint32_t)(r0 + kStep * h) * 128u + 2u * (uint32_t)col;
                        if (FP8) {
                            sts128(x + swizzle<128>(off), adapter_e4m3x2(c.x & 0xffffu), adapter_e4m3x2(c.x >> 16),
                                   adapter_e4m3x2(c.y & 0xffffu), adapter_e4m3x2(c.y >> 16));
                            sts128(x + swizzle<128>(off + 16u), adapter_e4m3x2(c.z & 0xffffu), adapter_e4m3x2(c.z >> 16),
                                   adapter_e4m3x2(c.w & 0xffffu), adapter_e4m3x2(c.w >> 16));
                        } else {
                            sts128(x + swizzle<128>(off), c.x, c.y, c.z, c.w);
                        }
                        if (src[h] && kb + d + kAhead < k1)
                            next[d][h] = load_piece<FP8>(src[h], (kb + d + kAhead) * kBlockK + col, p.hidden_size);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bar_full[st.at]));
                    st.next();
                }
            }
            ok = ok && tile_wait(smem_u32(&bar_acc), done & 1u, abort_flag);
            const float scale = p.adapter_scales ? p.adapter_scales[a] : 1.0f;
            auto token_scale = [&](int t) { return t >= 0 && p.hidden_scales ? scale * p.hidden_scales[t] : scale; };
            const int mine = tokens[quarter * 32 + lane];
            const float c = token_scale(mine);
            if (ok)
                tc_fence_after();
            // Through the ring, which is free after the last item, so that four lanes write 64 bytes of
            // a row (each lane a row of its own: 7.5 us more of 32); rows 80 bytes apart lie on
            // different banks.  An earlier item writes its rows as they are, and so does one that a wait
            // ran out for: copies may still be landing in the ring.
            const bool last = ok && item + (int)gridDim.x >= work;
            const uint32_t buf = ring + (uint32_t)(warp - 2) * (32u * 80u);
            int out[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[j] = __shfl_sync(0xffffffffu, mine, 8 * j + (lane >> 2));
            for (int c0 = 16 * part; c0 < rows; c0 += 16 * (kWorkers / 4)) {
                uint32_t v[16];
                if (ok) {
                    tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c0, v);
                    tc_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[e] = ok ? __float_as_uint(c * __uint_as_float(v[e])) : 0x7fc00000u;
                if (last) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sts128(buf + (uint32_t)lane * 80u + 16u * j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = c0 + 4 * (lane & 3);
                        const uint4 x = lds128(buf + (uint32_t)(8 * j + (lane >> 2)) * 80u + 16u * (lane & 3));
                        if (out[j] >= 0 && at < rows)
                            *reinterpret_cast<uint4 *>(p.u + ((int64_t)split * p.num_tokens + out[j]) * rows + at) = x;
                    }
                } else if (mine >= 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c0 + 4 * j < rows)
                            *reinterpret_cast<uint4 *>(p.u + ((int64_t)split * p.num_tokens + mine) * rows + c0 + 4 * j) =
                                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
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

}  // namespace

cudaError_t adapter_tile_allow()
{
    for (const void *fn : {reinterpret_cast<const void *>(&msa_adapter_down_tile_kernel<true>),
                           reinterpret_cast<const void *>(&msa_adapter_down_tile_kernel<false>)}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

bool adapter_tile_plan(const AdapterParams &p, AdapterTilePlan *plan)
{
    const int rows = p.num_slices * p.rank;
    AdapterTileShape &s = plan->shape;
    s.boxes = rows > 256 ? 2 : 1;
    s.n = (rows + 16 * s.boxes - 1) / (16 * s.boxes) * (16 * s.boxes);
    s.tmem = 32;
    while (s.tmem < s.n)
        s.tmem *= 2;
    s.stage_bytes = kTileX + (uint32_t)s.n * 128u;
    // two CTAs on an SM where at least three stages fit into half of its shared memory
    s.stages = (int)((3 * s.stage_bytes <= kHalfSm ? kHalfSm : 2 * kHalfSm) / s.stage_bytes);
    if (s.stages > kMaxStages)
        s.stages = kMaxStages;
    const int64_t wdims[2] = {p.hidden_size, (int64_t)p.num_adapters * rows}, wstride[1] = {2 * p.down_stride};
    const int32_t wbox[2] = {kBlockK, s.n / s.boxes};
    return msa_internal_encode_tiled(&plan->down, p.down, 2, 2, wdims, wstride, wbox, 128);
}

cudaError_t adapter_tile_launch(const AdapterParams &p, const AdapterTilePlan &plan, int64_t tiles, cudaStream_t stream)
{
    const AdapterTileShape &s = plan.shape;
    const void *fn = p.fp8 ? reinterpret_cast<const void *>(&msa_adapter_down_tile_kernel<true>)
                           : reinterpret_cast<const void *>(&msa_adapter_down_tile_kernel<false>);
    const int64_t work = tiles * p.max_splits, fill = 3 * s.stage_bytes <= kHalfSm ? 2 * 152 : 152;
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof lc);
    lc.gridDim = dim3((unsigned)(work < fill ? work : fill));
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = (size_t)s.stages * s.stage_bytes + 1024;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    void *args[] = {const_cast<AdapterParams *>(&p), const_cast<AdapterTileShape *>(&s), const_cast<CUtensorMap *>(&plan.down)};
    return cudaLaunchKernelExC(&lc, fn, args);
}
