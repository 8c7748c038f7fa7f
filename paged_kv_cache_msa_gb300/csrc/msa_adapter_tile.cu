// The adapters' down-projection for large batches: tiles of 128 tokens on the tcgen05 tensor
// cores (include/msa_adapter.h).
//
// A CTA takes 128 consecutive tokens, a piece of K, and every second distinct adapter of the tile
// (a prefill chunk has one, two at its border); all of an adapter's num_slices * rank rows are
// the MMA's N, so that the hidden states are read once, which is what bounds the kernel: 8,192
// tokens of 6,144 E4M3 values are 50 MB, 7.5 us at the copy rate.
//   warp 0      copies: 64-element K blocks of the adapter's rows (and of bf16 hidden states) by
//               TMA into a ring of stages, 128-byte rows in the 128-byte swizzle
//   warp 1      tensor-memory owner; issues the MMAs (M 128, N up to 2 x 256, K 16)
//   warps 2..9  E4M3 hidden states: loaded a few K blocks ahead into registers, made bf16 (exact)
//               and stored in the swizzle; then the accumulator, scaled, to the partial sums
// A token of another adapter has a row of its own in the MMA, which is not written.
// Every wait is bounded; rows that a CTA could not finish are NaN.

#include "msa_adapter_internal.h"
#include "msa_tcgen05.cuh"

#include <cstring>

namespace {

constexpr int kM = 128;                       // tokens of a tile
constexpr int kBlockK = 64;                   // K elements of a stage: 128 bytes of bf16
constexpr int kMaxStages = 8;
constexpr int kWorkers = 8;                   // conversion and epilogue warps
constexpr int kPieces = 4 * kM / (32 * kWorkers);   // pieces of 16 codes of a K block a thread has
constexpr int kThreads = 64 + 32 * kWorkers;
constexpr int kAhead = 4;                     // K blocks of E4M3 values loaded ahead
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
                // this thread's pieces of 16 codes: of row w / 4, and of rows that many further
                const int col = 16 * (w & 3);
                const uint8_t *src[kPieces];
#pragma unroll
                for (int h = 0; h < kPieces; ++h) {
                    const int r = (w >> 2) + 8 * kWorkers * h;
                    src[h] = s_id[r] == a ? p.hidden + (t0 + r) * p.hidden_stride : nullptr;
                }
                uint4 next[kAhead][kPieces];
#pragma unroll
                for (int d = 0; d < kAhead; ++d)
#pragma unroll
                    for (int h = 0; h < kPieces; ++h)
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
                        for (int h = 0; h < kPieces; ++h) {
                            const uint4 c = next[d][h];
                            const uint32_t off = (uint32_t)((w >> 2) + 8 * kWorkers * h) * 128u + 2u * (uint32_t)col;
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
            // Through the ring, which is free after the last pass, so that four lanes write 64
            // bytes of a row (each lane a row of its own: 7.5 us more of 32); rows 80 bytes apart lie
            // on different banks.  An earlier pass, of a tile of many adapters, writes its rows as
            // they are.
            const bool last = pass + pass_step >= count;
            const uint32_t buf = ring + (uint32_t)(warp - 2) * (32u * 80u);
            for (int col = 16 * part; col < rows; col += 16 * (kWorkers / 4)) {
                uint32_t v[16];
                if (ok) {
                    tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)col, v);
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
                        const int r = quarter * 32 + 8 * j + (lane >> 2), at = col + 4 * (lane & 3);
                        const uint4 x = lds128(buf + (uint32_t)(8 * j + (lane >> 2)) * 80u + 16u * (lane & 3));
                        if (s_id[r] == a && at < rows)
                            *reinterpret_cast<uint4 *>(p.u + ((int64_t)blockIdx.y * p.num_tokens + t0 + r) * rows + at) = x;
                    }
                } else if (mine) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (col + 4 * j < rows)
                            *reinterpret_cast<uint4 *>(dst + col + 4 * j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
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

bool adapter_down_tiles(const AdapterParams &p, cudaStream_t stream, cudaError_t *error)
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
    lc.numAttrs = 1;
    AdapterParams params = p;
    void *args[] = {&params, &s, &xmap, &wmap};
    *error = cudaLaunchKernelExC(&lc, fn, args);
    return true;
}
