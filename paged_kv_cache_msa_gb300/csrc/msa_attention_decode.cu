// Attention of single queries on the tcgen05 tensor cores, and the join of pieces.
//
// What is computed is stated in include/msa_attention.h.  Each query has its own list of
// visible tokens (the blocks selected for it, or its own history), each K/V head of which
// is read exactly once, so the kernel aims at the HBM roofline.
//
// The lists, cut into tiles of 128 tokens, are laid end to end over (query, K/V head,
// tile) and one persistent CTA per SM takes an equal share, so a batch of one query uses
// as many SMs as it has tiles.  Keys and values are the A operands of the MMAs, whose 128
// rows they fill whatever the number of query heads on a K/V head; the heads (8 or 16)
// are the columns:
//   S [token, head]  = K [128 tokens x D, K-major]  . Q^T [D x heads, K-major]
//   O [dim, head]    = V^T [D x 128 tokens, M-major] . P [128 tokens x heads, N-major]
// K and V tiles are multiplied as TMA copied them (128- or 64-byte swizzle).  E4M3 caches
// run on kind::f8f6f4 with Q and P split into E4M3 halves hi | lo side by side in the
// columns, so that a tile is still read once from shared memory; bf16 on kind::f16.
//
// Up to kChunk tiles of one (query, K/V head) form a chunk: all of their scores are held
// in tensor memory, so that the maximum is reduced over the 128 threads once a chunk, and
// their value products accumulate in one tensor-memory tile.  The key tiles of the next
// chunk are copied and multiplied before the value tiles of the current one, which keeps
// the copies going while the softmax runs.
//   warp 0    TMA: page lookups and tile copies into a ring of stages
//   warp 1    query tiles, one (query, K/V head) ahead
//   warp 2    MMAs; zeroes value rows past the history before they are multiplied
//   warps 4-7 softmax and output: a thread is a token of each tile, then a dim
// A (query, K/V head) that one CTA holds whole is written as bf16 right away; the pieces
// of one that is cut between CTAs (at most two a CTA) go to the workspace, and a second,
// dependent kernel joins them, together with the pieces of a shared prefix.

#include "msa_attention_internal.h"
#include "msa_tcgen05.cuh"

#include <cstring>

namespace {

constexpr int kThreads = 256;
constexpr int kInfo = 4;          // chunks whose box lists are held
constexpr int kQSlots = 3;
constexpr int kMaxBoxes = 16;     // boxes of a tile: 128 / 8 rows

template <int D, bool FP8, int NH>
struct Shape {
    static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
    static constexpr int kSwz = kRowBytes < 128 ? kRowBytes : 128;      // swizzle and TMA box width
    static constexpr int kAtoms = kRowBytes / kSwz;                      // boxes side by side in a row
    static constexpr int kTileBytes = 128 * kRowBytes;
    static constexpr int kN = FP8 ? 2 * NH : 16;                         // MMA columns: hi | lo, or at least 16
    static constexpr int kChunk = NH == 8 ? 8 : 4;                       // 64 scores a thread
    static constexpr int kPBytes = 128 * kN * (FP8 ? 1 : 2);             // weights of one tile
    static constexpr int kQBytes = kN * kRowBytes;
    static constexpr int kRest = 1024 + kChunk * kPBytes + kQSlots * kQBytes;
    static constexpr int kStages = (210 * 1024 - kRest) / kTileBytes;    // what the lists below leave of 227 KB
    static constexpr int kSmem = kRest + kStages * kTileBytes;
    static constexpr int kSCols = kChunk * kN;                           // columns of one chunk's scores
    static constexpr int kTmem = 512;
    static_assert(2 * kSCols + kN <= kTmem, "tensor memory");
    static_assert(kQBytes % 1024 == 0 && (kChunk * kPBytes) % 1024 == 0, "swizzle pattern alignment");
};

// A chunk: tiles [tile, tile + n) of (query q, head chunk hc), item `it` of the CTA's share.
struct Walk {
    const int64_t *pre;      // tiles before each query
    int64_t it, end;
    int nq, hcs, q, hc;
    int32_t nt, tile;        // tiles of the query; the chunk's first

    __device__ void start(const int64_t *pre_, int nq_, int hcs_, int64_t i0, int64_t i1, int q0)
    {
        pre = pre_; nq = nq_; hcs = hcs_; it = i0; end = i1; q = q0; hc = 0; nt = 0; tile = 0;
        if (it < end) {
            const int64_t base = pre[q] * hcs;
            nt = (int32_t)(pre[q + 1] - pre[q]);
            hc = (int)((it - base) / nt);
            tile = (int32_t)((it - base) - (int64_t)hc * nt);
        }
    }
    __device__ bool done() const { return it >= end; }
    __device__ int count(int chunk) const
    {
        const int64_t a = min((int64_t)(nt - tile), end - it);
        return (int)min((int64_t)chunk, a);
    }
    __device__ void step(int n)
    {
        it += n;
        tile += n;
        if (tile == nt) {
            tile = 0;
            if (++hc == hcs) {
                hc = 0;
                do
                    ++q;
                while (q < nq && pre[q + 1] == pre[q]);
                if (q < nq)
                    nt = (int32_t)(pre[q + 1] - pre[q]);
            }
        }
    }
};

// After the level with offset o a lane keeps the half of its values that bit o of its lane
// id selects, combined with its partner's: NH values over 32 lanes in 31 steps or fewer.
// Returns the result of head lane / (32 / NH).
template <int NH, bool MAX>
__device__ __forceinline__ float butterfly(const float (&in)[NH], int lane)
{
    float v[NH];
#pragma unroll
    for (int i = 0; i < NH; ++i)
        v[i] = in[i];
#pragma unroll
    for (int o = 16, n = NH; o >= 1; o >>= 1) {
        if (n > 1) {
            const bool hi = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < NH / 2; ++i)
                if (i < n / 2) {
                    const float send = hi ? v[i] : v[i + n / 2];
                    const float keep = hi ? v[i + n / 2] : v[i];
                    const float other = __shfl_xor_sync(0xffffffffu, send, o);
                    v[i] = MAX ? fmaxf(keep, other) : keep + other;
                }
            n /= 2;
        } else {
            const float other = __shfl_xor_sync(0xffffffffu, v[0], o);
            v[0] = MAX ? fmaxf(v[0], other) : v[0] + other;
        }
    }
    return v[0];
}

template <int D, bool FP8, int NH>
__global__ void __launch_bounds__(kThreads, 1)
msa_attention_decode_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnPieces w,
                            const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = Shape<D, FP8, NH>;
    constexpr int ST = S::kStages, N = S::kN, CH = S::kChunk;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[ST], bar_empty[ST];
    __shared__ __align__(8) uint64_t bar_info_full[kInfo], bar_info_empty[kInfo];
    __shared__ __align__(8) uint64_t bar_q_full[kQSlots], bar_q_empty[kQSlots];
    __shared__ __align__(8) uint64_t bar_s_full[2], bar_s_empty[2];
    __shared__ __align__(8) uint64_t bar_p_full, bar_o_full, bar_drain;
    __shared__ int64_t s_pre[kAttnWindow + 1];
    __shared__ int64_t s_toff[kAttnWindow];
    __shared__ int32_t s_len[kAttnWindow];
    __shared__ int64_t s_wsum[kThreads / 32];
    __shared__ int2 s_box[kInfo][CH][kMaxBoxes];       // row in the page, page
    __shared__ uint8_t s_nv[kInfo][CH][kMaxBoxes];     // visible rows of the box
    __shared__ int32_t s_list[64];                     // block ids of the loader's query
    __shared__ float s_qinv[kQSlots];
    __shared__ float s_red[4][16];
    __shared__ int s_qlo;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t pbase = ring + (uint32_t)(ST * S::kTileBytes);
    const uint32_t qbase = pbase + (uint32_t)(CH * S::kPBytes);
    volatile int *abort_flag = &s_abort;
    const int nq = (int)w.nq;

    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        for (int i = 0; i < ST; ++i) {
            mbar_init(smem_u32(&bar_full[i]), 1);
            mbar_init(smem_u32(&bar_empty[i]), 1);
        }
        for (int i = 0; i < kInfo; ++i) {
            mbar_init(smem_u32(&bar_info_full[i]), 1);
            mbar_init(smem_u32(&bar_info_empty[i]), 5);    // the MMA warp and the softmax warps
        }
        for (int i = 0; i < kQSlots; ++i) {
            mbar_init(smem_u32(&bar_q_full[i]), 1);
            mbar_init(smem_u32(&bar_q_empty[i]), 5);       // the MMAs and the softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar_s_full[i]), 1);
            mbar_init(smem_u32(&bar_s_empty[i]), 4);
        }
        mbar_init(smem_u32(&bar_p_full), 4);
        mbar_init(smem_u32(&bar_o_full), 1);
        mbar_init(smem_u32(&bar_drain), 1);
        s_abort = 0;
        s_qlo = 0;
        s_pre[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2)
        tmem_alloc(smem_u32(&s_tmem), S::kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);

    // tiles of each query, and their prefix sums: thread t holds queries 2t and 2t + 1
    constexpr int kPer = kAttnWindow / kThreads;
    int64_t mine[kPer], sum = 0;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        const int q = tid * kPer + r;
        int64_t nt = 0;
        if (q < nq) {
            const int32_t len = max(__ldg(p.kv_len + w.q0 + q), 0);
            s_len[q] = len;
            s_toff[q] = __ldg(p.table_offset + w.q0 + q);
            nt = ((int64_t)len + 127) / 128;
            if (p.topk_ids) {
                const int64_t nb = ((int64_t)len + p.block_tokens - 1) / p.block_tokens;
                const int32_t *ids = p.topk_ids + (w.q0 + q) * p.topk;
                int n = 0;
#pragma unroll 8
                for (int i = 0; i < p.topk; ++i) {
                    const int32_t id = __ldg(ids + i);
                    n += id >= 0 && id < nb;
                }
                nt = ((int64_t)n * p.block_tokens + 127) / 128;
            }
        }
        mine[r] = nt;
        sum += nt;
    }
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += x;
    }
    if (lane == 31)
        s_wsum[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    int64_t before = inc - sum, total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        before += i < warp ? s_wsum[i] : 0;
        total += s_wsum[i];
    }
    const int hcs = w.head_chunks;
    total *= hcs;
    const int64_t i0 = total * blockIdx.x / gridDim.x, i1 = total * (blockIdx.x + 1) / gridDim.x;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        const int q = tid * kPer + r;
        if (q < nq) {
            if (before * hcs <= i0 && i0 < (before + mine[r]) * hcs)
                s_qlo = q;
            before += mine[r];
            s_pre[q + 1] = before;
            if (blockIdx.x == 0)
                w.pre[q + 1] = before;
        }
    }
    if (blockIdx.x == 0 && tid == 0)
        w.pre[0] = 0;
    __syncthreads();
    Walk wk;
    wk.start(s_pre, nq, hcs, i0, i1, s_qlo);
    const int nchunk_heads = (p.group + NH - 1) / NH;      // head chunks of a K/V head

    if (warp == 0) {
        // ---------------- tile copies ----------------
        const int BR = w.box_rows, lb = __ffs(BR) - 1, nbox = 128 >> lb;
        uint32_t ring_it = 0, c = 0;
        int list_q = -1, cnt = 0;
        bool ok = true;
        // copies the tiles of the chunk in info slot `slot` into the ring
        auto copy = [&](const CUtensorMap *map, int slot, int n, int head) {
            for (int i = 0; i < n && ok; ++i, ++ring_it) {
                const uint32_t s = ring_it % ST, par = ((ring_it / ST) & 1u) ^ 1u;
                ok = warp_wait(smem_u32(&bar_empty[s]), par, abort_flag);
                if (!ok)
                    break;
                const uint32_t full = smem_u32(&bar_full[s]);
#ifndef MSA_STARVE
                if (lane == 0)
                    mbar_expect_tx(full, (uint32_t)S::kTileBytes);
                __syncwarp();
                if (lane < nbox * S::kAtoms) {
                    const int b = lane & (nbox - 1), at = lane / nbox;
                    const int2 box = s_box[slot][i][b];
                    tma_load_box(ring + s * (uint32_t)S::kTileBytes + (uint32_t)(at * 128 + b * BR) * S::kSwz, map,
                                 at * (S::kSwz / (FP8 ? 1 : 2)), box.x, head, box.y, full);
                }
#endif
            }
        };
        int pn = 0, phead = 0, pslot = 0;
        for (; !wk.done() && ok; ++c) {
            const int n = wk.count(CH), slot = (int)(c % kInfo);
            ok = warp_wait(smem_u32(&bar_info_empty[slot]), ((c / kInfo) & 1u) ^ 1u, abort_flag);
            if (!ok)
                break;
            const int64_t len = s_len[wk.q];
            if (p.topk_ids && list_q != wk.q) {
                // the ids that name a block, in order; a repeated one is kept as -1
                list_q = wk.q;
                const int64_t nb = (len + p.block_tokens - 1) / p.block_tokens;
                const int32_t *ids = p.topk_ids + (w.q0 + wk.q) * p.topk;
                const int32_t a0 = lane < p.topk ? __ldg(ids + lane) : -1;
                const int32_t a1 = lane + 32 < p.topk ? __ldg(ids + lane + 32) : -1;
                const bool v0 = a0 >= 0 && a0 < nb, v1 = a1 >= 0 && a1 < nb;
                const uint32_t m0 = __ballot_sync(0xffffffffu, v0), m1 = __ballot_sync(0xffffffffu, v1);
                const uint32_t below = (1u << lane) - 1u;
                const uint32_t same0 = __match_any_sync(0xffffffffu, v0 ? a0 : -1 - lane);
                const uint32_t same1 = __match_any_sync(0xffffffffu, v1 ? a1 : -1 - lane);
                bool dup0 = (same0 & below) != 0, dup1 = (same1 & below) != 0;
                if (m1)   // the second half against the first
                    for (int i = 0; i < 32; ++i)
                        dup1 |= __shfl_sync(0xffffffffu, a0, i) == a1;
                __syncwarp();
                if (v0)
                    s_list[__popc(m0 & below)] = dup0 ? -1 : a0;
                if (v1)
                    s_list[__popc(m0) + __popc(m1 & below)] = dup1 ? -1 : a1;
                cnt = __popc(m0) + __popc(m1);
                __syncwarp();
            }
            for (int x = lane; x < n * nbox; x += 32) {
                const int i = x / nbox, b = x & (nbox - 1);
                const int64_t v = (int64_t)(wk.tile + i) * 128 + b * BR;
                int64_t j = v;
                bool in = true;
                if (p.topk_ids) {
                    const int64_t k = v / p.block_tokens;
                    const int32_t id = k < cnt ? s_list[k] : -1;
                    in = id >= 0;
                    j = (int64_t)id * p.block_tokens + (v - k * p.block_tokens);
                }
                in = in && j < len;
                const int32_t pg = in ? attn_page(p, s_toff[wk.q], j) : -1;
                // a box that shows nothing is copied from past the last page: zeros
                s_box[slot][i][b] = pg >= 0 ? make_int2(attn_page_row(p, j), pg) : make_int2(0, w.oob_page);
                s_nv[slot][i][b] = (uint8_t)(pg >= 0 ? min((int64_t)BR, len - j) : 0);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_info_full[slot]));
            const int head = wk.hc / nchunk_heads;
            copy(&kmap, slot, n, head);
            if (c > 0)
                copy(&vmap, pslot, pn, phead);
            pn = n;
            phead = head;
            pslot = slot;
            wk.step(n);
        }
        if (ok && c > 0)
            copy(&vmap, pslot, pn, phead);
#ifndef MSA_STARVE
        // every copy has landed before the CTA finishes
        for (uint32_t s = 0; s < (uint32_t)ST && s < ring_it; ++s)
            (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_full[s]), ((ring_it - 1u - s) / ST) & 1u));
#endif
    } else if (warp == 1) {
        // ---------------- query tiles ----------------
        uint32_t seg = 0;
        bool ok = true;
        while (!wk.done() && ok) {
            const uint32_t x = seg % kQSlots;
            ok = warp_wait(smem_u32(&bar_q_empty[x]), ((seg / kQSlots) & 1u) ^ 1u, abort_flag);
            if (!ok)
                break;
            const int c = wk.hc / nchunk_heads, h0 = (wk.hc % nchunk_heads) * NH;
            const int nh = min(NH, p.group - h0);
            const uint16_t *src = p.q + ((w.q0 + wk.q) * p.hq + c * p.group + h0) * D;
            constexpr int E = D / 32;                       // elements of a lane
            uint32_t v[NH][E / 2];
            float amax = 0.0f;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    v[h][e] = h < nh ? __ldg(reinterpret_cast<const uint32_t *>(src + h * D) + lane * (E / 2) + e) : 0u;
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(v[h][e] << 16)),
                                             fabsf(__uint_as_float(v[h][e] & 0xFFFF0000u))));
                }
            const uint32_t tile = qbase + x * (uint32_t)S::kQBytes;
            if (FP8) {
                // halves hi | lo under the power of two that brings the largest magnitude
                // of the heads into [128, 256): hi has 4 significant bits, lo the next 4
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                int e2 = 0;
                if (amax > 0.0f) {
                    e2 = 7 - ((int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127);
                    e2 = e2 > 126 ? 126 : e2;
                }
                const float sc = __int_as_float((e2 + 127) << 23);
                const uint32_t byte = (uint32_t)lane * E;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    uint32_t hw = 0, lw = 0;
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const float x0 = __uint_as_float(v[h][e] << 16) * sc;
                        const float x1 = __uint_as_float(v[h][e] & 0xFFFF0000u) * sc;
                        const uint32_t hi = e4m3x2_from_f32(x0, x1);
                        const float2 d = attn_e4m3x2_to_f2(hi);
                        hw |= hi << (16 * e);
                        lw |= e4m3x2_from_f32(x0 - d.x, x1 - d.y) << (16 * e);
                    }
                    const uint32_t a = tile + swizzle<S::kSwz>((uint32_t)h * S::kSwz + byte);
                    const uint32_t b = tile + swizzle<S::kSwz>((uint32_t)(NH + h) * S::kSwz + byte);
                    if (E == 4) {
                        sts32(a, hw);
                        sts32(b, lw);
                    } else {
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"((unsigned short)hw) : "memory");
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(b), "h"((unsigned short)lw) : "memory");
                    }
                }
                if (lane == 0)
                    s_qinv[x] = __int_as_float((127 - e2) << 23);
            } else {
                const uint32_t byte = (uint32_t)lane * 2 * E, at = byte / S::kSwz, col = byte % S::kSwz;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const uint32_t a = tile + at * (uint32_t)(N * S::kSwz) + swizzle<S::kSwz>((uint32_t)h * S::kSwz + col);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e)
                        sts32(a + 4 * e, v[h][e]);
                }
                if (lane == 0)
                    s_qinv[x] = 1.0f;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_q_full[x]));
            // the rest of this (query, head chunk)
            wk.step((int)min((int64_t)(wk.nt - wk.tile), wk.end - wk.it));
            ++seg;
        }
    } else if (warp == 2) {
        // ---------------- MMAs ----------------
        constexpr uint32_t kIdS = mma_idesc(FP8, 128, N, false, false);
        constexpr uint32_t kIdO = mma_idesc(FP8, 128, N, true, true);
        constexpr int kKB = 32;                               // bytes of K a step takes of a K-major row
        constexpr int kTok = FP8 ? 32 : 16;                   // tokens of a step
        const int BR = w.box_rows, nbox = 128 / BR;
        const uint32_t o_tmem = tmem + 2 * S::kSCols;
        uint32_t ring_it = 0, c = 0, seg = 0;
        bool ok = true, fresh = true;
        auto values = [&](uint32_t cc, int n) {   // the value products of chunk cc
            ok = warp_wait(smem_u32(&bar_p_full), cc & 1u, abort_flag);
            tc_fence_after();
            const int slot = (int)(cc % kInfo);
            for (int i = 0; i < n && ok; ++i, ++ring_it) {
                const uint32_t s = ring_it % ST;
                ok = warp_wait(smem_u32(&bar_full[s]), (ring_it / ST) & 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t vt = ring + s * (uint32_t)S::kTileBytes;
                // rows past the history may hold anything: a weight of zero would not
                // hide an infinity or a NaN
                const int nv = lane < nbox ? s_nv[slot][i][lane] : 0;
                uint32_t partial = __ballot_sync(0xffffffffu, nv > 0 && nv < BR);
                if (partial) {
                    while (partial) {
                        const int b = __ffs(partial) - 1;
                        partial &= partial - 1;
                        const int r0 = b * BR + __shfl_sync(0xffffffffu, nv, b), r1 = (b + 1) * BR;
                        for (int at = 0; at < S::kAtoms; ++at)
                            for (int x = r0 * (S::kSwz / 16) + lane; x < r1 * (S::kSwz / 16); x += 32)
                                sts128(vt + (uint32_t)at * (128u * S::kSwz) + (uint32_t)x * 16u, 0u, 0u, 0u, 0u);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                const uint32_t pt = pbase + (uint32_t)(i * S::kPBytes);
#pragma unroll
                for (int ks = 0; ks < 128 / kTok; ++ks) {
                    // of 64 dims the 128 rows are the same 64 twice
                    const uint64_t a = smem_desc(vt + (uint32_t)(ks * kTok * S::kSwz), S::kSwz,
                                                 S::kAtoms == 2 ? 128u * S::kSwz : 0u, 8u * S::kSwz);
                    const uint64_t b = smem_desc(pt + (uint32_t)(ks * kTok * 16), 0, 128u, 2048u);
                    mma_ss<FP8>(o_tmem, a, b, kIdO, i > 0 || ks > 0);
                }
                mma_commit(smem_u32(&bar_empty[s]));
            }
            __syncwarp();
            if (ok) {
                mma_commit(smem_u32(&bar_o_full));
                if (lane == 0)
                    mbar_arrive(smem_u32(&bar_info_empty[slot]));
            }
        };
        int pn = 0;
        for (; !wk.done() && ok; ++c) {
            const int n = wk.count(CH);
            const uint32_t x = seg % kQSlots;
            if (fresh)
                ok = warp_wait(smem_u32(&bar_q_full[x]), (seg / kQSlots) & 1u, abort_flag);
            ok = ok && warp_wait(smem_u32(&bar_s_empty[c & 1]), ((c >> 1) & 1u) ^ 1u, abort_flag);
            // the chunk's box list, which the value products read
            ok = ok && warp_wait(smem_u32(&bar_info_full[c % kInfo]), (c / kInfo) & 1u, abort_flag);
            if (!ok)
                break;
            tc_fence_after();
            const uint32_t qt = qbase + x * (uint32_t)S::kQBytes;
            for (int i = 0; i < n; ++i, ++ring_it) {
                const uint32_t s = ring_it % ST;
                ok = warp_wait(smem_u32(&bar_full[s]), (ring_it / ST) & 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t kt = ring + s * (uint32_t)S::kTileBytes;
                const uint32_t d = tmem + (c & 1u) * S::kSCols + (uint32_t)(i * N);
#pragma unroll
                for (int ks = 0; ks < S::kRowBytes / kKB; ++ks) {
                    const uint32_t at = (uint32_t)(ks * kKB) / S::kSwz, col = (uint32_t)(ks * kKB) % S::kSwz;
                    mma_ss<FP8>(d, smem_desc(kt + at * (128u * S::kSwz) + col, S::kSwz, 16u, 8u * S::kSwz),
                                smem_desc(qt + at * (uint32_t)(N * S::kSwz) + col, S::kSwz, 16u, 8u * S::kSwz), kIdS, ks > 0);
                }
                mma_commit(smem_u32(&bar_empty[s]));
            }
            __syncwarp();
            if (!ok)
                break;
            mma_commit(smem_u32(&bar_s_full[c & 1]));
            fresh = wk.tile + n == wk.nt || wk.it + n == wk.end;
            if (fresh) {
                mma_commit(smem_u32(&bar_q_empty[x]));
                ++seg;
            }
            wk.step(n);
            if (c > 0)
                values(c - 1, pn);
            pn = n;
        }
        if (ok && c > 0)
            values(c - 1, pn);
        if (!ok)
            *abort_flag = 1;
        mma_commit(smem_u32(&bar_drain));   // every MMA has completed before tensor memory is released
        (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_drain), 0));
    } else if (warp >= 4) {
        // ---------------- softmax and output ----------------
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const int BR = w.box_rows, lb = __ffs(BR) - 1;
        const uint32_t o_tmem = tmem + lane_off + 2 * S::kSCols;
        constexpr float kPScale = FP8 ? 256.0f : 1.0f;   // E4M3 weights use the range up to 448
        float m[NH], l[NH], acc[NH];
        uint32_t c = 0, seg = 0;
        bool ok = true, first = true, pending = false;
        auto group_sync = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        auto add_output = [&](uint32_t cc) {   // adds the value products of chunk cc
            ok = ok && warp_wait(smem_u32(&bar_o_full), cc & 1u, abort_flag);
            if (ok) {
                tc_fence_after();
                uint32_t r[N];
                if (N == 16)
                    tmem_ld16(o_tmem, r);
                else
                    tmem_ld32(o_tmem, r);
                tc_wait_ld();
                tc_fence_before();
#pragma unroll
                for (int h = 0; h < NH; ++h)
                    acc[h] += FP8 ? __uint_as_float(r[h]) + __uint_as_float(r[NH + h]) : __uint_as_float(r[h]);
            }
        };
        for (; !wk.done(); ++c) {
            const int n = wk.count(CH), slot = (int)(c % kInfo);
            const uint32_t x = seg % kQSlots;
            const int hcol = wk.hc % nchunk_heads * NH, head = wk.hc / nchunk_heads;
            if (first) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    m[h] = -INFINITY;
                    l[h] = 0.0f;
                    acc[h] = 0.0f;
                }
                pending = false;
            }
            const bool last = wk.tile + n == wk.nt || wk.it + n == wk.end;
            ok = ok && warp_wait(smem_u32(&bar_info_full[slot]), (c / kInfo) & 1u, abort_flag);
            ok = ok && warp_wait(smem_u32(&bar_q_full[x]), (seg / kQSlots) & 1u, abort_flag);
            ok = ok && warp_wait(smem_u32(&bar_s_full[c & 1]), (c >> 1) & 1u, abort_flag);
            // all four warps go on or none does
            if (!ok)
                *abort_flag = 1;
            float s[CH][NH];
            uint32_t seen = 0;          // tiles whose row `row` is visible
            float mx[NH];
            if (ok) {
                tc_fence_after();
                const float qs = p.scale_log2 * attn_k_scale(p, head) * s_qinv[x];
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (i < n && (row & (BR - 1)) < s_nv[slot][i][row >> lb])
                        seen |= 1u << i;
#pragma unroll
                for (int i0c = 0; i0c < CH; i0c += 4) {
                    uint32_t r[4][N];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i0c + i < CH) {
                            const uint32_t a = tmem + lane_off + (c & 1u) * S::kSCols + (uint32_t)((i0c + i) * N);
                            if (N == 16)
                                tmem_ld16(a, r[i]);
                            else
                                tmem_ld32(a, r[i]);
                        }
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i0c + i < CH)
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                const float z = FP8 ? __uint_as_float(r[i][h]) + __uint_as_float(r[i][NH + h])
                                                    : __uint_as_float(r[i][h]);
                                s[i0c + i][h] = (seen >> (i0c + i)) & 1u ? z * qs : -INFINITY;
                            }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (ok && lane == 0) {
                mbar_arrive(smem_u32(&bar_s_empty[c & 1]));
                mbar_arrive(smem_u32(&bar_info_empty[slot]));
                if (last)
                    mbar_arrive(smem_u32(&bar_q_empty[x]));
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                mx[h] = -INFINITY;
                if (ok)
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        mx[h] = fmaxf(mx[h], s[i][h]);
            }
            const float wm = butterfly<NH, true>(mx, lane);
            if ((lane & (32 / NH - 1)) == 0)
                s_red[quarter][lane / (32 / NH)] = wm;
            group_sync();
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float cm = fmaxf(fmaxf(s_red[0][h], s_red[1][h]), fmaxf(s_red[2][h], s_red[3][h]));
                mx[h] = fmaxf(m[h], cm);
            }
            if (pending)
                add_output(c - 1);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float alpha = m[h] == mx[h] ? 1.0f : exp2_approx(m[h] - mx[h]);
                m[h] = mx[h];
                l[h] *= alpha;
                acc[h] *= alpha;
            }
            if (ok) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if (i >= n)
                        break;
                    float e[NH];
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        e[h] = (seen >> i) & 1u ? exp2_approx(s[i][h] - m[h]) : 0.0f;
                        l[h] += e[h];
                    }
                    const uint32_t a = pbase + (uint32_t)(i * S::kPBytes + row * 16);
                    if (FP8) {
                        uint32_t hw[NH / 4], lw[NH / 4];
#pragma unroll
                        for (int h = 0; h < NH; h += 4) {
                            const float x0 = e[h] * kPScale, x1 = e[h + 1] * kPScale, x2 = e[h + 2] * kPScale,
                                        x3 = e[h + 3] * kPScale;
                            const uint32_t h01 = e4m3x2_from_f32(x0, x1), h23 = e4m3x2_from_f32(x2, x3);
                            const float2 d01 = attn_e4m3x2_to_f2(h01), d23 = attn_e4m3x2_to_f2(h23);
                            hw[h / 4] = h01 | (h23 << 16);
                            lw[h / 4] = e4m3x2_from_f32(x0 - d01.x, x1 - d01.y) |
                                        (e4m3x2_from_f32(x2 - d23.x, x3 - d23.y) << 16);
                        }
                        if (NH == 8) {
                            sts128(a, hw[0], hw[1], lw[0], lw[1]);
                        } else {
                            sts128(a, hw[0], hw[1], hw[NH / 4 - 2], hw[NH / 4 - 1]);
                            sts128(a + 2048u, lw[0], lw[1], lw[NH / 4 - 2], lw[NH / 4 - 1]);
                        }
                    } else {
                        uint32_t b[NH / 2];
#pragma unroll
                        for (int h = 0; h < NH; h += 2)
                            b[h / 2] = bf16x2_from_f32(e[h], e[h + 1]);
                        sts128(a, b[0], b[1], b[2], b[3]);
                        if (NH == 16)
                            sts128(a + 2048u, b[NH / 2 - 4], b[NH / 2 - 3], b[NH / 2 - 2], b[NH / 2 - 1]);
                    }
                }
                tc_fence_before();
                fence_async_smem();
            }
            __syncwarp();
            if (ok && lane == 0)
                mbar_arrive(smem_u32(&bar_p_full));
            pending = true;
            if (last) {
                add_output(c);
                // the sum over the tokens; then a thread is a dim
                const float ws = butterfly<NH, false>(l, lane);
                group_sync();                    // s_red has been read
                if ((lane & (32 / NH - 1)) == 0)
                    s_red[quarter][lane / (32 / NH)] = ws;
                group_sync();
                // a wait of any warp that ran out spoils the whole (query, head chunk)
                const bool good = ok && *abort_flag == 0;
                const float bad = __int_as_float(0x7fc00000);
                const bool whole = wk.tile + n == wk.nt && wk.it + n - i0 >= wk.nt;
                const int nh = min(NH, p.group - hcol);
                const int64_t t = w.q0 + wk.q;
                const float vs = attn_v_scale(p, head);
                float *piece = nullptr;
                if (w.joined || !whole) {
                    const int64_t sl = whole ? 2 * (int64_t)gridDim.x + (int64_t)wk.q * hcs + wk.hc
                                       : wk.it + n - i0 < wk.tile + n ? (int64_t)blockIdx.x      // began in another CTA
                                                                      : (int64_t)gridDim.x + blockIdx.x;
                    piece = w.pieces + sl * (int64_t)(NH * (D + 2));
                }
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float sum = s_red[0][h] + s_red[1][h] + s_red[2][h] + s_red[3][h];
                    if (h < nh && row < D) {
                        const int64_t hr = t * p.hq + head * p.group + hcol + h;
                        if (piece) {
                            piece[h * D + row] = good ? acc[h] * (vs * (1.0f / kPScale)) : bad;
                            if (row == 0) {
                                piece[NH * D + h] = good ? m[h] : bad;
                                piece[NH * D + NH + h] = good ? sum : bad;
                            }
                        } else {
                            const float o = sum == 0.0f ? 0.0f : acc[h] * (vs * (1.0f / kPScale) / sum);
                            p.out[hr * D + row] = attn_bf16(good ? o : bad);
                            if (row == 0 && p.lse)
                                p.lse[hr] = good ? attn_lse(m[h], sum) : bad;
                        }
                    }
                }
                group_sync();                    // s_red is free again
                ++seg;
            }
            first = last;
            wk.step(n);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_free(tmem, S::kTmem);
    }
}

// ---------------------------------------------------------------------------
// the join: one warp per (query, query head)
// ---------------------------------------------------------------------------
//
// Adds the pieces of a (query, K/V head) that was cut between CTAs, those of its group's
// prefix, and writes the queries that see nothing.  The pieces lie in the workspace, most
// of them in L2.  A warp whose rows are already written leaves at once.
constexpr int kJoinWarps = 8;

// a / b for a >= 0, b > 0, in 32 bits where both fit
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b)
{
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
msa_attention_join_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnPieces w)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (r >= w.nq * p.hq)
        return;
    const int q = (int)(r / p.hq), h = (int)(r % p.hq);
    const int NH = w.heads;
    const int c = h / p.group, hg = h % p.group, nch = (p.group + NH - 1) / NH;
    const int hc = c * nch + hg / NH, col = hg % NH;
    constexpr int E = D / 32;
    float m = -INFINITY, l = 0.0f, acc[E] = {};
    auto add = [&](const float *o, float pm, float pl) {
        if (pl == 0.0f)                       // nothing seen (a NaN goes on)
            return;
        const float mn = isnan(pm) ? pm : fmaxf(m, pm);
        const float a = m == -INFINITY ? 0.0f : exp2f(m - mn), b = exp2f(pm - mn);
        l = l * a + pl * b;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = acc[e] * a + o[lane + 32 * e] * b;
        m = mn;
    };
    const int64_t nt = w.pre[q + 1] - w.pre[q];
    if (nt > 0) {
        const int64_t total = w.pre[w.nq] * w.head_chunks, n = w.ctas;
        const int64_t base = w.pre[q] * w.head_chunks + hc * nt;
        // CTA i holds items [total * i / n, total * (i + 1) / n), maybe none
        const int64_t c0 = div64((base + 1) * n - 1, total), c1 = div64((base + nt) * n - 1, total);
        if (c0 == c1 && !w.joined)
            return;
        const int64_t size = (int64_t)NH * (D + 2);
        for (int64_t i = c0;;) {
            const int64_t sl = i > c0 ? i : c0 == c1 ? 2 * n + (int64_t)q * w.head_chunks + hc : n + c0;
            const float *piece = w.pieces + sl * size;
            add(piece + col * D, piece[NH * D + col], piece[NH * D + NH + col]);
            if (i >= c1)
                break;
            i = div64((div64(total * (i + 1), n) + 1) * n - 1, total);   // the CTA of the next item
        }
    }
    const int64_t row = (w.q0 + q) * p.hq + h;
#pragma unroll
    for (int e = 0; e < E; ++e)
        p.out[row * D + lane + 32 * e] = attn_bf16(l == 0.0f ? 0.0f : acc[e] / l);
    if (lane == 0 && p.lse)
        p.lse[row] = attn_lse(m, l);
}

template <int D, bool FP8, int NH>
cudaError_t launch_decode(const AttnParams &p, const AttnPieces &w, const CUtensorMap &kmap, const CUtensorMap &vmap,
                          bool pdl, cudaStream_t stream)
{
    using S = Shape<D, FP8, NH>;
    const void *fn = reinterpret_cast<const void *>(&msa_attention_decode_kernel<D, FP8, NH>);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess)
        return e;
    void *args[] = {const_cast<AttnParams *>(&p), const_cast<AttnPieces *>(&w), const_cast<CUtensorMap *>(&kmap),
                    const_cast<CUtensorMap *>(&vmap)};
    return attn_launch(fn, w.ctas, kThreads, S::kSmem, pdl, stream, args);
}

}  // namespace

int attn_decode_heads(int group) { return group <= 8 ? 8 : 16; }

cudaError_t attn_decode(const AttnParams &p, const AttnPieces &w, int head_dim, const CUtensorMap &kmap,
                        const CUtensorMap &vmap, bool pdl, cudaStream_t stream)
{
    const bool f8 = p.k.fp8, h8 = w.heads == 8;
    if (head_dim == 128)
        return f8 ? (h8 ? launch_decode<128, true, 8>(p, w, kmap, vmap, pdl, stream)
                        : launch_decode<128, true, 16>(p, w, kmap, vmap, pdl, stream))
                  : (h8 ? launch_decode<128, false, 8>(p, w, kmap, vmap, pdl, stream)
                        : launch_decode<128, false, 16>(p, w, kmap, vmap, pdl, stream));
    return f8 ? (h8 ? launch_decode<64, true, 8>(p, w, kmap, vmap, pdl, stream)
                    : launch_decode<64, true, 16>(p, w, kmap, vmap, pdl, stream))
              : (h8 ? launch_decode<64, false, 8>(p, w, kmap, vmap, pdl, stream)
                    : launch_decode<64, false, 16>(p, w, kmap, vmap, pdl, stream));
}

cudaError_t attn_join(const AttnParams &p, const AttnPieces &w, int head_dim, cudaStream_t stream)
{
    void *args[] = {const_cast<AttnParams *>(&p), const_cast<AttnPieces *>(&w)};
    const int64_t grid = (w.nq * p.hq + kJoinWarps - 1) / kJoinWarps;
    return attn_launch(head_dim == 128 ? reinterpret_cast<const void *>(&msa_attention_join_kernel<128>)
                                       : reinterpret_cast<const void *>(&msa_attention_join_kernel<64>),
                       grid, kJoinWarps * 32, 0, true, stream, args);
}
