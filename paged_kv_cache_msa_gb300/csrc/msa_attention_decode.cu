// Attention of single queries on the tcgen05 tensor cores, and the join of pieces.
//
// What is computed is stated in include/msa_attention.h.  Each query has its own list of
// visible tokens (the blocks selected for it, or its own history), each K/V head of which
// is read exactly once, so the kernel aims at the HBM roofline.
//
// The lists, cut into tiles of 128 tokens, are laid end to end over (query, K/V head,
// tile) and one persistent CTA per SM takes an equal share, so a batch of one query uses
// as many SMs as it has tiles.  Keys and values are the A operands of the MMAs, whose 128
// rows they fill whatever the number of query heads on a K/V head; the heads (8, or 16 of
// bf16 caches) are the columns:
//   S [token, head]  = K [128 tokens x D, K-major]  . Q^T [D x heads, K-major]
//   O [dim, head]    = V^T [D x 128 tokens, M-major] . P [128 tokens x heads, N-major]
// K and V tiles are multiplied as TMA copied them (128- or 64-byte swizzle).  E4M3 caches
// run on kind::f8f6f4 with Q split into E4M3 halves and P into three E5M2 parts side by side
// in the columns, so that a tile is still read once from shared memory; bf16 on kind::f16.
//
// Up to kChunk tiles of one (query, K/V head) form a chunk, whose scores are held in
// tensor memory together, so that the maximum is reduced over the 128 threads once a
// chunk, and whose value products accumulate in one tensor-memory tile.  Keys are
// copied and multiplied ahead of the values, and successive (query, K/V head)s go to
// kGroups softmax groups in turn, so that neither the copies nor the MMAs wait for one
// softmax: short histories make chunks of one tile, whose
// softmax (about 1 us of latency) is longer than their copies (0.7 us).
//   warps 0, 1 TMA: key tiles, value tiles, each into a ring of stages
//   warps 2, 3 MMAs of the scores, of the values (one MMA costs its warp about 85 cycles of
//              issue, a tile 8 of them, close to the tile's share of HBM time: two warps);
//              warp 3 zeroes value rows past the history before they are multiplied
//   warp 4     block lists and page lookups
//   warps 5-7  query tiles, in turn, ahead of their use; queries that see nothing
//   warps 8-15 two softmax and output groups: a thread is a token of each tile, then a dim
// Measured: 64 queries, 16 blocks of 128 tokens (64 heads on 8 of 128 dims, E4M3, 233 MB)
// 52 us, 4.5 TB/s, 0.66 of the copy rate; one query 13.3 us and 256 short ones 19.6 us,
// bound by latency: 4.9 us from the dependency wait to the first scores (instructions
// fetched for the first time, length -> ids -> page -> keys), the softmax of a chunk, the
// join's launch.  256 bf16 queries of 32 heads on 2 (524 MB): 94 us, 0.82 of the copy rate.
// A (query, K/V head) that one CTA holds whole is written as bf16 right away; the pieces
// of one that is cut between CTAs (at most two a CTA) go to the workspace, and a second,
// dependent kernel joins them.

#include "msa_attention_internal.h"
#include "msa_tcgen05.cuh"

#include <cfloat>
#include <cstring>
#include <type_traits>

namespace {

constexpr int kGroups = 2;        // softmax groups
constexpr int kThreads = 256 + 128 * kGroups;
// Score buffers and box lists belong to a group, in turn: a group that waits on a barrier
// has then waited on every phase before, as waiting by parity needs.
constexpr int kGroupBufs = 3, kSBufs = kGroups * kGroupBufs;
constexpr int kGroupInfo = 4, kInfo = kGroups * kGroupInfo;
constexpr int kBuilders = 3;      // warps that make query tiles, in turn
constexpr int kQSlots = 6;        // a multiple of the groups and builders: a slot belongs to one of each
constexpr int kSmallIds = 1024;   // ids of a window kept in shared memory
constexpr int kMaxBoxes = 16;     // boxes of a tile: 128 / 8 rows

template <int D, bool FP8, int NH>
struct Shape {
    static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
    static constexpr int kSwz = kRowBytes < 128 ? kRowBytes : 128;      // swizzle and TMA box width
    static constexpr int kAtoms = kRowBytes / kSwz;                      // boxes side by side in a row
    static constexpr int kTileBytes = 128 * kRowBytes;
    static_assert(NH == 8 || (NH == 16 && !FP8), "heads of a chunk");
    static constexpr int kN = 16;                                        // score columns: hi | lo, or 8 or 16 heads
    static constexpr int kNO = FP8 ? 32 : 16;                            // output columns: three parts of 8, or heads
    static constexpr int kChunk = 4;                                     // 64 columns of scores
    // Weights of one tile: [token][16 bytes] pieces of the columns.  bf16 weights of 8 heads
    // are the first piece alone, taken twice for the 16 columns.
    static constexpr int kPBytes = 128 * (FP8 ? kNO : NH * 2);
    static constexpr int kQBytes = kN * kRowBytes;
    static constexpr int kRest = 1024 + kGroups * kChunk * kPBytes + kQSlots * kQBytes;
    // of each ring, in what the lists (20 KB) leave of 227 KB
    static constexpr int kStages = (207 * 1024 - kRest) / kTileBytes / 2;
    static constexpr int kSmem = kRest + 2 * kStages * kTileBytes;
    static constexpr int kSCols = kChunk * kN;                           // columns of one chunk's scores
    static constexpr int kTmem = 512;
    static_assert(kSBufs * kSCols + kGroups * kNO <= kTmem, "tensor memory");
    static_assert(kQSlots % kGroups == 0 && kQSlots % kBuilders == 0, "slots");
    static_assert(kQBytes % 1024 == 0 && (kChunk * kPBytes) % 1024 == 0, "swizzle pattern alignment");
};

__device__ __noinline__ int64_t div_slow(int64_t a, int64_t b) { return a / b; }

// a / b for a >= 0, b > 0, in 32 bits where both fit
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b)
{
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : div_slow(a, b);
}

// A chunk: tiles [tile, tile + n) of (query q, head chunk hc), item `it` of the CTA's share.
// A (query, head chunk) has `segment` items without a tile, then its tiles.
struct Walk {
    const int64_t *pre;      // items of a head chunk before each query
    int64_t it, end;
    int nq, hcs, q, hc;
    int32_t segment, nt, tile;     // nt: tiles of the query; the chunk's first

    __device__ void start(const int64_t *pre_, int nq_, int hcs_, int32_t segment_, int64_t i0, int64_t i1, int q0)
    {
        pre = pre_; nq = nq_; hcs = hcs_; segment = segment_; it = i0; end = i1; q = q0; hc = 0; nt = 0; tile = 0;
        if (it < end) {
            const int64_t base = pre[q] * hcs, items = pre[q + 1] - pre[q];
            nt = (int32_t)items - segment;
            hc = (int)div64(it - base, items);
            tile = max((int32_t)((it - base) - hc * items) - segment, 0);
            it = base + hc * items + segment + tile;
        }
    }
    __device__ bool done() const { return it >= end; }
    __device__ int count(int chunk) const
    {
        const int64_t a = min((int64_t)(nt - tile), end - it);
        return (int)min((int64_t)chunk, a);
    }
    __device__ bool last(int n) const { return tile + n == nt || it + n == end; }   // of its segment
    __device__ void step(int n)
    {
        it += n;
        tile += n;
        if (tile == nt) {
            tile = 0;
            it += segment;
            if (++hc == hcs) {
                hc = 0;
                do
                    ++q;
                while (q < nq && pre[q + 1] == pre[q]);
                if (q < nq)
                    nt = (int32_t)(pre[q + 1] - pre[q]) - segment;
            }
        }
    }
};

// The group of each segment and, in it, the number of the chunk: every role counts alike.
struct Turn {
    uint32_t seg = 0, count[kGroups] = {};

    __device__ int group() const { return (int)(seg % kGroups); }
    __device__ uint32_t chunk() const
    {
        uint32_t k = count[0];
#pragma unroll
        for (int i = 1; i < kGroups; ++i)
            k = group() == i ? count[i] : k;
        return k;
    }
    __device__ int info() const { return group() * kGroupInfo + (int)(chunk() % kGroupInfo); }
    __device__ uint32_t info_phase() const { return (chunk() / kGroupInfo) & 1u; }
    __device__ int buf() const { return group() * kGroupBufs + (int)(chunk() % kGroupBufs); }
    __device__ uint32_t buf_phase() const { return (chunk() / kGroupBufs) & 1u; }
    __device__ void step(bool last)
    {
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
            count[i] += group() == i;
        seg += last;
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
    constexpr int ST = S::kStages, N = S::kN, NO = S::kNO, CH = S::kChunk;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_k_full[ST], bar_k_empty[ST], bar_v_full[ST], bar_v_empty[ST];
    __shared__ __align__(8) uint64_t bar_info_full[kInfo], bar_info_empty[kInfo];
    __shared__ __align__(8) uint64_t bar_q_full[kQSlots], bar_q_empty[kQSlots];
    __shared__ __align__(8) uint64_t bar_s_full[kSBufs], bar_s_empty[kSBufs];
    __shared__ __align__(8) uint64_t bar_p_full[kGroups], bar_o_full[kGroups], bar_drain;
    __shared__ int64_t s_pre[kAttnWindow + 1];
    __shared__ int64_t s_toff[kAttnWindow];
    __shared__ int32_t s_len[kAttnWindow];
    __shared__ int32_t s_cnt[kAttnWindow];             // ids that name a block
    __shared__ int32_t s_ids[kSmallIds];               // of a small batch
    __shared__ int64_t s_wsum[kThreads / 32];
    __shared__ int2 s_box[kInfo][CH][kMaxBoxes];       // row in the page, page
    __shared__ uint8_t s_nv[kInfo][CH][kMaxBoxes];     // visible rows of the box
    __shared__ int32_t s_list[64];                     // block ids of the list warp's query
    __shared__ __align__(16) float s_qscale[kQSlots][FP8 ? NH : 4];  // of each head's scores (bf16: the first)
    __shared__ float s_red[kGroups][2][4][16];         // by turns: see group_reduce
    __shared__ int s_qlo;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t pbase = ring + (uint32_t)(2 * ST * S::kTileBytes);     // key stages, value stages
    const uint32_t qbase = pbase + (uint32_t)(kGroups * CH * S::kPBytes);
    volatile int *abort_flag = &s_abort;
    const int nq = (int)w.nq;

    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        for (int i = 0; i < ST; ++i) {
            mbar_init(smem_u32(&bar_k_full[i]), 1);
            mbar_init(smem_u32(&bar_k_empty[i]), 1);
            mbar_init(smem_u32(&bar_v_full[i]), 1);
            mbar_init(smem_u32(&bar_v_empty[i]), 1);
        }
        for (int i = 0; i < kInfo; ++i) {
            mbar_init(smem_u32(&bar_info_full[i]), 1);
            mbar_init(smem_u32(&bar_info_empty[i]), 7);    // the copy warps, the value MMAs, a group
        }
        for (int i = 0; i < kQSlots; ++i) {
            mbar_init(smem_u32(&bar_q_full[i]), 1);
            mbar_init(smem_u32(&bar_q_empty[i]), 5);       // the MMAs and a softmax group
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(smem_u32(&bar_s_full[i]), 1);
            mbar_init(smem_u32(&bar_s_empty[i]), 4);
        }
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(smem_u32(&bar_p_full[i]), 4);
            mbar_init(smem_u32(&bar_o_full[i]), 1);
        }
        mbar_init(smem_u32(&bar_drain), 2);
        s_abort = 0;
        s_qlo = 0;
        s_pre[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2)
        tmem_alloc(smem_u32(&s_tmem), S::kTmem);
    // Behind a shared prefix the kernel ahead is the tile kernel, which waited for all before
    // it and whose pieces are not read here: this one may run beside it, and waits for it
    // only at the end, so that the join comes after both.
    if (!w.joined)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);

    // Items of a head chunk of each query and their prefix sums, a query a thread.  Lengths, table offsets
    // and the first ids are read in one round of loads; the ids of small batches stay in
    // shared memory for the lists.
    static_assert(kAttnWindow <= kThreads, "a thread holds one query");
    constexpr int kBatch = 4;
    const int ids = p.topk_ids ? nq * p.topk : 0;
    const int32_t *src = p.topk_ids + w.q0 * p.topk;
    int32_t len = tid < nq ? __ldg(p.kv_len + w.q0 + tid) : 0;
    const int64_t toff = tid < nq ? __ldg(p.table_offset + w.q0 + tid) : 0;
    for (int x0 = 0; x0 == 0 || x0 < ids; x0 += kBatch * kThreads) {
        int32_t id[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int x = x0 + i * kThreads + tid;
            id[i] = x < ids ? __ldg(src + x) : -1;
        }
        if (x0 == 0) {
            len = attn_len(p, len, toff);
            if (tid < nq) {
                s_toff[tid] = toff;
                s_len[tid] = len;
                s_cnt[tid] = 0;
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int x = x0 + i * kThreads + tid;
            if (x < kSmallIds && x < ids)
                s_ids[x] = id[i];
            if (id[i] >= 0) {
                const int q = (int)((uint32_t)x / (uint32_t)p.topk);
                // the id names a block when the block's first token is visible
                if ((int64_t)id[i] * p.block_tokens < s_len[q])
                    atomicAdd(&s_cnt[q], 1);
            }
        }
    }
    if (ids > 0)
        __syncthreads();
    int64_t sum = 0;
    if (tid < nq)
        sum = p.topk_ids ? (s_cnt[tid] * p.block_tokens + 127) / 128 : ((int64_t)len + 127) / 128;
    sum += sum > 0 ? w.segment : 0;
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
    int64_t before = inc - sum, items = 0;
    for (int i = 0; i < (nq + 31) / 32; ++i) {
        before += i < warp ? s_wsum[i] : 0;
        items += s_wsum[i];
    }
    // equal shares, the last ones shorter or empty
    const int hcs = w.head_chunks;
    const int64_t total = items * hcs, share = div64(total + gridDim.x - 1, gridDim.x);
    const int64_t i0 = min(total, share * blockIdx.x), i1 = min(total, i0 + share);
    if (tid < nq) {
        if (before * hcs <= i0 && i0 < (before + sum) * hcs)
            s_qlo = tid;
        s_pre[tid + 1] = before + sum;
        if (blockIdx.x == 0 && w.joined)
            w.pre[tid + 1] = before + sum;
    }
    if (tid == 0) {
        if (blockIdx.x == 0 && w.joined)
            w.pre[0] = 0;
        w.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    Walk wk;
    wk.start(s_pre, nq, hcs, w.segment, i0, i1, s_qlo);
    const int nchunk_heads = (p.group + NH - 1) / NH;      // head chunks of a K/V head

    if (warp < 2) {
        // ---------------- tile copies: warp 0 keys, warp 1 values ----------------
        const int BR = w.box_rows, lb = __ffs(BR) - 1, nbox = 128 >> lb;
        const CUtensorMap *map = warp == 0 ? &kmap : &vmap;
        uint64_t *full_bars = warp == 0 ? bar_k_full : bar_v_full, *empty_bars = warp == 0 ? bar_k_empty : bar_v_empty;
        const uint32_t stages = ring + (uint32_t)(warp * ST * S::kTileBytes);
        uint32_t it = 0;
        Turn turn;
        bool ok = true;
        while (!wk.done() && ok) {
            const int n = wk.count(CH), slot = turn.info(), head = wk.hc / nchunk_heads;
            ok = warp_wait(smem_u32(&bar_info_full[slot]), turn.info_phase(), abort_flag);
            for (int i = 0; i < n && ok; ++i, ++it) {
                const uint32_t s = it % ST;
                ok = warp_wait(smem_u32(&empty_bars[s]), ((it / ST) & 1u) ^ 1u, abort_flag);
                if (!ok)
                    break;
#ifndef MSA_STARVE
                const uint32_t full = smem_u32(&full_bars[s]);
                if (lane == 0)
                    mbar_expect_tx(full, (uint32_t)S::kTileBytes);
                __syncwarp();
                if (lane < nbox * S::kAtoms) {
                    const int b = lane & (nbox - 1), at = lane >> (7 - lb);
                    const int2 box = s_box[slot][i][b];
                    tma_load_box(stages + s * (uint32_t)S::kTileBytes + (uint32_t)(at * 128 + b * BR) * S::kSwz, map,
                                 at * (S::kSwz / (FP8 ? 1 : 2)), box.x, head, box.y, full);
                }
#endif
            }
            __syncwarp();
            if (ok && lane == 0)
                mbar_arrive(smem_u32(&bar_info_empty[slot]));
            turn.step(wk.last(n));
            wk.step(n);
        }
#ifndef MSA_STARVE
        // every copy has landed before the CTA finishes
        for (uint32_t s = 0; s < (uint32_t)ST && s < it; ++s)
            (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&full_bars[s]), ((it - 1u - s) / ST) & 1u));
#endif
    } else if (warp >= 5 && warp < 5 + kBuilders) {
        // ---------------- query tiles: warp 5 + b the segments s with s % kBuilders == b ----------------
        uint32_t seg = 0;
        bool ok = true;
        while (!wk.done() && ok) {
            const uint32_t x = seg % kQSlots;
            if ((int)(seg % kBuilders) != warp - 5) {
                wk.step((int)min((int64_t)(wk.nt - wk.tile), wk.end - wk.it));
                ++seg;
                continue;
            }
            ok = warp_wait(smem_u32(&bar_q_empty[x]), ((seg / kQSlots) & 1u) ^ 1u, abort_flag);
            if (!ok)
                break;
            const int c = wk.hc / nchunk_heads, h0 = (wk.hc % nchunk_heads) * NH;
            const int nh = min(NH, p.group - h0);
            const uint16_t *src = p.q + ((w.q0 + wk.q) * p.hq + c * p.group + h0) * D;
            const float ks = attn_k_scale(p, c) * p.scale_log2;
            constexpr int E = D / 32;                       // elements of a lane
            auto load = [&](int h, uint32_t (&v)[E / 2]) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    v[e] = h < nh ? __ldg(reinterpret_cast<const uint32_t *>(src + h * D) + lane * (E / 2) + e) : 0u;
            };
            const uint32_t tile = qbase + x * (uint32_t)S::kQBytes;
            if (FP8) {
                // halves hi | lo under the power of two that brings the head's largest
                // magnitude into [128, 256): hi has 4 significant bits, lo the next 4
#pragma unroll 4
                for (int h = 0; h < NH; ++h) {
                    uint32_t v[E / 2], big = 0, hw = 0, lw = 0;
                    load(h, v);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e)         // magnitudes compare as integers
                        big = max(big, max((v[e] & 0x7FFFu) << 16, v[e] & 0x7FFF0000u));
                    big = __reduce_max_sync(0xffffffffu, big) >> 23;
                    const int e2 = big > 0 ? min(7 - ((int)big - 127), 126) : 0;
                    const float sc = __int_as_float((e2 + 127) << 23);
                    if (lane == 0)      // an infinity would saturate: no score of such a head is a number
                        s_qscale[x][h] = big == 255 ? __int_as_float(0x7fc00000) : ks * __int_as_float((127 - e2) << 23);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const float x0 = __uint_as_float(v[e] << 16) * sc, x1 = __uint_as_float(v[e] & 0xFFFF0000u) * sc;
                        const uint32_t hi = e4m3x2_from_f32(x0, x1);
                        const float2 d = attn_e4m3x2_to_f2(hi);
                        hw |= hi << (16 * e);
                        lw |= e4m3x2_from_f32(x0 - d.x, x1 - d.y) << (16 * e);
                    }
                    const uint32_t a = tile + swizzle<S::kSwz>((uint32_t)(h * S::kSwz + lane * E));
                    const uint32_t b = tile + swizzle<S::kSwz>((uint32_t)((NH + h) * S::kSwz + lane * E));
                    if (E == 4) {
                        sts32(a, hw);
                        sts32(b, lw);
                    } else {
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"((unsigned short)hw) : "memory");
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(b), "h"((unsigned short)lw) : "memory");
                    }
                }
            } else {
                const uint32_t byte = (uint32_t)lane * 2 * E, at = byte / S::kSwz, col = byte % S::kSwz;
#pragma unroll 4
                for (int h = 0; h < NH; ++h) {
                    uint32_t v[E / 2];
                    load(h, v);
                    const uint32_t a = tile + at * (uint32_t)(N * S::kSwz) + swizzle<S::kSwz>((uint32_t)h * S::kSwz + col);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e)
                        sts32(a + 4 * e, v[e]);
                }
                if (lane == 0)
                    s_qscale[x][0] = ks;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_q_full[x]));
            // the rest of this (query, head chunk)
            wk.step((int)min((int64_t)(wk.nt - wk.tile), wk.end - wk.it));
            ++seg;
        }
        // queries that see nothing are in no CTA's share
        for (int q = blockIdx.x; q < nq && !w.joined && warp == 5; q += gridDim.x)
            if (s_pre[q + 1] == s_pre[q]) {
                const int64_t row = (w.q0 + q) * p.hq;
                uint32_t *out = reinterpret_cast<uint32_t *>(p.out + row * D);
                for (int64_t i = lane; i < (int64_t)p.hq * D / 2; i += 32)
                    out[i] = 0u;
                for (int h = lane; h < p.hq && p.lse; h += 32)
                    p.lse[row + h] = -INFINITY;
            }
    } else if (warp == 2) {
        // ---------------- MMAs of the scores ----------------
        constexpr uint32_t kId = mma_idesc(!FP8, !FP8, 128, N, false, false);
        constexpr int kKB = 32;                               // bytes of K a step takes of a K-major row
        uint32_t it = 0;
        Turn turn;
        bool ok = true, fresh = true;
        while (!wk.done() && ok) {
            const int n = wk.count(CH), sb = turn.buf();
            const uint32_t x = turn.seg % kQSlots;
            if (fresh)
                ok = warp_wait(smem_u32(&bar_q_full[x]), (turn.seg / kQSlots) & 1u, abort_flag);
            ok = ok && warp_wait(smem_u32(&bar_s_empty[sb]), turn.buf_phase() ^ 1u, abort_flag);
            const uint32_t qt = qbase + x * (uint32_t)S::kQBytes;
            for (int i = 0; i < n && ok; ++i, ++it) {
                const uint32_t s = it % ST;
                ok = warp_wait(smem_u32(&bar_k_full[s]), (it / ST) & 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t kt = ring + s * (uint32_t)S::kTileBytes;
                const uint32_t d = tmem + (uint32_t)(sb * S::kSCols + i * N);
#pragma unroll
                for (int ks = 0; ks < S::kRowBytes / kKB; ++ks) {
                    const uint32_t at = (uint32_t)(ks * kKB) / S::kSwz, col = (uint32_t)(ks * kKB) % S::kSwz;
                    mma_ss<FP8>(d, smem_desc(kt + at * (128u * S::kSwz) + col, S::kSwz, 16u, 8u * S::kSwz),
                                smem_desc(qt + at * (uint32_t)(N * S::kSwz) + col, S::kSwz, 16u, 8u * S::kSwz), kId, ks > 0);
                }
                mma_commit(smem_u32(&bar_k_empty[s]));
            }
            __syncwarp();
            if (!ok)
                break;
            mma_commit(smem_u32(&bar_s_full[sb]));
            fresh = wk.last(n);
            if (fresh)
                mma_commit(smem_u32(&bar_q_empty[x]));
            turn.step(fresh);
            wk.step(n);
        }
        if (!ok)
            *abort_flag = 1;
        mma_commit(smem_u32(&bar_drain));   // every MMA has completed before tensor memory is released
        (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_drain), 0));
    } else if (warp == 3) {
        // ---------------- MMAs of the values ----------------
        constexpr uint32_t kId = mma_idesc(!FP8, 1, 128, NO, true, true);     // weights E5M2 or bf16
        constexpr int kTok = FP8 ? 32 : 16;                   // tokens of a step
        const int BR = w.box_rows, nbox = 128 / BR;
        const uint32_t vring = ring + (uint32_t)(ST * S::kTileBytes);
        uint32_t it = 0;
        Turn turn;
        bool ok = true;
        while (!wk.done() && ok) {
            const int n = wk.count(CH), slot = turn.info(), g = turn.group();
            ok = warp_wait(smem_u32(&bar_info_full[slot]), turn.info_phase(), abort_flag);
            ok = ok && warp_wait(smem_u32(&bar_p_full[g]), turn.chunk() & 1u, abort_flag);
            const uint32_t d = tmem + (uint32_t)(kSBufs * S::kSCols + g * NO);
            for (int i = 0; i < n && ok; ++i, ++it) {
                const uint32_t s = it % ST;
                ok = warp_wait(smem_u32(&bar_v_full[s]), (it / ST) & 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t vt = vring + s * (uint32_t)S::kTileBytes;
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
                            for (int y = r0 * (S::kSwz / 16) + lane; y < r1 * (S::kSwz / 16); y += 32)
                                sts128(vt + (uint32_t)at * (128u * S::kSwz) + (uint32_t)y * 16u, 0u, 0u, 0u, 0u);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                const uint32_t pt = pbase + (uint32_t)((g * CH + i) * S::kPBytes);
#pragma unroll
                for (int ks = 0; ks < 128 / kTok; ++ks)
                    // of 64 dims the 128 rows are the same 64 twice
                    mma_ss<FP8>(d, smem_desc(vt + (uint32_t)(ks * kTok * S::kSwz), S::kSwz,
                                             S::kAtoms == 2 ? 128u * S::kSwz : 0u, 8u * S::kSwz),
                                smem_desc(pt + (uint32_t)(ks * kTok * 16), 0, 128u, S::kPBytes == 2048 ? 0u : 2048u), kId,
                                i > 0 || ks > 0);
                mma_commit(smem_u32(&bar_v_empty[s]));
            }
            __syncwarp();
            if (!ok)
                break;
            mma_commit(smem_u32(&bar_o_full[g]));
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_info_empty[slot]));
            turn.step(wk.last(n));
            wk.step(n);
        }
        if (!ok)
            *abort_flag = 1;
        mma_commit(smem_u32(&bar_drain));
        (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_drain), 0));
    } else if (warp == 4) {
        // ---------------- block lists and page lookups ----------------
        const int BR = w.box_rows, lb = __ffs(BR) - 1, nbox = 128 >> lb;
        int list_q = -1, cnt = 0;
        Turn turn;
        bool ok = true;
        while (!wk.done() && ok) {
            const int n = wk.count(CH), slot = turn.info();
            ok = warp_wait(smem_u32(&bar_info_empty[slot]), turn.info_phase() ^ 1u, abort_flag);
            if (!ok)
                break;
            const int64_t len = s_len[wk.q];
            if (p.topk_ids && list_q != wk.q) {
                // the ids that name a block, in order; a repeated one is kept as -1
                list_q = wk.q;
                int32_t a0 = -1, a1 = -1;
                if (nq * p.topk <= kSmallIds) {
                    a0 = lane < p.topk ? s_ids[wk.q * p.topk + lane] : -1;
                    a1 = lane + 32 < p.topk ? s_ids[wk.q * p.topk + lane + 32] : -1;
                } else {
                    const int32_t *ids = p.topk_ids + (w.q0 + wk.q) * p.topk;
                    a0 = lane < p.topk ? __ldg(ids + lane) : -1;
                    a1 = lane + 32 < p.topk ? __ldg(ids + lane + 32) : -1;
                }
                const bool v0 = a0 >= 0 && (int64_t)a0 * p.block_tokens < len;
                const bool v1 = a1 >= 0 && (int64_t)a1 * p.block_tokens < len;
                const uint32_t m0 = __ballot_sync(0xffffffffu, v0), m1 = __ballot_sync(0xffffffffu, v1);
                const uint32_t below = (1u << lane) - 1u;
                const bool dup0 = __match_any_sync(0xffffffffu, a0) & below;       // of an id before it
                bool dup1 = false;
                if (p.topk > 32) {
                    dup1 = __match_any_sync(0xffffffffu, a1) & below;
                    for (int i = 0; i < 32; ++i)
                        dup1 |= __shfl_sync(0xffffffffu, a0, i) == a1;
                }
                if (v0)
                    s_list[__popc(m0 & below)] = dup0 ? -1 : a0;
                if (v1)
                    s_list[__popc(m0) + __popc(m1 & below)] = dup1 ? -1 : a1;
                cnt = __popc(m0) + __popc(m1);
                __syncwarp();
            }
            for (int x = lane; x < n * nbox; x += 32) {
                const int i = x >> (7 - lb), b = x & (nbox - 1);
                const int64_t v = (int64_t)(wk.tile + i) * 128 + b * BR;
                int64_t j = v;
                bool in = true;
                if (p.topk_ids) {
                    const int64_t k = p.block_shift >= 0 ? (uint32_t)v >> p.block_shift
                                                         : (uint32_t)v / (uint32_t)p.block_tokens;   // below 64 * 1024 tokens
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
            turn.step(wk.last(n));
            wk.step(n);
        }
    } else if (warp >= 8) {
        // ---------------- softmax and output: group g takes the segments s with s % kGroups == g ----------------
        // (a segment: what the CTA holds of a (query, head chunk))
        const int g = (warp - 8) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const int BR = w.box_rows, lb = __ffs(BR) - 1;
        const uint32_t o_tmem = tmem + lane_off + (uint32_t)(kSBufs * S::kSCols + g * NO);
        const uint32_t ptile = pbase + (uint32_t)(g * CH * S::kPBytes);
        constexpr float kPScale = FP8 ? 32768.0f : 1.0f; // E5M2 parts use the range up to 57,344
        float m[NH], l[NH], acc[NH];
        uint32_t k = 0, seg = 0, o_phase = 0;      // k: chunks of this group
        bool ok = true, first = true;
        float vs = 1.0f;
        auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); };
        auto add_output = [&]() {   // adds the value products of this group's last chunk
            ok = ok && warp_wait(smem_u32(&bar_o_full[g]), o_phase, abort_flag);
            o_phase ^= 1u;
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int part = 0; part < (FP8 ? 3 : 1); ++part) {
                    uint32_t r[NH];
                    if (NH == 8)
                        tmem_ld8(o_tmem + (uint32_t)(part * NH), r);
                    else
                        tmem_ld16(o_tmem + (uint32_t)(part * NH), r);
                    tc_wait_ld();
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        acc[h] += __uint_as_float(r[h]);
                }
                tc_fence_before();
            }
        };
        // reduces a value of each head over the 128 threads of the group; every thread gets all.
        // Successive calls exchange in two places by turns: a warp that writes one has passed
        // the barrier of the call before, which every warp reaches after it has read what the
        // call before that left in the same place.
        auto group_reduce = [&](float (&v)[NH], uint32_t turn, auto max_tag) {
            constexpr bool MAX = decltype(max_tag)::value;
            float (*red)[16] = s_red[g][turn & 1u];
            const float x = butterfly<NH, MAX>(v, lane);
            if ((lane & (32 / NH - 1)) == 0)
                red[quarter][lane / (32 / NH)] = x;
            group_sync();
            test_lag(quarter == 1);
#pragma unroll
            for (int h = 0; h < NH; ++h)
                v[h] = MAX ? fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h]))
                           : (red[0][h] + red[1][h]) + (red[2][h] + red[3][h]);
        };
        while (!wk.done()) {
            if ((int)(seg % kGroups) != g) {
                wk.step((int)min((int64_t)(wk.nt - wk.tile), wk.end - wk.it));
                ++seg;
                continue;
            }
            const int n = wk.count(CH), slot = g * kGroupInfo + (int)(k % kGroupInfo);
            const int sb = g * kGroupBufs + (int)(k % kGroupBufs);
            const bool last = wk.last(n);
            const uint32_t x = seg % kQSlots;
            const int hcol = wk.hc % nchunk_heads * NH, head = wk.hc / nchunk_heads;
            if (first) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    // finite, so that a score of -infinity (a token that is not visible, or an
                    // infinite key) has no weight under any maximum
                    m[h] = -FLT_MAX;
                    l[h] = 0.0f;
                    acc[h] = 0.0f;
                }
                vs = attn_v_scale(p, head);
            }
            ok = ok && warp_wait(smem_u32(&bar_info_full[slot]), (k / kGroupInfo) & 1u, abort_flag);
            ok = ok && warp_wait(smem_u32(&bar_q_full[x]), (seg / kQSlots) & 1u, abort_flag);
            ok = ok && warp_wait(smem_u32(&bar_s_full[sb]), (k / kGroupBufs) & 1u, abort_flag);
            if (!ok)
                *abort_flag = 1;
            // Two passes over the chunk's scores in tensor memory, each a loop over the
            // tiles: the unrolled form held them in registers, and its length cost more in
            // instruction fetches (2.3 of the 4 cycles a warp instruction took) than
            // reading them twice does.
            const uint32_t sbuf = tmem + lane_off + (uint32_t)(sb * S::kSCols);
            auto scores = [&](int i, float (&z)[NH]) {     // of this thread's token of tile i
                uint32_t r[N];
                tmem_ld16(sbuf + (uint32_t)(i * N), r);
                const bool seen = (row & (BR - 1)) < s_nv[slot][i][row >> lb];
                tc_wait_ld();
#pragma unroll
                for (int h0 = 0; h0 < NH; h0 += 4) {
                    const float4 qs4 = *reinterpret_cast<const float4 *>(&s_qscale[x][FP8 ? h0 : 0]);
                    const float qs[4] = {qs4.x, qs4.y, qs4.z, qs4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int h = h0 + e;
                        z[h] = FP8 ? __uint_as_float(r[h]) + __uint_as_float(r[NH + h]) : __uint_as_float(r[h]);
                        z[h] = seen ? z[h] * qs[FP8 ? e : 0] : -INFINITY;
                    }
                }
            };
            float mx[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h)
                mx[h] = -INFINITY;
            if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    float z[NH];
                    scores(i, z);
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        mx[h] = fmaxf(mx[h], z[h]);
                }
            }
            group_reduce(mx, k, std::true_type());
            if (!first)
                add_output();
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                mx[h] = fmaxf(m[h], mx[h]);
                const float alpha = m[h] == mx[h] ? 1.0f : exp2_approx(m[h] - mx[h]);
                m[h] = mx[h];
                l[h] *= alpha;
                acc[h] *= alpha;
            }
            if (ok) {
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    float e[NH];
                    scores(i, e);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        e[h] = exp2_approx(e[h] - m[h]);
                        l[h] += e[h];
                    }
                    const uint32_t a = ptile + (uint32_t)(i * S::kPBytes + row * 16);
                    if (FP8) {
                        uint32_t hw[2], mw[2], lw[2];
#pragma unroll
                        for (int h = 0; h < 8; h += 4)
                            split_weights(e[h] * kPScale, e[h + 1] * kPScale, e[h + 2] * kPScale, e[h + 3] * kPScale,
                                          hw[h / 4], mw[h / 4], lw[h / 4]);
                        sts128(a, hw[0], hw[1], mw[0], mw[1]);
                        sts128(a + 2048u, lw[0], lw[1], 0u, 0u);         // columns that nobody reads
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
            if (ok && lane == 0) {
                mbar_arrive(smem_u32(&bar_p_full[g]));
                mbar_arrive(smem_u32(&bar_s_empty[sb]));
                mbar_arrive(smem_u32(&bar_info_empty[slot]));
                if (last)
                    mbar_arrive(smem_u32(&bar_q_empty[x]));
            }
            if (last) {
                // the sum over the tokens while the values are multiplied; then a thread is a dim
                group_reduce(l, k + 1, std::false_type());
                add_output();
                if (!ok)
                    *abort_flag = 1;
                group_sync();                    // the next maxima come where these sums were
                // a wait of any warp that ran out spoils the whole (query, head chunk)
                const bool good = *abort_flag == 0;
                const float bad = __int_as_float(0x7fc00000);
                const bool whole = wk.tile + n == wk.nt && wk.it + n - i0 >= wk.nt;
                const bool began = wk.it - wk.tile >= i0;      // in this CTA
                const int nh = min(NH, p.group - hcol);
                const int64_t hr = (w.q0 + wk.q) * p.hq + head * p.group + hcol;
                float hm = m[0], hl = l[0];      // of head `row`, for the threads that have one
#pragma unroll
                for (int h = 1; h < NH; ++h) {
                    hm = row == h ? m[h] : hm;
                    hl = row == h ? l[h] : hl;
                }
                const float scale = vs * (1.0f / kPScale);
                if (whole && !w.joined) {
                    uint16_t *out = p.out + hr * D + row;
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        if (h < nh && row < D) {
                            const float o = l[h] == 0.0f ? 0.0f : acc[h] * __fdividef(scale, l[h]);
                            out[h * D] = attn_bf16(good ? o : bad);
                        }
                    if (row < nh && p.lse)
                        p.lse[hr + row] = good ? attn_lse(hm, hl) : bad;
                } else if (whole) {
                    float *rows = w.rows + ((int64_t)wk.q * p.hq + head * p.group + hcol) * (D + 4);
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        if (h < nh && row < D)
                            rows[h * (D + 4) + row] = good ? acc[h] * scale : bad;
                    if (row < nh) {
                        rows[row * (D + 4) + D] = good ? hm : bad;
                        rows[row * (D + 4) + D + 1] = good ? hl : bad;
                    }
                } else {
                    float *piece = w.pieces + ((began ? (int64_t)gridDim.x : 0) + blockIdx.x) * (int64_t)(NH * (D + 2));
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        if (row < D)
                            piece[h * D + row] = good ? acc[h] * scale : bad;
                    if (row < NH) {
                        piece[NH * D + row] = good ? hm : bad;
                        piece[NH * D + NH + row] = good ? hl : bad;
                    }
                    // the CTA in which it began lists it for the join
                    if (began && !w.joined && row == 0) {
                        const int64_t base = wk.it - wk.tile;
                        w.cut[blockIdx.x] = make_int4(wk.q, wk.hc, (int)div64(base + wk.nt - 1, share), 0);
                    }
                }
                ++seg;
            }
            first = last;
            ++k;
            wk.step(n);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_free(tmem, S::kTmem);
    }
    if (w.joined)
        asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------------------
// the join of pieces
// ---------------------------------------------------------------------------
//
// One block joins the pieces of up to 16 heads of one query on one K/V head: the maxima
// and sums of 32 pieces at a time are brought a piece a lane and become weights in shared
// memory, then a thread adds four dims over the pieces.  The pieces lie in L2, so the time
// is a few rounds of loads; the code is kept short because it runs once.  Alone it takes 5
// to 6 us after the decode kernel, 11.5 us for 64 queries behind a prefix and 20 us for 190
// (64 heads, fp32 rows of both halves: 13 and 37 MB), 14 us for the 152 pieces of a long
// prefix of six queries.
enum JoinMode { kJoinCut, kJoinRows, kJoinSplits };

constexpr int kJoinHeads = 16;

// Where piece i is: output rows and maxima of the block's heads, each `stride` floats
// apart, the sums `sums` floats after the maxima.
struct PieceAt {
    const float *o, *m;
    int stride, mstride, sums;
};

template <int D, JoinMode MODE>
__global__ void __launch_bounds__(kJoinHeads * D / 4)
msa_attention_join_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnPieces w,
                          const __grid_constant__ AttnTiles tl)
{
    __shared__ float s_w[32][kJoinHeads];            // weights of the pieces
    __shared__ float s_scale[kJoinHeads];            // of what was added before them
    __shared__ float s_m[kJoinHeads], s_l[kJoinHeads];
    __shared__ const float *s_at[32];                // output of the pieces' first head
    __shared__ int s_stride[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
    int q, c, hcol, nh;                              // query of the window, K/V head, its first head here, heads
    int own0 = 0, own1 = -1, pre0 = 0, pre1 = -1;    // CTAs that hold the pieces
    int prow = 0;                                    // row of the first head in a tile slot
    if (MODE == kJoinCut) {
        const int4 cut = __ldcg(w.cut + blockIdx.x);
        if (cut.x < 0)
            return;
        const int nch = (p.group + w.heads - 1) / w.heads;
        q = cut.x;
        c = cut.y / nch;
        hcol = cut.y % nch * w.heads;
        nh = min(w.heads, p.group - hcol);
        own0 = blockIdx.x;
        own1 = cut.z;
    } else {
        const int nch = (p.group + w.heads - 1) / w.heads, x = blockIdx.x / nch;
        hcol = (blockIdx.x - x * nch) * w.heads;
        q = x / p.hkv;
        c = x - q * p.hkv;
        nh = min(w.heads, p.group - hcol);
        const int qt = 128 >> tl.gp_shift;
        if (MODE == kJoinSplits) {
            pre0 = ((q / qt) * p.hkv + c) * tl.splits;
            pre1 = pre0 + tl.splits - 1;
            prow = ((q % qt) << tl.gp_shift) + hcol;
        } else {
            const int64_t lo = __ldcg(w.pre + q), items = __ldcg(w.pre + q + 1) - lo, total = __ldcg(w.pre + w.nq);
            // the group before the first that starts after the query
            int g = -1;
            for (int i0 = 0; i0 <= p.num_groups && g < 0; i0 += 32) {
                const bool after = i0 + lane <= p.num_groups && __ldcg(tl.groups->start + min(i0 + lane, p.num_groups)) > q;
                const uint32_t first = __ballot_sync(0xffffffffu, after);
                if (first)
                    g = i0 + __ffs(first) - 1;
            }
            if (items > 0) {
                const int64_t share = div64(total * w.head_chunks + w.ctas - 1, w.ctas);
                const int64_t base = lo * w.head_chunks + (int64_t)(c * nch + hcol / w.heads) * items;
                own0 = (int)div64(base + w.segment, share);
                own1 = (int)div64(base + items - 1, share);
            }
            if (--g >= 0) {
                const int nb = (int)(((uint32_t)__ldcg(tl.groups->len + g) + kAttnTokens - 1) / kAttnTokens);
                if (nb > 0) {
                    const int at = q - __ldcg(tl.groups->start + g);
                    const int64_t share = __ldcg(&tl.groups->share);
                    const int64_t base = __ldcg(tl.groups->item + g) + kAttnUnit +
                                         (int64_t)((at / qt) * p.hkv + c) * (nb + kAttnUnit);
                    pre0 = (int)div64(base, share);
                    pre1 = (int)div64(base + nb - 1, share);
                    prow = ((at % qt) << tl.gp_shift) + hcol;
                }
            }
        }
    }
    const int n_own = own1 - own0 + 1, n = n_own + pre1 - pre0 + 1;
    const int head0 = c * p.group + hcol;
    auto piece = [&](int i) {
        PieceAt a;
        const bool own = i < n_own;
        const int c0 = own ? own0 : pre0, c1 = own ? own1 : pre1;
        if (!own)
            i -= n_own;
        if (MODE == kJoinRows && c0 == c1) {         // one CTA held it whole
            a.o = (own ? w.rows : tl.rows) + ((int64_t)q * p.hq + head0) * (D + 4);
            a.m = a.o + D;
            a.stride = a.mstride = D + 4;
            a.sums = 1;
        } else if (own) {
            a.o = w.pieces + (int64_t)(i > 0 ? c0 + i : w.ctas + c0) * (w.heads * (D + 2));
            a.m = a.o + w.heads * D;
            a.stride = D;
            a.mstride = 1;
            a.sums = w.heads;
        } else {
            const int slot = MODE == kJoinSplits ? c0 + i : i > 0 ? c0 + i : tl.ctas + c0;
            const float *base = tl.pieces + (int64_t)slot * (tl.slot_rows * (D + 2));
            a.o = base + prow * D;
            a.m = base + tl.slot_rows * D + 2 * prow;
            a.stride = D;
            a.mstride = 2;
            a.sums = 1;
        }
        return a;
    };
    const int h = tid / (D / 4), d = tid % (D / 4) * 4;        // this thread's head and dims
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (tid < kJoinHeads) {
        s_m[tid] = -INFINITY;
        s_l[tid] = 0.0f;
    }
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int count = min(32, n - i0);
        __syncthreads();
        // weights: a warp per head, a lane per piece
        const PieceAt a = piece(i0 + min(lane, count - 1));
        if (warp == 0) {
            s_at[lane] = a.o;
            s_stride[lane] = a.stride;
        }
        for (int k = warp; k < nh; k += blockDim.x >> 5) {
            const float pm = __ldcg(a.m + k * a.mstride);
            const float pl = lane < count ? __ldcg(a.m + k * a.mstride + a.sums) : 0.0f;
            const bool seen = pl != 0.0f;                       // a NaN goes on
            float mx = seen ? pm : -INFINITY;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float before = s_m[k];
            mx = fmaxf(mx, before);
            const float wt = seen ? exp2_approx(pm - mx) : 0.0f;
            float sum = pl * wt;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, x);
            s_w[lane][k] = wt;
            __syncwarp();
            if (lane == 0) {
                const float a = before == -INFINITY ? 0.0f : exp2_approx(before - mx);
                s_scale[k] = a;
                s_m[k] = mx;
                s_l[k] = s_l[k] * a + sum;
            }
        }
        __syncthreads();
        if (h < nh) {
            const float a = s_scale[h];
            acc.x *= a;
            acc.y *= a;
            acc.z *= a;
            acc.w *= a;
            // eight loads in flight; past the last piece, that one again with no weight
            for (int i = 0; i < count; i += 8) {
                float4 x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = min(i + e, count - 1);
                    x[e] = __ldcg(reinterpret_cast<const float4 *>(s_at[j] + h * s_stride[j] + d));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float wt = i + e < count ? s_w[i + e][h] : 0.0f;
                    const bool seen = wt != 0.0f;               // nothing seen: the row may hold anything
                    acc.x = seen ? fmaf(x[e].x, wt, acc.x) : acc.x;
                    acc.y = seen ? fmaf(x[e].y, wt, acc.y) : acc.y;
                    acc.z = seen ? fmaf(x[e].z, wt, acc.z) : acc.z;
                    acc.w = seen ? fmaf(x[e].w, wt, acc.w) : acc.w;
                }
            }
        }
    }
    __syncthreads();
    if (h < nh) {
        const int64_t row = (w.q0 + q) * p.hq + head0 + h;
        const float l = s_l[h], inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
        uint2 o;
        o.x = bf16x2_from_f32(acc.x * inv, acc.y * inv);
        o.y = bf16x2_from_f32(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(p.out + row * D + d) = o;
        if (d == 0 && p.lse)
            p.lse[row] = attn_lse(s_m[h], l);
    }
}

template <int D, bool FP8, int NH>
cudaError_t launch_decode(const AttnParams &p, const AttnPieces &w, const CUtensorMap &kmap, const CUtensorMap &vmap,
                          cudaStream_t stream)
{
    using S = Shape<D, FP8, NH>;
    const void *fn = reinterpret_cast<const void *>(&msa_attention_decode_kernel<D, FP8, NH>);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess)
        return e;
    void *args[] = {const_cast<AttnParams *>(&p), const_cast<AttnPieces *>(&w), const_cast<CUtensorMap *>(&kmap),
                    const_cast<CUtensorMap *>(&vmap)};
    return attn_launch(fn, w.ctas, kThreads, S::kSmem, stream, args);
}

}  // namespace

// Heads a chunk: 16 where a K/V head of a bf16 cache has more than eight, so that its tokens
// are read once: 256 queries of 16 heads on each, 16 blocks, 94 us, 163 in two chunks of eight;
// 37 queries 25.4 and 24.6.  E4M3 caches take eight: 16 heads side by side, 32 and 48 columns
// of two-tile chunks, were slower or alike (37 queries 25.6 us, 18.1 in two chunks of eight;
// 256 104 and 87, with 32 blocks 176 and 178; 64 queries of 64 heads on one 55 and 46).
int attn_decode_heads(int group, bool fp8) { return group <= 8 || fp8 ? 8 : 16; }

cudaError_t attn_decode(const AttnParams &p, const AttnPieces &w, int head_dim, const CUtensorMap &kmap,
                        const CUtensorMap &vmap, cudaStream_t stream)
{
    const bool h8 = w.heads == 8;
    if (head_dim == 128)
        return p.k.fp8 ? launch_decode<128, true, 8>(p, w, kmap, vmap, stream)
               : h8    ? launch_decode<128, false, 8>(p, w, kmap, vmap, stream)
                       : launch_decode<128, false, 16>(p, w, kmap, vmap, stream);
    return p.k.fp8 ? launch_decode<64, true, 8>(p, w, kmap, vmap, stream)
           : h8    ? launch_decode<64, false, 8>(p, w, kmap, vmap, stream)
                   : launch_decode<64, false, 16>(p, w, kmap, vmap, stream);
}

namespace {

template <JoinMode MODE>
cudaError_t launch_join(const AttnParams &p, const AttnPieces &w, const AttnTiles &tiles, int head_dim, int64_t grid,
                        cudaStream_t stream)
{
    void *args[] = {const_cast<AttnParams *>(&p), const_cast<AttnPieces *>(&w), const_cast<AttnTiles *>(&tiles)};
    return attn_launch(head_dim == 128 ? reinterpret_cast<const void *>(&msa_attention_join_kernel<128, MODE>)
                                       : reinterpret_cast<const void *>(&msa_attention_join_kernel<64, MODE>),
                       grid, w.heads * head_dim / 4, 0, stream, args);
}

}  // namespace

cudaError_t attn_join_cut(const AttnParams &p, const AttnPieces &w, int head_dim, cudaStream_t stream)
{
    return launch_join<kJoinCut>(p, w, AttnTiles(), head_dim, w.ctas, stream);
}

cudaError_t attn_join_rows(const AttnParams &p, const AttnPieces &w, const AttnTiles &tiles, int head_dim,
                           cudaStream_t stream)
{
    return launch_join<kJoinRows>(p, w, tiles, head_dim, w.nq * w.head_chunks, stream);
}

cudaError_t attn_join_splits(const AttnParams &p, const AttnPieces &w, const AttnTiles &tiles, int head_dim,
                             cudaStream_t stream)
{
    return launch_join<kJoinSplits>(p, w, tiles, head_dim, p.num_queries * w.head_chunks, stream);
}
