// Attention of tiles of queries on the tcgen05 tensor cores: prefill chunks over the
// blocks their queries selected, and groups of queries over a prefix they share.
//
// What is computed is stated in include/msa_attention.h.
//
// A tile is 128 rows: QT queries times the heads of one K/V head, padded to a power of two.
// Per 128 tokens the CTA computes S [128 rows, 128 tokens] = Q . K^T and
// O [128 rows, D] += P . V, each product read from shared memory as TMA copied it (K-major
// keys, N-major values) with P as the A operand in tensor memory, where it takes the place
// of the scores.  E4M3 caches run on kind::f8f6f4 with Q split into E4M3 halves hi | lo and P
// into three E5M2 parts (MMAs at twice the rate: no conversion of keys or values, and half
// the bytes in shared memory); bf16 on kind::f16.
//   warp 0     TMA: page lookups one tile ahead, key and value copies
//   warp 1     MMAs; zeroes value rows past the history before they are multiplied
//   warps 2-9  softmax and output: two groups of four, a thread per row; group g takes the
//              tokens 64 g .. 64 g + 63 of every tile, then D / 2 of the dims
// Scores are made 64 tokens at a time into two buffers, one a group, so that the scores of
// one half are ready while the other's softmax runs, and two CTAs share an SM (half the
// tensor memory and half the shared memory each).
// Measured: 8,192 prefill queries in four chunks (64 query heads on 8 of 128 dims, E4M3, 16
// blocks of 128 tokens each) 1.00 ms, 0.28 of the measured bf16 rate by the tokens that the
// queries selected.  A tile of 16 queries runs over the union of their lists, 19 to 27
// blocks, so a third of the products is masked.  Nothing is full: 55 % of the issue slots,
// 48 % of the ALU's (the split of the weights is 15 of about 25 instructions for four
// tokens), tensor pipe 51 %, DRAM 4 %; a tile is a chain of scores, maximum, weights and
// values, which two CTAs an SM do not hide.  Weights in two E4M3 halves took 0.93 ms (4,400
// cycles a tile), but lost those below 2^-14 of a row's largest.  With them were slower: all
// 64 scores of a row held in registers (1.04 ms), 64-token tiles with weights beside the
// scores (1.08), 128-token scores in one MMA group (1.11 to 1.17), separate warps for the two
// products (1.16).
// About 15,000 of a CTA's cycles go by before its first scores.
// 64 queries behind 8,192 shared tokens: 69 us with their own tokens and the join.
// The running maximum is a reference that follows the true one lazily: weights are taken
// relative to it until the true maximum is kLazy powers of two above, and only then is the
// output in tensor memory rescaled, which few tiles after the first need.  The groups hand
// the reference of a row to one another half by half.
//
// Sparse (DENSE = false): the tile's queries run over the union of their blocks, each row
// masked to its own.  A weight of zero does not hide an infinity or a NaN in the values of
// a token that another row of the tile sees, so a row whose output is not finite is
// computed again from its own tokens alone.
// Prefix (DENSE = true): (tile, K/V head, 128 tokens) items laid end to end over the groups,
// an equal share for each CTA; every piece goes to the workspace and is joined with the
// queries' own tokens.

#include "msa_attention_internal.h"
#include "msa_tcgen05.cuh"

#include <cstring>

namespace {

constexpr int kThreads = 320;
constexpr int kInfo = 4;            // tiles whose validity words are held
constexpr int kMaxBoxes = 16;
constexpr int kMaxList = kAttnTileList;      // blocks of a tile's list
constexpr int kTileQueries = 32;    // queries of a tile at most (a mask word)

template <int D, bool FP8>
struct TileShape {
    static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
    static constexpr int kSwz = kRowBytes < 128 ? kRowBytes : 128;
    static constexpr int kAtoms = kRowBytes / kSwz;
    static constexpr int kTileBytes = 128 * kRowBytes;
    static constexpr int kQBytes = 128 * D * 2;                   // bf16, or E4M3 hi | lo
    static constexpr int kStages = kTileBytes == 32768 ? 1 : 2;   // of keys, and of values
    static constexpr int kSmem = 1024 + kQBytes + 2 * kStages * kTileBytes;
    static constexpr int kTmem = 256;                             // scores (and weights) | output
    static_assert(2 * kStages * kTileBytes >= 4 * kMaxList * 8, "scratch of the list");
};

constexpr float kLazyBf16 = 8.0f, kLazyFp8 = 4.0f;
// Weights over E4M3 values are 2^11 times larger, up to 2^15 of E5M2's 57,344: their parts
// reach down to 2^-28 of the reference.
constexpr float kPOffset = 11.0f;

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Pairs of fp32 as one 64-bit operand: two multiply-adds or sums an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpack2(uint64_t x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// What a CTA works on: rows of the tile, a K/V head and a range of 128-token tiles.
struct Segment {
    int t0;                  // first query (prefix: of the window)
    int nq;                  // queries in the tile
    int c;                   // K/V head
    int p0, p1;              // 128-token tiles
    int group, len;          // prefix: the group, its tokens
    bool whole, began;       // prefix: all of its unit; it starts the unit
};

struct DenseWalk {
    // group g has tiles x K/V heads units of kAttnUnit items without a tile, then nb
    // 128-token tiles
    const AttnGroups *tab;
    int64_t it, end, base;   // base: the item of the unit's first tile
    int ngroups, hkv, qt, g, unit;

    __device__ int nb() const { return (int)(((uint32_t)tab->len[g] + 127u) / 128u); }
    __device__ void find()
    {
        while (g < ngroups && tab->item[g + 1] <= it) {
            ++g;
            unit = 0;
        }
        if (g < ngroups && it < end) {
            const int n = nb() + kAttnUnit;
            unit = (int)((it - tab->item[g]) / n);
            base = tab->item[g] + (int64_t)unit * n + kAttnUnit;
            it = max(it, base);
        }
    }
    __device__ bool get(Segment &s) const
    {
        if (it >= end || g >= ngroups)
            return false;
        const int tile = unit / hkv;
        s.c = unit - tile * hkv;
        s.t0 = tab->start[g] + tile * qt;
        s.nq = min(qt, tab->start[g + 1] - s.t0);
        s.group = g;
        s.len = tab->len[g];
        s.p0 = (int)(it - base);
        s.p1 = (int)min((int64_t)nb(), end - base);
        s.began = s.p0 == 0;
        s.whole = s.began && s.p1 == nb();
        return true;
    }
    __device__ void next(const Segment &s)
    {
        it = base + s.p1;
        find();
    }
};

template <int D, bool FP8, bool DENSE>
__global__ void __launch_bounds__(kThreads, 2)
msa_attention_tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnTiles w,
                          const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = TileShape<D, FP8>;
    constexpr int ST = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_k_full[ST], bar_k_empty[ST], bar_v_full[ST], bar_v_empty[ST];
    __shared__ __align__(8) uint64_t bar_info[kInfo];
    __shared__ __align__(8) uint64_t bar_q, bar_s[2], bar_p[2], bar_pv, bar_o, bar_drain;
    __shared__ __align__(8) uint64_t bar_ref[2][4];
    __shared__ uint8_t s_nv[kInfo][kMaxBoxes];     // visible rows of each box
    __shared__ uint32_t s_gap[kInfo];              // boxes without a page before the history's end
    __shared__ union {
        AttnGroups groups;                         // DENSE
        struct {
            int32_t block[kMaxList];               // the list: block, and the sequence's first query above it
            uint32_t mask[kMaxList];               // the tile's queries that selected it
            int64_t toff[kTileQueries];
            int32_t len[kTileQueries], lead[kTileQueries], maxlen[kTileQueries];
        } sp;
    } u;
    __shared__ float s_ref[128], s_row[2][128];    // exchange between the two threads of a row
    __shared__ int s_ok[2][4];
    __shared__ int s_n;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t qsm = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t kring = qsm + S::kQBytes, vring = kring + ST * S::kTileBytes;
    volatile int *abort_flag = &s_abort;
    const int qt = 128 >> w.gp_shift;

    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        for (int i = 0; i < ST; ++i) {
            mbar_init(smem_u32(&bar_k_full[i]), 1);
            mbar_init(smem_u32(&bar_k_empty[i]), 1);
            mbar_init(smem_u32(&bar_v_full[i]), 1);
            mbar_init(smem_u32(&bar_v_empty[i]), 1);
        }
        for (int i = 0; i < kInfo; ++i)
            mbar_init(smem_u32(&bar_info[i]), 1);
        mbar_init(smem_u32(&bar_q), 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar_s[i]), 1);
            mbar_init(smem_u32(&bar_p[i]), 4);
            for (int j = 0; j < 4; ++j)
                mbar_init(smem_u32(&bar_ref[i][j]), 1);
        }
        mbar_init(smem_u32(&bar_pv), 1);
        mbar_init(smem_u32(&bar_o), 1);
        mbar_init(smem_u32(&bar_drain), 1);
        s_abort = 0;
        s_n = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&s_tmem), S::kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);

    Segment seg;
    DenseWalk dw;
    if (DENSE) {
        // the groups' queries within the window, and their items, by one warp
        if (warp == 0) {
            int64_t items = 0;
            int32_t edge = 0;                        // queries before, a running maximum
            const int n = p.num_groups;
            for (int g0 = 0; g0 <= n; g0 += 32) {
                const int g = g0 + lane;
                int64_t e64 = g <= n ? (int64_t)__ldg(p.group_start + g) - w.q0 : 0;
                int32_t e = (int32_t)max((int64_t)0, min(e64, w.nq));
                const int32_t len = g < n ? attn_len(p, __ldg(p.prefix_len + g), __ldg(p.prefix_offset + g)) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int32_t x = __shfl_up_sync(0xffffffffu, e, o);
                    if (lane >= o)
                        e = max(e, x);
                }
                e = max(e, edge);
                if (g <= n)
                    u.groups.start[g] = e;
                if (g < n)
                    u.groups.len[g] = len;
                edge = __shfl_sync(0xffffffffu, e, 31);
            }
            __syncwarp();
            for (int g0 = 0; g0 < n; g0 += 32) {
                const int g = g0 + lane;
                int64_t x = 0;
                if (g < n) {
                    const int q = u.groups.start[g + 1] - u.groups.start[g];
                    const int64_t nb = ((int64_t)u.groups.len[g] + 127) / 128;
                    x = (int64_t)((q + qt - 1) / qt) * p.hkv * (nb > 0 ? nb + kAttnUnit : 0);
                }
                int64_t inc = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o)
                        inc += y;
                }
                if (g < n)
                    u.groups.item[g] = items + inc - x;
                items += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0)
                u.groups.item[n] = items;
        }
    } else {
        // the union of the queries' blocks: a hash of (sequence, block) in the ring's memory,
        // then sorted by rank, so that the order does not depend on the insertions'
        seg.t0 = (int)(blockIdx.x / (p.hkv * w.splits)) * qt;
        seg.nq = (int)min((int64_t)qt, p.num_queries - seg.t0);
        seg.c = (int)(blockIdx.x / w.splits % p.hkv);
        if (tid < kTileQueries) {
            u.sp.len[tid] = tid < seg.nq ? max(__ldg(p.kv_len + seg.t0 + tid), 0) : 0;
            u.sp.toff[tid] = tid < seg.nq ? __ldg(p.table_offset + seg.t0 + tid) : 0;
            u.sp.maxlen[tid] = 0;
        }
        const int ids = seg.nq * p.topk;
        int slots = 64;
        while (slots < 2 * ids)
            slots *= 2;
        int32_t *keys = reinterpret_cast<int32_t *>(smem_raw + (kring - smem_u32(smem_raw)));
        uint32_t *masks = reinterpret_cast<uint32_t *>(keys + slots);
        for (int i = tid; i < slots; i += kThreads) {
            keys[i] = -1;
            masks[i] = 0;
        }
        __syncthreads();
        if (tid < seg.nq) {   // the first query of the same sequence
            int l = 0;
            while (u.sp.toff[l] != u.sp.toff[tid])
                ++l;
            u.sp.lead[tid] = l;
            atomicMax(&u.sp.maxlen[l], u.sp.len[tid]);
        }
        __syncthreads();
        for (int i = tid; i < ids; i += kThreads) {
            const int q = i / p.topk;
            const int32_t id = __ldg(p.topk_ids + (int64_t)seg.t0 * p.topk + i);
            if (id >= 0 && (int64_t)id * p.block_tokens < u.sp.len[q]) {
                // below 2^24 blocks of at least 128 tokens, and 32 sequences
                const int32_t key = (u.sp.lead[q] << 24) | id;
                uint32_t h = ((uint32_t)key * 2654435761u) & (uint32_t)(slots - 1);
                for (;;) {      // at most half of the slots fill up
                    const int32_t old = atomicCAS(&keys[h], -1, key);
                    if (old == -1 || old == key)
                        break;
                    h = (h + 1) & (uint32_t)(slots - 1);
                }
                atomicOr(&masks[h], 1u << q);
            }
        }
        __syncthreads();
        int32_t *found = reinterpret_cast<int32_t *>(masks + slots);     // the entries, in no order
        uint32_t *found_mask = reinterpret_cast<uint32_t *>(found + slots);
        for (int i = tid; i < slots; i += kThreads)
            if (keys[i] != -1) {
                const int k = atomicAdd(&s_n, 1);
                found[k] = keys[i];
                found_mask[k] = masks[i];
            }
        __syncthreads();
        for (int i = tid; i < s_n; i += kThreads) {
            int rank = 0;
            for (int j = 0; j < s_n; ++j)
                rank += found[j] < found[i];
            u.sp.block[rank] = found[i];
            u.sp.mask[rank] = found_mask[i];
        }
        // the scratch is TMA's from here on
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int per_block = DENSE ? 1 : p.block_tokens / 128;     // 128-token tiles of a block
    if (DENSE) {
        const int64_t total = u.groups.item[p.num_groups], share = (total + gridDim.x - 1) / gridDim.x;
        dw.tab = &u.groups;
        dw.ngroups = p.num_groups;
        dw.hkv = p.hkv;
        dw.qt = qt;
        dw.g = 0;
        dw.unit = 0;
        dw.it = min(total, share * blockIdx.x);
        dw.end = min(total, dw.it + share);
        dw.base = 0;
        dw.find();
        if (blockIdx.x == 0)   // what the join needs of the groups
            for (int g = tid; g <= p.num_groups; g += kThreads) {
                w.groups->item[g] = u.groups.item[g];
                w.groups->start[g] = u.groups.start[g];
                if (g < p.num_groups)
                    w.groups->len[g] = u.groups.len[g];
                else
                    w.groups->share = share;
            }
    } else {
        const int n = s_n * per_block, sp = (int)(blockIdx.x % w.splits);
        seg.p0 = n * sp / w.splits;
        seg.p1 = n * (sp + 1) / w.splits;
    }
    // first token of tile v of the list, and its entry
    auto list_tile = [&](int v, int &e) -> uint32_t {
        e = per_block == 1 ? v : v / per_block;
        return (uint32_t)(u.sp.block[e] & 0xFFFFFF) * (uint32_t)p.block_tokens + (uint32_t)(v - e * per_block) * 128u;
    };
    bool once = true;
    // the next segment of this CTA
    auto next_segment = [&](bool first) -> bool {
        if (DENSE) {
            if (!first)
                dw.next(seg);
            return dw.get(seg);
        }
        const bool r = once;
        once = false;
        return r;
    };

    if (warp == 0) {
        // ---------------- copies ----------------
        const int BR = w.box_rows, lb = __ffs(BR) - 1, nbox = 128 >> lb;
        uint32_t it = 0;
        bool ok = true;
        for (bool first = true; ok && next_segment(first); first = false) {
            // A batch of 32 / nbox tiles is looked up at once, a box a lane: row in the page, page
            // (one past the last for a box that shows nothing: zeros), rows that some query
            // sees, and whether the history goes on without a page.  The ring hides the wait.
            const int64_t prefix_off = DENSE ? __ldg(p.prefix_offset + seg.group) : 0;
            const int batch = 32 >> (7 - lb);
            int2 boxes = make_int2(0, 0);
            int nvs = 0;
            bool gaps_of = false;
            for (int v = seg.p0; v < seg.p1 && ok; ++v, ++it) {
                const int k = (v - seg.p0) & (batch - 1);
                if (k == 0) {
                    boxes = make_int2(0, w.oob_page);
                    nvs = 0;
                    gaps_of = false;
                    const int x = v + (lane >> (7 - lb));
                    if (x < seg.p1) {
                        uint32_t tok, len;
                        int64_t off;
                        if (DENSE) {
                            tok = (uint32_t)x * 128u;
                            off = prefix_off;
                            len = (uint32_t)seg.len;
                        } else {
                            int e;
                            tok = list_tile(x, e);
                            off = u.sp.toff[u.sp.block[e] >> 24];
                            len = (uint32_t)u.sp.maxlen[u.sp.block[e] >> 24];
                        }
                        tok += (uint32_t)((lane & (nbox - 1)) * BR);
                        if (tok < len) {
                            const int32_t pg = attn_page(p, off, tok);
                            gaps_of = pg < 0;
                            if (pg >= 0) {
                                boxes = make_int2(attn_page_row(p, tok), pg);
                                nvs = (int)min((uint32_t)BR, len - tok);
                            }
                        }
                    }
                    __syncwarp();
                }
                const int from = k * nbox + (lane & (nbox - 1));
                const int2 box = make_int2(__shfl_sync(0xffffffffu, boxes.x, from), __shfl_sync(0xffffffffu, boxes.y, from));
                const int nv = __shfl_sync(0xffffffffu, nvs, from);
                const uint32_t gaps = (__ballot_sync(0xffffffffu, gaps_of) >> (k * nbox)) & ((1u << nbox) - 1u);
                const uint32_t s = it % ST, par = ((it / ST) & 1u) ^ 1u, slot = it % kInfo;
                ok = warp_wait(smem_u32(&bar_k_empty[s]), par, abort_flag);
                if (!ok)
                    break;
                // the slot's last readers were done before this stage's keys were multiplied
                if (lane < nbox)
                    s_nv[slot][lane] = (uint8_t)nv;
                if (lane == 0)
                    s_gap[slot] = gaps;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&bar_info[slot]));
                auto copy = [&](const CUtensorMap *map, uint32_t dst, uint32_t full) {
#ifndef MSA_STARVE
                    if (lane == 0)
                        mbar_expect_tx(full, (uint32_t)S::kTileBytes);
                    __syncwarp();
                    if (lane < nbox)
#pragma unroll
                        for (int at = 0; at < S::kAtoms; ++at)
                            tma_load_box(dst + (uint32_t)(at * 128 + lane * BR) * S::kSwz, map,
                                         at * (S::kSwz / (FP8 ? 1 : 2)), box.x, seg.c, box.y, full);
#endif
                };
                copy(&kmap, kring + s * (uint32_t)S::kTileBytes, smem_u32(&bar_k_full[s]));
                ok = warp_wait(smem_u32(&bar_v_empty[s]), par, abort_flag);
                if (!ok)
                    break;
                copy(&vmap, vring + s * (uint32_t)S::kTileBytes, smem_u32(&bar_v_full[s]));
            }
        }
        if (!ok)
            *abort_flag = 1;
#ifndef MSA_STARVE
        // every copy has landed before the CTA finishes (of the last tile of an aborted
        // CTA the values may not have been asked for; that wait runs out)
        for (uint32_t s = 0; s < (uint32_t)ST && s < it; ++s) {
            const uint32_t par = ((it - 1u - s) / ST) & 1u;
            (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_k_full[s]), par));
            (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_v_full[s]), par));
        }
        if (!ok)
            for (uint32_t s = 0; s < (uint32_t)ST; ++s)
                (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_k_full[s]), (it / ST) & 1u));
#endif
    } else if (warp == 1) {
        // ---------------- MMAs ----------------
        constexpr uint32_t kIdS = mma_idesc(!FP8, !FP8, 128, 64, false, false);
        constexpr uint32_t kIdO = mma_idesc(1, !FP8, 128, D, false, true);      // weights E5M2 or bf16
        constexpr int kTok = FP8 ? 32 : 16;                   // tokens of a step of the values
        constexpr int kStep = kTok * S::kSwz / 16;
        const int BR = w.box_rows, nbox = 128 / BR;
        const uint64_t q_desc = smem_desc(qsm, S::kSwz, 16u, 8u * S::kSwz);
        const uint64_t k_desc = smem_desc(kring, S::kSwz, 16u, 8u * S::kSwz);
        const uint64_t v_desc = smem_desc(vring, S::kSwz, 128u * S::kSwz, 8u * S::kSwz);
        uint32_t it = 0, nseg = 0;        // it: tiles whose values were multiplied
        bool ok = true;
        for (bool first = true; ok && next_segment(first); first = false, ++nseg) {
            // the scores of half g of the CTA's tile i; `after`: right after the values of that
            // half of tile i - 1 (the first tile of a segment comes after everything, since
            // its queries are made when the output before was read)
            auto scores = [&](uint32_t i, int g, bool after) {
                const uint32_t s = i % ST;
                if (g == 0)
                    ok = warp_wait(smem_u32(&bar_k_full[s]), (i / ST) & 1u, abort_flag);
                // the weights of the half before, whose place the scores take, are multiplied
                ok = ok && (!after || warp_wait(smem_u32(&bar_pv), (uint32_t)g, abort_flag));
                if (!ok)
                    return;
                tc_fence_after();
                const uint64_t kd = k_desc + (uint64_t)(s * (uint32_t)(S::kTileBytes / 16) + g * (64 * S::kSwz / 16));
                const uint32_t d = tmem + (uint32_t)(g * 64);
                if (S::kSwz == 128) {
                    // a swizzle atom is four steps; the halves, or the atoms of a row, follow
                    mma_ss4<FP8, 2, 2>(d, q_desc, kd, kIdS, 0);
                    if (D == 128)
                        mma_ss4<FP8, 2, 2>(d, q_desc + 128 * 128 / 16, FP8 ? kd : kd + 128 * 128 / 16, kIdS, 1);
                } else {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)    // two steps of hi, two of lo
                        mma_ss<FP8>(d, q_desc + (uint64_t)((ks >> 1) * (128 * 64 / 16) + (ks & 1) * 2),
                                    kd + (uint64_t)((ks & 1) * 2), kIdS, ks > 0);
                }
                mma_commit(smem_u32(&bar_s[g]));
                if (g == 1)
                    mma_commit(smem_u32(&bar_k_empty[s]));
            };
            ok = warp_wait(smem_u32(&bar_q), nseg & 1u, abort_flag);
            if (ok && seg.p0 < seg.p1) {
                scores(it, 0, false);
                if (ok)
                    scores(it, 1, false);
            }
            for (int v = seg.p0; v < seg.p1 && ok; ++v, ++it) {
                const uint32_t s = it % ST;
                for (int g = 0; g < 2 && ok; ++g) {
                    const uint32_t vt = vring + s * (uint32_t)S::kTileBytes;
                    if (g == 0) {
                        ok = warp_wait(smem_u32(&bar_v_full[s]), (it / ST) & 1u, abort_flag);
                        if (!ok)
                            break;
                        // rows past the history may hold anything: a weight of zero would not
                        // hide an infinity or a NaN
                        const int nv = lane < nbox ? s_nv[it % kInfo][lane] : 0;
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
                    }
                    ok = warp_wait(smem_u32(&bar_p[g]), it & 1u, abort_flag);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint64_t vd = v_desc + (uint64_t)(s * (uint32_t)(S::kTileBytes / 16) + g * (64 * S::kSwz / 16));
                    const uint32_t pt = tmem + (uint32_t)(g * 64), acc = v > seg.p0 || g > 0;
                    if (FP8)        // two steps, each of three parts against the same values
                        mma_ts33<kStep>(tmem + 128u, pt, vd, kIdO, acc);
                    else
                        mma_ts4<FP8, 8, kStep>(tmem + 128u, pt, vd, kIdO, acc);
                    mma_commit(smem_u32(&bar_pv));
                    if (g == 1)
                        mma_commit(smem_u32(&bar_v_empty[s]));
                    // the half's next scores, when these values are multiplied
                    if (v + 1 < seg.p1)
                        scores(it + 1, g, true);
                }
            }
            __syncwarp();
            if (ok)
                mma_commit(smem_u32(&bar_o));
        }
        if (!ok)
            *abort_flag = 1;
        mma_commit(smem_u32(&bar_drain));   // every MMA has completed before tensor memory is released
        (void)__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_drain), 0));
    } else {
        // ---------------- softmax and output ----------------
        const int quarter = warp & 3, row = quarter * 32 + lane, half = (warp - 2) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t st = lanes + (uint32_t)(half * 64), ot = lanes + 128u;
        const int gp = 1 << w.gp_shift, qi = row >> w.gp_shift, hi = row & (gp - 1);
        const int BR = w.box_rows, lb = __ffs(BR) - 1;
        constexpr float kLazy = FP8 ? kLazyFp8 : kLazyBf16, kOff = FP8 ? kPOffset : 0.0f;
        constexpr int kD2 = D / 2;                      // dims of this thread
        const float nan = __int_as_float(0x7fc00000);
        // the two warps that hold a row's halves
        auto pair_sync = [&]() {
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
            test_lag(half == 1);
        };
        auto softmax_sync = [&]() { asm volatile("bar.sync 5, 256;" ::: "memory"); };
        uint32_t it = 0, nseg = 0;
        bool ok = true;
        for (bool first = true; next_segment(first); first = false, ++nseg) {
            // ---- the queries into shared memory: 16 rows a warp, 16 bytes a lane ----
            const bool real = qi < seg.nq && hi < p.group;
            // a row of q and out
            auto head_row_of = [&](int r) -> int64_t {
                return (w.q0 + seg.t0 + (r >> w.gp_shift)) * p.hq + seg.c * p.group + (r & (gp - 1));
            };
            auto head_row = [&]() -> int64_t { return head_row_of(row); };
            const float ks = attn_k_scale(p, seg.c) * p.scale_log2;
            float qs = fabsf(ks);                          // a negative scale goes into the query
            softmax_sync();                                // everyone is through with the segment before
            {
                constexpr int kLanes = D / 8, kRows = 32 / kLanes;      // lanes of a row, rows of a load
                const uint32_t flip = ks < 0.0f ? 0x80008000u : 0u;
                const int chunk = lane % kLanes;
#pragma unroll
                for (int i = 0; i < 16 / kRows; i += 4) {
                    uint4 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = (warp - 2) * 16 + (i + j) * kRows + lane / kLanes;
                        const bool there = (r >> w.gp_shift) < seg.nq && (r & (gp - 1)) < p.group;
                        x[j] = there ? __ldg(reinterpret_cast<const uint4 *>(p.q + head_row_of(r) * D) + chunk)
                                     : make_uint4(0, 0, 0, 0);
                    }
                    // (the loads of four rows at once, then a loop that is short to fetch)
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        const int r = (warp - 2) * 16 + (i + j) * kRows + lane / kLanes;
                        const uint4 y = x[0];
                        x[0] = x[1];
                        x[1] = x[2];
                        x[2] = x[3];
                        const uint32_t xs[4] = {y.x ^ flip, y.y ^ flip, y.z ^ flip, y.w ^ flip};
                        if (FP8) {
                            // halves hi | lo under the power of two that brings the row's largest
                            // magnitude (magnitudes compare as integers) into [128, 256)
                            uint32_t big = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                big = max(big, max((xs[k] & 0x7FFFu) << 16, xs[k] & 0x7FFF0000u));
#pragma unroll
                            for (int o = kLanes / 2; o > 0; o >>= 1)
                                big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                            big >>= 23;
                            const int e2 = big > 0 ? min(7 - ((int)big - 127), 126) : 0;
                            const float sc = __int_as_float((e2 + 127) << 23);
                            uint32_t hw[2], lw[2];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float x0 = __uint_as_float(xs[k] << 16) * sc;
                                const float x1 = __uint_as_float(xs[k] & 0xFFFF0000u) * sc;
                                const uint32_t h = e4m3x2_from_f32(x0, x1);
                                const float2 d = attn_e4m3x2_to_f2(h);
                                const uint32_t l = e4m3x2_from_f32(x0 - d.x, x1 - d.y);
                                hw[k / 2] = k & 1 ? hw[k / 2] | (h << 16) : h;
                                lw[k / 2] = k & 1 ? lw[k / 2] | (l << 16) : l;
                            }
                            const uint32_t a = swizzle<S::kSwz>((uint32_t)(r * S::kSwz + chunk * 8));
                            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qsm + a), "r"(hw[0]), "r"(hw[1]) : "memory");
                            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qsm + 128 * D + a), "r"(lw[0]), "r"(lw[1])
                                         : "memory");
                            if (chunk == 0)     // an infinity would saturate: no score of such a row is a number
                                s_row[0][r] = big == 255 ? nan : __int_as_float((127 - e2) << 23);
                        } else {
                            const uint32_t byte = (uint32_t)chunk * 16, at = byte / S::kSwz, col = byte % S::kSwz;
                            sts128(qsm + at * (128u * S::kSwz) + swizzle<S::kSwz>((uint32_t)r * S::kSwz + col), xs[0], xs[1],
                                   xs[2], xs[3]);
                        }
                    }
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bar_q));
            if (FP8) {
                softmax_sync();
                qs *= s_row[0][row];
                // a scale of 0, or one that comes out as 0: scores are 0 by the smallest normal
                // too, and the -infinity of a masked one stays what it is
                qs = qs == 0.0f ? 1.17549435e-38f : qs;
            }
            const int len = DENSE ? seg.len : (qi < seg.nq ? u.sp.len[qi] : 0);
            float m = -INFINITY, l = 0.0f;                 // the reference that l is relative to
            for (int v = seg.p0; v < seg.p1; ++v, ++it) {
                ok = ok && warp_wait(smem_u32(&bar_info[it % kInfo]), (it / kInfo) & 1u, abort_flag);
                // tokens of this thread's half that the row sees, from its first
                int vis;
                if (DENSE) {
                    vis = len - v * 128;
                } else {
                    int e;
                    // a row sees the first token of a block that its query selected
                    const uint32_t tok = list_tile(v, e);
                    vis = (u.sp.mask[e] >> qi) & 1u ? (int)((uint32_t)len - tok) : -1;
                }
                vis = real ? vis - half * 64 : -1;
                const uint32_t gaps = ok ? s_gap[it % kInfo] : 0u;
                ok = ok && warp_wait(smem_u32(&bar_s[half]), it & 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after();
                // Two passes over the scores in tensor memory, each a loop over 32 tokens: half
                // the instructions of one that holds 64 in registers, and the kernel is bound
                // by fetching them.
                float mx = -INFINITY;
                const bool any = __any_sync(0xffffffffu, vis > 0);
                // rows that see all or nothing need no masks: a row that sees nothing takes an
                // offset that clears its weights
                const bool masks = __any_sync(0xffffffffu, (vis > 0 && vis < 64) || gaps != 0);
                auto scores = [&](int j0, uint32_t (&x)[32]) {
                    tmem_ld32(st + (uint32_t)j0, x);
                    tc_wait_ld();
                    if (masks) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j0 + j >= vis || ((gaps >> ((half * 64 + j0 + j) >> lb)) & 1u))
                                x[j] = 0xff800000u;
                    }
                };
                if (any) {
#pragma unroll 1
                    for (int j0 = 0; j0 < 64; j0 += 32) {
                        uint32_t x[32];
                        scores(j0, x);
                        auto score = [&](int j) { return __uint_as_float(x[j]); };
                        float a = max3(mx, score(0), score(1)), b = fmaxf(score(2), score(3));
#pragma unroll
                        for (int j = 4; j < 32; j += 4) {
                            a = max3(a, score(j), score(j + 1));
                            b = max3(b, score(j + 2), score(j + 3));
                        }
                        mx = fmaxf(a, b);
                    }
                    mx = vis > 0 ? mx * qs : -INFINITY;
                }
                // the reference, from the half before
                float ref = -INFINITY;
                if (half > 0 || v > seg.p0) {
                    ok = warp_wait(smem_u32(&bar_ref[half ^ 1][quarter]), (half > 0 ? it : it - 1u) & 1u, abort_flag);
                    if (!ok)
                        break;
                    ref = s_ref[row];
                }
                // (-inf + kLazy is -inf: the first visible half sets the reference)
                const bool grow = mx > ref + kLazy;
                if (__any_sync(0xffffffffu, grow)) {
                    const float alpha = grow ? exp2_approx(ref - mx) : 1.0f;
                    ref = grow ? mx : ref;
                    if (half > 0 || v > seg.p0) {
                        // the values of the half before are in the output
                        ok = warp_wait(smem_u32(&bar_pv), (uint32_t)(half ^ 1), abort_flag);
                        if (!ok)
                            break;
                        tc_fence_after();
#pragma unroll 1
                        for (int j = 0; j < D; j += 8) {
                            uint32_t o[8];
                            tmem_ld8(ot + (uint32_t)j, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st8(ot + (uint32_t)j, o);
                        }
                    }
                }
                s_ref[row] = ref;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&bar_ref[half][quarter]));
                l = m == ref ? l : l * exp2_approx(m - ref);
                m = ref;
                if (any) {
                    const float off = vis > 0 && m > -INFINITY ? kOff - m : -INFINITY;
                    const uint64_t qs2 = pack2(qs, qs), off2 = pack2(off, off);
                    uint64_t sum0 = 0, sum1 = 0;
#pragma unroll 1
                    for (int j0 = 0; j0 < 64; j0 += 32) {
                        uint32_t x[32];
                        scores(j0, x);
                        auto score = [&](int j) { return __uint_as_float(x[j]); };
                        uint32_t hw[FP8 ? 8 : 16], mw[8], lw[8];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            float p0, p1, p2, p3;
                            unpack2(fma2(pack2(score(e), score(e + 1)), qs2, off2), p0, p1);
                            unpack2(fma2(pack2(score(e + 2), score(e + 3)), qs2, off2), p2, p3);
                            p0 = exp2_approx(p0);
                            p1 = exp2_approx(p1);
                            p2 = exp2_approx(p2);
                            p3 = exp2_approx(p3);
                            sum0 = add2(sum0, pack2(p0, p1));
                            sum1 = add2(sum1, pack2(p2, p3));
                            if (FP8) {
                                split_weights(p0, p1, p2, p3, hw[e / 4], mw[e / 4], lw[e / 4]);
                            } else {
                                hw[e / 2] = bf16x2_from_f32(p0, p1);
                                hw[e / 2 + 1] = bf16x2_from_f32(p2, p3);
                            }
                        }
                        // over columns that have been read
                        if (FP8) {      // 8 columns of each part
                            tmem_st8(st + (uint32_t)j0, hw);
                            tmem_st8(st + (uint32_t)j0 + 8u, mw);
                            tmem_st8(st + (uint32_t)j0 + 16u, lw);
                        } else {
                            tmem_st16(st + (uint32_t)(j0 / 2), hw);
                        }
                    }
                    float a, b;
                    unpack2(add2(sum0, sum1), a, b);
                    l += vis > 0 ? a + b : 0.0f;
                } else {
                    uint32_t z[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        z[j] = 0u;
                    tmem_st16(st, z);
                    tmem_st16(st + (FP8 ? 8u : 16u), z);
                    if (FP8) {          // 24 columns of each step
                        tmem_st16(st + 32u, z);
                        tmem_st16(st + 40u, z);
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&bar_p[half]));
            }
            if (!ok)
                *abort_flag = 1;
            ok = ok && warp_wait(smem_u32(&bar_o), nseg & 1u, abort_flag);
            // ---- output ----
            tc_fence_after();
            s_ok[half][quarter] = ok;
            pair_sync();                              // both halves are through
            ok = ok && s_ok[half ^ 1][quarter];
            const float top = seg.p1 > seg.p0 ? s_ref[row] : -INFINITY;
            s_row[half][row] = m == top ? l : l * exp2_approx(m - top);
            m = top;
            pair_sync();
            l = s_row[0][row] + s_row[1][row];
            pair_sync();                              // read before the next segment writes
            const bool empty = seg.p1 <= seg.p0;
            bool bad = !ok;                           // a row that the CTA could not finish
            if (!DENSE && !ok) {                      // and that sees anything
                bad = false;
                for (int e = 0; e < s_n; ++e)
                    bad = bad || ((u.sp.mask[e] >> qi) & 1u);
                m = bad ? m : -INFINITY;
                l = bad ? l : 0.0f;
            }
            const float vs = attn_v_scale(p, seg.c);
            const bool piece = DENSE || w.splits > 1;
            const float inv = piece ? vs * (1.0f / (1 << (int)kOff)) : l == 0.0f ? 0.0f : vs / l;
            l *= 1.0f / (1 << (int)kOff);             // the sum itself
            float *slot = nullptr, *dst = nullptr, *ml = nullptr;
            // output of row r of a piece
            auto piece_row = [&](int r) -> float * {
                return DENSE && seg.whole ? w.rows + (head_row_of(r) - w.q0 * p.hq) * (D + 4) : slot + r * D;
            };
            if (piece) {
                const int64_t sl = DENSE ? (seg.began ? (int64_t)gridDim.x : 0) + blockIdx.x : (int64_t)blockIdx.x;
                slot = w.pieces + sl * (int64_t)(w.slot_rows * (D + 2));
                dst = piece_row(row);
                ml = DENSE && seg.whole ? dst + D : slot + w.slot_rows * D + 2 * row;
                dst += half * kD2;
            }
            bool finite = true;
            // this warp's place for its half rows, in the query tile, which no MMA reads any more
            const uint32_t stage = qsm + (uint32_t)((half * 4 + quarter) * 32 * kD2 * 2);
#pragma unroll 1
            for (int j = 0; j < kD2; j += 16) {
                uint32_t o[16];
                if (ok && !empty) {
                    tmem_ld16(ot + (uint32_t)(half * kD2 + j), o);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float y = l == 0.0f ? 0.0f : __uint_as_float(o[e]) * inv;
                    finite = finite && fabsf(y) < INFINITY;
                    o[e] = __float_as_uint(bad ? nan : y);
                }
                if (piece) {
                    // 16 dims of 32 rows, through shared memory: four lanes a row
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        sts128(stage + (uint32_t)(lane * 64 + (((e / 4) ^ ((lane >> 1) & 3)) << 4)), o[e], o[e + 1], o[e + 2],
                               o[e + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = lane / 4; k < 32; k += 8) {
                        const int r = quarter * 32 + k;
                        uint4 y;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                                     : "r"(stage + (uint32_t)(k * 64 + (((lane & 3) ^ ((k >> 1) & 3)) << 4))));
                        if ((r >> w.gp_shift) < seg.nq && (r & (gp - 1)) < p.group)
                            *reinterpret_cast<uint4 *>(piece_row(r) + half * kD2 + j + (lane & 3) * 4) = y;
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        sts128(stage + (uint32_t)(lane * kD2 * 2 + ((((j + e) / 8) ^ (lane & (kD2 / 8 - 1))) << 4)),
                               bf16x2_from_f32(__uint_as_float(o[e]), __uint_as_float(o[e + 1])),
                               bf16x2_from_f32(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                               bf16x2_from_f32(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])),
                               bf16x2_from_f32(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
                }
            }
            tc_fence_before();
            if (piece) {
                if (real && half == 0) {
                    ml[0] = bad ? nan : m;
                    ml[1] = bad ? nan : l;
                }
            } else {
                if (real && half == 0 && p.lse)
                    p.lse[head_row()] = bad ? nan : attn_lse(m, l);
                __syncwarp();
                constexpr int kLanes = kD2 / 8;      // 16-byte pieces of a half row
                for (int r = lane / kLanes; r < 32; r += 32 / kLanes) {
                    const int rr = quarter * 32 + r, q2 = rr >> w.gp_shift, h2 = rr & (gp - 1), ch = lane % kLanes;
                    if (q2 < seg.nq && h2 < p.group) {
                        uint4 y;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                                     : "r"(stage + (uint32_t)(r * kD2 * 2 + ((ch ^ (r & (kLanes - 1))) << 4))));
                        const int64_t o = (w.q0 + seg.t0 + q2) * p.hq + seg.c * p.group + h2;
                        *reinterpret_cast<uint4 *>(p.out + o * D + half * kD2 + ch * 8) = y;
                    }
                }
                __syncwarp();
            }
            // ---- rows that values of tokens they do not see may have reached ----
            // (a row whose sum is NaN, from its own query or keys, has no other result)
            if (!DENSE && ok) {
                uint32_t again = __ballot_sync(0xffffffffu, real && !finite && l == l);
                while (again) {
                    const int src = __ffs(again) - 1;
                    again &= again - 1;
                    const int64_t hr2 = __shfl_sync(0xffffffffu, head_row(), src);
                    const int len2 = __shfl_sync(0xffffffffu, len, src), q2 = __shfl_sync(0xffffffffu, qi, src);
                    const float m2 = __shfl_sync(0xffffffffu, m, src), inv2 = __shfl_sync(0xffffffffu, inv, src);
                    float *dst2 = reinterpret_cast<float *>(__shfl_sync(0xffffffffu, (unsigned long long)dst, src));
                    float acc[kD2 / 32] = {};
                    for (int v = seg.p0; v < seg.p1; ++v) {
                        int e;
                        const int64_t tok0 = (int64_t)list_tile(v, e);
                        if (!((u.sp.mask[e] >> q2) & 1u))
                            continue;
                        for (int j = 0; j < 128 && tok0 + j < len2; ++j) {
                            const int32_t pg = attn_page(p, u.sp.toff[u.sp.block[e] >> 24], tok0 + j);
                            if (pg < 0)
                                continue;
                            const int64_t r = attn_page_row(p, tok0 + j);
                            const int64_t ko = (int64_t)pg * p.k.stride_page + seg.c * p.k.stride_head + r * p.k.stride_token;
                            const int64_t vo = (int64_t)pg * p.v.stride_page + seg.c * p.v.stride_head +
                                               r * p.v.stride_token + half * kD2;
                            float dot = 0.0f;
                            for (int d = lane; d < D; d += 32)
                                dot = fmaf(attn_value(p.k, ko + d), __uint_as_float((uint32_t)p.q[hr2 * D + d] << 16), dot);
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1)
                                dot += __shfl_xor_sync(0xffffffffu, dot, o);
                            const float wgt = exp2_approx(dot * ks - m2 + kOff);
#pragma unroll
                            for (int d = 0; d < kD2 / 32; ++d)
                                acc[d] = fmaf(wgt, attn_value(p.v, vo + lane + 32 * d), acc[d]);
                        }
                    }
#pragma unroll
                    for (int d = 0; d < kD2 / 32; ++d) {
                        if (dst2)
                            dst2[lane + 32 * d] = acc[d] * inv2;
                        else
                            p.out[hr2 * D + half * kD2 + lane + 32 * d] = attn_bf16(acc[d] * inv2);
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, S::kTmem);
    }
}

template <int D, bool FP8, bool DENSE>
cudaError_t launch_tiles(const AttnParams &p, const AttnTiles &w, const CUtensorMap &kmap, const CUtensorMap &vmap,
                         cudaStream_t stream)
{
    using S = TileShape<D, FP8>;
    const void *fn = reinterpret_cast<const void *>(&msa_attention_tile_kernel<D, FP8, DENSE>);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess)
        return e;
    void *args[] = {const_cast<AttnParams *>(&p), const_cast<AttnTiles *>(&w), const_cast<CUtensorMap *>(&kmap),
                    const_cast<CUtensorMap *>(&vmap)};
    return attn_launch(fn, w.ctas, kThreads, S::kSmem, stream, args);
}

template <int D>
cudaError_t launch_tiles_of(const AttnParams &p, const AttnTiles &w, const CUtensorMap &kmap, const CUtensorMap &vmap,
                            cudaStream_t stream)
{
    if (p.topk_ids)
        return p.k.fp8 ? launch_tiles<D, true, false>(p, w, kmap, vmap, stream)
                       : launch_tiles<D, false, false>(p, w, kmap, vmap, stream);
    return p.k.fp8 ? launch_tiles<D, true, true>(p, w, kmap, vmap, stream)
                   : launch_tiles<D, false, true>(p, w, kmap, vmap, stream);
}

}  // namespace

cudaError_t attn_tiles(const AttnParams &p, const AttnTiles &w, int head_dim, const CUtensorMap &kmap,
                       const CUtensorMap &vmap, cudaStream_t stream)
{
    return head_dim == 128 ? launch_tiles_of<128>(p, w, kmap, vmap, stream)
                           : launch_tiles_of<64>(p, w, kmap, vmap, stream);
}
