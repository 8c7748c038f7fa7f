// Barrier, shared-memory and tensor-core helpers of the attention kernels (not
// exported).
#pragma once

#include "msa_internal.h"

#include <cstdint>

namespace {

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// The lagging test build (MSA_LAG) makes one warp of several fall 20 us behind after an
// exchange through shared memory; nothing in the product.
__device__ __forceinline__ void test_lag(bool warp)
{
#ifdef MSA_LAG
    if (warp)
        __nanosleep(20000);
#else
    (void)warp;
#endif
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same, asleep for up to 20 us: a warp that polls takes issue slots from the others.
__device__ __forceinline__ bool mbar_try_asleep(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000)
        : "memory");
    return ok != 0;
}

// true once the phase with the given parity has completed; false after the limit
// (MSA_WAIT_LIMIT_NS, 2 s)
__device__ __noinline__ bool mbar_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer();
    do
        if (mbar_try_asleep(bar, parity))
            return true;
    while (globaltimer() - t0 <= MSA_WAIT_LIMIT_NS);
    return false;
}

// A whole warp waits; false (and the CTA's abort flag set) when the wait ran out or
// another warp gave up.  The flag is read only when the phase is not complete yet.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (__all_sync(0xffffffffu, mbar_try(bar, parity)))
        return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0))
        return false;
    if (__all_sync(0xffffffffu, mbar_wait(bar, parity)))
        return true;
    *abort_flag = 1;
    return false;
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t x)
{
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Generic writes to shared memory made visible to the tensor cores and TMA.
__device__ __forceinline__ void fence_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Byte offset within a tile of rows of SWB bytes (64 or 128) under the SWB-byte swizzle:
// the 16-byte chunk index is XORed with the row index of the 1,024- or 512-byte pattern.
template <int SWB>
__device__ __forceinline__ uint32_t swizzle(uint32_t off)
{
    return off ^ ((off >> 3) & (SWB == 128 ? 0x70u : 0x30u));
}

// Shared-memory matrix descriptor.  swizzle_bytes 0, 64 or 128; lbo and sbo in bytes:
//   K-major, swizzled   sbo = 8 rows, lbo unused;
//   MN-major, swizzled  lbo = the next swizzle-wide piece along M or N, sbo = 8 steps
//                       along K;
//   MN-major, none      sbo = the next 16 bytes along M or N, lbo = 8 steps along K.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, int swizzle_bytes, uint32_t lbo, uint32_t sbo)
{
    uint64_t d = (uint64_t)((addr & 0x3FFFF) >> 4);
    d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(swizzle_bytes == 128 ? 2 : swizzle_bytes == 64 ? 4 : 0) << 61;
    return d;
}

// Instruction descriptor: fp32 accumulators; 8-bit (kind::f8f6f4: 0 E4M3, 1 E5M2) or bf16
// (kind::f16: 1) operands; an operand is K-major unless its mn flag is set.
__host__ __device__ constexpr uint32_t mma_idesc(uint32_t a_type, uint32_t b_type, int m, int n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (a_type << 7) | (b_type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One MMA by an elected lane of a converged warp, both operands in shared memory.
template <bool FP8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (FP8)
        asm volatile(
            "{\n\t.reg .pred pp, pe;\n\telect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pp, %4, 0;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, pp;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred pp, pe;\n\telect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pp, %4, 0;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pp;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Four MMAs in a row, whose operands lie AS and BS apart (in descriptor units of 16 bytes;
// for A in tensor memory, columns): one election, and operands made in place, since the
// issue of an MMA costs its warp several times the instructions that describe it.
template <bool FP8, int AS, int BS>
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (FP8)
        asm volatile(
            "{\n\t.reg .pred pp, pe;\n\t.reg .b64 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pp, %4, 0;\n\t"
            "add.u64 a1, %1, %5;\n\tadd.u64 b1, %2, %6;\n\t"
            "add.u64 a2, a1, %5;\n\tadd.u64 b2, b1, %6;\n\t"
            "add.u64 a3, a2, %5;\n\tadd.u64 b3, b2, %6;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, pp;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(AS), "n"(BS)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred pp, pe;\n\t.reg .b64 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pp, %4, 0;\n\t"
            "add.u64 a1, %1, %5;\n\tadd.u64 b1, %2, %6;\n\t"
            "add.u64 a2, a1, %5;\n\tadd.u64 b2, b1, %6;\n\t"
            "add.u64 a3, a2, %5;\n\tadd.u64 b3, b2, %6;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pp;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(AS), "n"(BS)
            : "memory");
}

template <bool FP8, int AS, int BS>
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (FP8)
        asm volatile(
            "{\n\t.reg .pred pp, pe;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pp, %4, 0;\n\t"
            "add.u32 a1, %1, %5;\n\tadd.u64 b1, %2, %6;\n\t"
            "add.u32 a2, a1, %5;\n\tadd.u64 b2, b1, %6;\n\t"
            "add.u32 a3, a2, %5;\n\tadd.u64 b3, b2, %6;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, pp;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a1], b1, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a2], b2, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(AS), "n"(BS)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred pp, pe;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pp, %4, 0;\n\t"
            "add.u32 a1, %1, %5;\n\tadd.u64 b1, %2, %6;\n\t"
            "add.u32 a2, a1, %5;\n\tadd.u64 b2, b1, %6;\n\t"
            "add.u32 a3, a2, %5;\n\tadd.u64 b3, b2, %6;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pp;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n\t"
            "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(AS), "n"(BS)
            : "memory");
}

// Six 8-bit MMAs with A in tensor memory: three parts, 8 columns apart, against one B, and
// three parts 32 columns further against the B that is BS further.
template <int BS>
__device__ __forceinline__ void mma_ts33(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred pp, pe;\n\t.reg .b32 a1, a2, a3, a4, a5;\n\t.reg .b64 b1;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\tsetp.ne.b32 pp, %4, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u64 b1, %2, %5;\n\t"
        "add.u32 a3, %1, 32;\n\tadd.u32 a4, %1, 40;\n\tadd.u32 a5, %1, 48;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, pp;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a1], %2, %3, 1;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a2], %2, %3, 1;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a3], b1, %3, 1;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a4], b1, %3, 1;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a5], b1, %3, 1;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(BS)
        : "memory");
}

// Arrives on `bar` when every MMA this warp's elected lane has issued is complete.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred pe;\n\telect.sync _|pe, 0xffffffff;\n\t"
        "@pe tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// A box of a cache map (dims, rows of a page, heads, pages) into shared memory; a page
// at or past the map's extent fills the box with zeros.  The bytes are counted on `bar`.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t row,
                                             int32_t head, int32_t page, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (x0, x1) -> two E4M3 codes, x0 in the low byte; round to nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float x0, float x1)
{
    unsigned short c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x1), "f"(x0));
    return (uint32_t)c;
}

// Four weights (0 to 2^15) -> three E5M2 parts, four codes each, whose sum is the weight to
// 2^-9 + 2^-11 of itself or 2^-17, whichever is more: no weight has to be small against its
// row's largest (two E4M3 parts, of 2^-8, lost what was below 2^-14 of it).  E5M2 is the upper
// byte of f16, so the first two parts are cut out of f16, each taking three bits, and
// subtracted exactly; the last is rounded.
__device__ __forceinline__ void split_weights(float x0, float x1, float x2, float x3, uint32_t &hi, uint32_t &mid,
                                              uint32_t &lo)
{
    asm("{\n\t.reg .b32 p, q, b, c;\n\t.reg .b16 l0, l1;\n\t"
        "cvt.rn.f16x2.f32 p, %4, %3;\n\t"
        "cvt.rn.f16x2.f32 q, %6, %5;\n\t"
        "prmt.b32 %0, p, q, 0x7531;\n\t"
        "and.b32 b, p, 0xff00ff00;\n\t"
        "and.b32 c, q, 0xff00ff00;\n\t"
        "sub.rn.f16x2 p, p, b;\n\t"
        "sub.rn.f16x2 q, q, c;\n\t"
        "prmt.b32 %1, p, q, 0x7531;\n\t"
        "and.b32 b, p, 0xff00ff00;\n\t"
        "and.b32 c, q, 0xff00ff00;\n\t"
        "sub.rn.f16x2 p, p, b;\n\t"
        "sub.rn.f16x2 q, q, c;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 l0, p;\n\t"
        "cvt.rn.satfinite.e5m2x2.f16x2 l1, q;\n\t"
        "mov.b32 %2, {l0, l1};\n\t}"
        : "=&r"(hi), "=&r"(mid), "=r"(lo)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
}

// (x0, x1) -> a bf16 pair, x0 in the low half
__device__ __forceinline__ uint32_t bf16x2_from_f32(float x0, float x1)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x1), "f"(x0));
    return d;
}

}  // namespace
