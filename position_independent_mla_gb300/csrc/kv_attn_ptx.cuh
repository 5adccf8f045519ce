// kv_attn_ptx.cuh -- what the attention kernels say in PTX: barriers, bulk copies,
// tensor memory, the tcgen05 MMAs, and the number formats of the cache.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "kv_serve.h"

namespace kvr {


__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_drop(uint32_t bar)
{
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_init_fence()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void bar_signal(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// `count` arrivals at once; the phase then also waits for `bytes` of bulk copies.
__device__ __forceinline__ void bar_signal_bulk(uint32_t bar, uint32_t count, uint32_t bytes)
{
    if (bytes)
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar),
                     "r"(bytes)
                     : "memory");
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Box of a tensor map at column x, row y; what lies outside the tensor is zero.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int y,
                                         uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}

// A box of a tensor map on its way to L2.
__device__ __forceinline__ void prefetch_box(const CUtensorMap *map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(x),
                 "r"(y)
                 : "memory");
}

// Signals `bar` when this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void bar_signal_copies(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Signals `bar` when every MMA the lead lane issued before has finished.
__device__ __forceinline__ void bar_signal_mma(uint32_t bar, uint32_t lead)
{
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
                 "r"(lead)
                 : "memory");
}

__device__ __forceinline__ uint32_t elect_lane()
{
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 "selp.b32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Bounded wait of a whole warp for a phase; false, for every lane, when it ran
// out here or elsewhere in the block (*abort).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                         int64_t limit_ns)
{
    if (__all_sync(0xFFFFFFFFu, bar_try(bar, parity)))
        return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 1; it < (1u << 26); ++it) {
        if (__all_sync(0xFFFFFFFFu, bar_try(bar, parity)))
            return true;
        if ((it & 15u) == 0u &&
            __any_sync(0xFFFFFFFFu, *abort != 0 || (int64_t)(global_ns() - t0) > limit_ns))
            break;
    }
    *abort = 1;
    return false;
}

__device__ __forceinline__ void mma_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mma_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int R>
__device__ __forceinline__ void reg_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

template <int R>
__device__ __forceinline__ void reg_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ void copy4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but this thread's newest N groups of copies have landed.
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void sts4(uint32_t dst, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(v) : "memory");
}

// A float at this block's address `src` in block `rank` of the cluster.
__device__ __forceinline__ float lds4_of(uint32_t src, uint32_t rank)
{
    float v;
    asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %1, %2;\n"
                 "ld.shared::cluster.f32 %0, [a];\n}"
                 : "=f"(v)
                 : "r"(src), "r"(rank)
                 : "memory");
    return v;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

__device__ __forceinline__ float lds4(uint32_t src)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(src) : "memory");
    return v;
}

// 16-byte copy to shared memory; bytes = 0 writes zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void sts16(uint32_t dst, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t src)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(src)
                 : "memory");
    return v;
}

// Columns of tensor memory for the block, by one warp; the address is left at `to`.
__device__ __forceinline__ void tmem_alloc(uint32_t to, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}

#define KV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), \
                    "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define KV_P8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), \
                    "+r"(a[i + 5]), "+r"(a[i + 6]), "+r"(a[i + 7])
#define KV_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), \
                    "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of this thread's tensor-memory lane (no wait).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : KV_R8(r, 0), KV_R8(r, 8), KV_R8(r, 16), KV_R8(r, 24)
                 : "r"(addr));
}

// Uses of r stay behind the wait that comes before this.
__device__ __forceinline__ void tmem_pin32(uint32_t *r)
{
    asm volatile("" : KV_P8(r, 0), KV_P8(r, 8), KV_P8(r, 16), KV_P8(r, 24));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::KV_W8(r, 0),
                 KV_W8(r, 8), KV_W8(r, 16), KV_W8(r, 24), "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : KV_R8(r, 0), KV_R8(r, 8)
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_pin16(uint32_t *r)
{
    asm volatile("" : KV_P8(r, 0), KV_P8(r, 8));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::KV_W8(r, 0),
                 KV_W8(r, 8), "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand in panels of 64 bf16 columns: rows of 128 bytes, the
// 16-byte piece c of row r at c ^ (r & 7) (128-byte swizzle), 1024 bytes per
// eight rows.  Along a K-major operand the next 16 columns are 32 bytes on;
// of an MN-major one (V: the MMA's N runs along the row) the next 16 keys are
// 2048 bytes on and the next 64 columns `lead` bytes.  The low word holds the
// address, in units of 16 bytes, and the lead; the high word is the same for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t lead)
{
    return ((addr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}

constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

// kind::f16: D fp32, A and B bf16; each along K (0) or along M / N (1).
template <int N, int BMAJOR, int AMAJOR = 0>
__device__ __forceinline__ constexpr uint32_t mma_desc()
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)AMAJOR << 15) | ((uint32_t)BMAJOR << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

// The MMA warp runs as one: every lane holds the same operands (they stay in
// uniform registers) and the lane with `lead` set issues.
template <int N, int MAJOR = 0>
__device__ __forceinline__ void mma_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t acc,
                                         uint32_t lead, uint32_t b_high = kOperandHigh)
{
    asm volatile("{\n.reg .pred p, q;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\n"
                 "setp.ne.b32 q, %6, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %7};\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d),
                 "r"(a), "r"(b), "r"(mma_desc<N, MAJOR, MAJOR>()), "r"(acc), "r"(kOperandHigh),
                 "r"(lead), "r"(b_high)
                 : "memory");
}

// kind::f8f6f4: D fp32, A e4m3, B e5m2.
template <int N, int MAJOR>
__device__ __forceinline__ void mma_smem_8bit(uint32_t d, uint32_t a, uint32_t b, uint32_t acc,
                                              uint32_t lead, uint32_t b_high)
{
    constexpr uint32_t desc = (1u << 4) | (1u << 10) | ((uint32_t)MAJOR << 15) | ((uint32_t)MAJOR << 16) |
                              ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
    asm volatile("{\n.reg .pred p, q;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\n"
                 "setp.ne.b32 q, %6, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %7};\n"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n}" ::"r"(d),
                 "r"(a), "r"(b), "r"(desc), "r"(acc), "r"(kOperandHigh), "r"(lead), "r"(b_high)
                 : "memory");
}

template <int N, int BMAJOR>
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t acc,
                                         uint32_t lead)
{
    asm volatile("{\n.reg .pred p, q;\n.reg .b64 y;\nsetp.ne.b32 p, %4, 0;\n"
                 "setp.ne.b32 q, %6, 0;\nmov.b64 y, {%2, %5};\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d),
                 "r"(a), "r"(b), "r"(mma_desc<N, BMAJOR>()), "r"(acc), "r"(kOperandHigh), "r"(lead)
                 : "memory");
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// 32 bytes, aligned so: a whole sector of a row.
__device__ __forceinline__ void st32(void *to, const uint32_t *r)
{
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::KV_W8(r, 0), "l"(to)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 values (bytes 1 and 3 of y) to a bf16 pair, times `mul`.  Moved into
// a bf16's exponent and top mantissa bits a value reads 2^-120 of itself,
// subnormal ones included, so one exact product with 2^120 * scale puts it right.
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t y, uint32_t mul)
{
    uint32_t b = (y & 0x80008000u) | ((y >> 4) & 0x07F007F0u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(b), "r"(mul));
    return b;
}

// A value of 0x7F or 0xFF (NaN) among four e4m3 values sets a bit.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Scale 2^e of a row as the multiplier pairs of convert16: 2^(120 + min(e, 7)),
// the largest that bf16 holds, and what is left of e (1 but for huge rows).
__device__ __forceinline__ uint32_t scale_mul(float scale)
{
    const int e = (int)(__float_as_uint(scale) >> 23) - 127;
    return (uint32_t)(247 + min(e, 7)) << 7 | (uint32_t)(127 + max(e - 7, 0)) << 23;
}

// A 16-byte piece needs convert_rare: it holds a NaN, or its scale is above 2^7.
__device__ __forceinline__ uint32_t rare16(uint4 v, uint32_t mul)
{
    return e4m3_nan(v.x) | e4m3_nan(v.y) | e4m3_nan(v.z) | e4m3_nan(v.w) |
           ((mul >> 16) ^ 0x3F80u);
}

// Sixteen e4m3 values (one 16-byte piece) to two pieces of bf16.  RARE: with the
// second factor of the scale, and NaN.  The callers test a whole batch of pieces
// first, so that the usual form is free of branches and its chains interleave.
template <bool RARE>
__device__ __forceinline__ void convert16(uint4 v, uint32_t mul, uint4 &lo, uint4 &hi)
{
    const uint32_t m = __byte_perm(mul, 0, 0x1010);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = e4m3_bf16(__byte_perm(w[i], 0, 0x1404), m);
        r[2 * i + 1] = e4m3_bf16(__byte_perm(w[i], 0, 0x3424), m);
    }
    if constexpr (RARE) {
        const uint32_t m2 = __byte_perm(mul, 0, 0x3232);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(r[i]), "r"(m2));
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (((w[i >> 2] >> ((i & 3) * 8)) & 0x7Fu) == 0x7Fu)
                r[i >> 1] |= (i & 1) ? 0x7FC00000u : 0x7FC0u;
    }
    lo = make_uint4(r[0], r[1], r[2], r[3]);
    hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// Sets bit 15 or 31 when the low or the high bf16 of a pair is not finite.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w)
{
    return (w & 0x7F807F80u) + 0x00800080u;
}

// The pair with values that are not finite zeroed.
__device__ __forceinline__ uint32_t finite2(uint32_t w)
{
    const uint32_t n = nonfinite2(w);
    return w & ((n & 0x8000u) ? 0xFFFF0000u : ~0u) & ((n & 0x80000000u) ? 0xFFFFu : ~0u);
}

} // namespace kvr
