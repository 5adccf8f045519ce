// kv_attention.cu -- attention of new tokens over the paged cache on the
// 5th-generation tensor cores (tcgen05).
//
//     S = scale * Q Kᵀ,  O = softmax(S) V,  lse = log Σ exp(S)
//
// for one layer of a paged pool, with one pass over the keys: for a tile of
// keys the running maximum m and sum l of every query row are updated, the
// weights 2^((s - m) * scale * log2 e) are rounded to bf16 and multiplied with
// V onto the accumulator O, which is rescaled when m moves.
//
// Rows.  The query heads that share a key head are packed with the tokens:
// row r of a (sequence, key head) is token r / group, head r % group, and a
// block owns NT tiles of 128 rows (the M of one MMA).  So 32 query heads of one
// new token over 8 key heads read each key once, and a chunk of many tokens
// fills whole tiles.
//
// Roles of a block's warps:
//   softmax  8 a row tile, two threads to a row, one for each half of its keys: read
//            the row of S from tensor memory, mask, keep m and l in registers,
//            write the bf16 weights back over S (they are the A operand of the
//            second MMA) and at the end O / l.  They vote for every tile whether a
//            maximum has outgrown its reference, and exchange maxima only then;
//   load     bring rows of the pool through the block table into shared memory
//            in the 128-byte swizzled layout that the MMAs read;
//   mma      one warp issues every MMA.
// O stays in tensor memory.  It is rescaled only when some row's maximum grew by
// more than 2^8 since it was last fixed: until then the weights stay below 2^8,
// which fp32 sums and bf16 weights hold without loss.
//
// Long axes are split: blocks take runs of `split_tiles` key tiles of a row
// tile, write normalised fp32 parts with their lse, and a second kernel joins
// them.  The split depends only on sizes, so results repeat bit for bit.
//
// Every wait is bounded; a block whose wait runs out reports KV_ERR_TIMEOUT.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "kv_serve.h"

namespace kvr {

namespace {

constexpr int kRows = 128;         // rows per tile: the M of an MMA
constexpr int64_t kExpandBytes = int64_t(2) << 30; // largest workspace for widened rows
constexpr float kLazy = 8.0f;      // log2 of the growth of a maximum that O tolerates

// ---------------------------------------------------------------------------
// PTX pieces
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
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

// kind::f8f6f4: D fp32, A and B e4m3.
template <int N, int MAJOR>
__device__ __forceinline__ void mma_smem_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t acc,
                                              uint32_t lead, uint32_t b_high)
{
    constexpr uint32_t desc = (1u << 4) | ((uint32_t)MAJOR << 15) | ((uint32_t)MAJOR << 16) |
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

// ---------------------------------------------------------------------------
// Geometry
// ---------------------------------------------------------------------------

// Head rows: K and V tiles of 128 keys x 128, a ring of stages.
template <bool QUANT_, int NT_>
struct HeadGeo {
    static constexpr bool MLA = false, QUANT = QUANT_;
    static constexpr int NT = NT_, KT = 128;
    static constexpr int QPANELS = 2, OC = 128;    // query panels in shared memory; columns of O
    static constexpr int DV = 128;
    static_assert(NT == 1 || !QUANT, "e4m3 rows are widened before two row tiles read them");
    static constexpr int SOFT_WARPS = 8 * NT, LOAD_WARPS = NT == 2 ? 4 : 8;
    static constexpr int STAGE = 2 * 128 * 128;    // bytes of a K or V tile
    // e4m3: RAW tiles of K or V as they are stored, and their scales, wait in
    // shared memory to be converted
    static constexpr int RAW = QUANT ? 5 : 0;
    static constexpr int STAGES = QUANT ? 3 : NT == 2 ? 4 : 5;
    static constexpr int BARS = 2 * STAGES;
    static constexpr int RAW_AT = STAGES * STAGE, RAW_STAGE = STAGE / 2 + 512;
    static constexpr int RING = RAW_AT + RAW * RAW_STAGE;
    // columns of tensor memory: S (and P over it) per tile or per buffer, O
    static constexpr int S_COL(int i) { return i * 128; }
    static constexpr int O_COL(int t) { return 256 + t * 128; }
};

// MLA rows: a tile of 64 latent rows is both K (9 panels: 512 + 64 columns) and
// V; a block makes one half of the 512 value columns (O of 128 x 512 fp32 would
// fill tensor memory).  The value panels of this half (4) serve both products
// and live longer than the other 5 panels, so they have rings of their own, two tiles
// each, and are halved again: the values' product of one pair of panels frees them while
// the other pair's runs.  Query panels: those of this half stay in tensor memory
// (they fit beside O and two S), the other five in shared memory.
template <bool QUANT_>
struct MlaGeo {
    static constexpr bool MLA = true, QUANT = QUANT_;
    static constexpr int NT = 1, KT = 64;
    static constexpr int QPANELS = 5, OC = 256;
    static constexpr int DV = 512;
    // e4m3 rows are converted by the load warps: twice as many
    static constexpr int SOFT_WARPS = 8, LOAD_WARPS = QUANT ? 16 : 8;
    static constexpr int PANEL = 64 * 128;
    static constexpr int OTHER = 5 * PANEL, OWN = 4 * PANEL; // bytes of a tile's parts
    static constexpr int PARTS = 3; // the other half and k_pe; two pairs of this half
    static constexpr int BARS = 4 * PARTS; // full, empty of two stages of each
    static constexpr int RING = 2 * (OTHER + OWN);
    static constexpr int S_COL(int i) { return 256 + i * 64; }
    static constexpr int O_COL(int) { return 0; }
    static constexpr int Q_COL = 384;
    __device__ static uint32_t part(uint32_t ring, int which, int i)
    {
        return ring + (which == 0 ? i * OTHER : 2 * OTHER + i * OWN + (which - 1) * 2 * PANEL);
    }
};

template <class G>
constexpr int kMmaWarp = G::SOFT_WARPS + G::LOAD_WARPS;

// Two row tiles: 16 softmax warps that hold 64 scores a thread need more registers than
// the other roles, which give some back; whole warpgroups, then.
template <class G>
constexpr bool kShares = G::NT == 2;

constexpr int kSoftRegs = 96, kLoadRegs = 56, kMmaRegs = 40;

template <class G>
constexpr int kAttnThreads = (kMmaWarp<G> + (kShares<G> ? 4 : 1)) * 32;

template <class G>
struct Smem {
    static constexpr int Q = 0;                                  // [NT][QPANELS][128 rows][128 B]
    static constexpr int RING = G::NT * G::QPANELS * 128 * 128;  // K and V
    static constexpr int BAR = RING + G::RING;                   // barriers
    // q, out; then per tile or buffer: S ready, P ready; O steps; then the ring's
    static constexpr int NBARS = 8 + G::BARS;
    static constexpr int BYTES = BAR + NBARS * 8 + 1024;         // + alignment of the base
};

enum { kBarQ = 0, kBarDone = 1, kBarS = 2, kBarP = 4, kBarO = 6, kBarRing = 8 };

// What a block works on, the same for every thread.
struct Work {
    int seq, head;       // sequence, key head (MLA: half of the value columns)
    int n, len;          // new tokens, cached tokens
    int64_t q0;          // first query token of the sequence
    int row0;            // first row of the block within (sequence, key head)
    int beg, end;        // virtual key tiles of this block
    int sink_tiles;      // virtual tile v < sink_tiles is tile v, else first + v - sink_tiles
    int first;
    int lo, hi, sk;      // keys that some row sees: [lo, hi) and [0, sk)
    int split, splits;
};

// Mask of the rows of one 128-row tile.
struct TileMask {
    int pos0, pos1;      // positions of the first and last token
    int hi0, hi1;        // first key not seen by the first / last token
    int lo0, lo1;        // first key in the window of the first / last token
    int sk;              // sinks outside the last token's window
    int rows;            // rows that exist
};

__device__ __forceinline__ TileMask tile_mask(const AttnParams &p, int n, int len, int row0)
{
    TileMask m;
    const int total = n * p.group;
    m.rows = max(0, min(kRows, total - row0));
    const int i0 = p.by_group.quotient(row0);
    const int i1 = p.by_group.quotient(row0 + max(m.rows, 1) - 1);
    m.pos0 = len - n + i0;
    m.pos1 = len - n + i1;
    m.hi0 = p.causal ? max(0, min(len, m.pos0 + 1)) : len;
    m.hi1 = p.causal ? max(0, min(len, m.pos1 + 1)) : len;
    m.lo0 = p.window ? max(0, m.pos0 - p.window + 1) : 0;
    m.lo1 = p.window ? max(0, m.pos1 - p.window + 1) : 0;
    m.sk = p.window ? min(p.sinks, m.lo1) : 0;
    return m;
}

// Key tile kt has a key that some row of the tile sees.
template <int KT>
__device__ __forceinline__ bool tile_active(const TileMask &m, int kt)
{
    const int k0 = kt * KT;
    return m.rows > 0 && k0 < m.hi1 && (k0 + KT > m.lo0 || k0 < m.sk);
}

// Every row of the tile sees every key of tile kt.
template <int KT>
__device__ __forceinline__ bool tile_full(const AttnParams &p, const TileMask &m, int kt)
{
    const int k0 = kt * KT;
    return k0 + KT <= m.hi0 && (k0 >= m.lo1 || k0 + KT <= p.sinks);
}

// The key range of the rows of a block and its virtual tiles: returns their
// number.
template <int KT, int NT>
__device__ __forceinline__ int key_tiles(const AttnParams &p, Work &w)
{
    const TileMask a = tile_mask(p, w.n, w.len, w.row0);
    TileMask b = a;
    if (NT == 2) {
        const TileMask c = tile_mask(p, w.n, w.len, w.row0 + kRows);
        if (c.rows > 0)
            b = c;
    }
    w.lo = a.lo0;
    w.hi = b.hi1;
    w.sk = p.window ? min(p.sinks, w.lo) : 0;
    w.first = w.lo / KT;
    w.sink_tiles = min((w.sk + KT - 1) / KT, w.first);
    return w.hi <= 0 ? 0 : w.sink_tiles + max(0, (w.hi + KT - 1) / KT - w.first);
}

__device__ __forceinline__ int real_tile(const Work &w, int v)
{
    return v < w.sink_tiles ? v : w.first + v - w.sink_tiles;
}

// The block's share of nv key tiles: as many equal runs as runs of split_tiles would be.
// False where there is none.
__device__ __forceinline__ bool take_split(const AttnParams &p, int nv, Work &w)
{
    w.splits = max(1, p.by_run.quotient(nv + p.split_tiles - 1));
    const int run = w.splits == 1 ? nv : (nv + w.splits - 1) / w.splits;
    w.beg = min(nv, w.split * run);
    w.end = min(nv, w.beg + run);
    return w.split < w.splits;
}

// Lengths of sequence s; false when they do not fit what the call stated.
__device__ __forceinline__ bool seq_queries(const AttnParams &p, int s, int64_t &q0, int &n)
{
    const int a = p.q_off[s], b = p.q_off[s + 1];
    q0 = a;
    n = b - a;
    if (a < 0 || b < a || b > p.total_q || n > p.max_q_len) {
        n = 0;
        return false;
    }
    return true;
}

__device__ __forceinline__ bool seq_keys(const AttnParams &p, int s, int &len)
{
    len = p.kv_len[s];
    return len >= 0 && len <= p.max_kv_len && (int64_t)len <= p.max_keys;
}

// Row tile `tile` of the call -> sequence, its queries and keys, and the row tile
// within it: one warp counts the sequences' tiles 32 at a time.  Returns false past
// the last tile or for a sequence whose keys do not fit; `bad`: some sequence's
// offsets, or this one's keys, do not fit what the call stated.
template <int ROWS>
__device__ __forceinline__ bool find_tile(const AttnParams &p, int tile, int lane, Work &w, int &at,
                                          bool &bad)
{
    int before = 0;
    bool found = false, wrong = false, keys = false;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
        int n = 0, tiles = 0, len = 0;
        int64_t q0 = 0;
        bool fits = false;
        if (s0 + lane < p.num_seqs) {
            fits = seq_keys(p, s0 + lane, len);
            if (!seq_queries(p, s0 + lane, q0, n))
                wrong = true;
            tiles = (n * p.group + ROWS - 1) / ROWS;
        }
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d)
                sum += o;
        }
        const bool mine = !found && tile >= before + sum - tiles && tile < before + sum;
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine);
        if (who) {
            const int l = __ffs((int)who) - 1;
            w.seq = s0 + l;
            w.n = __shfl_sync(0xFFFFFFFFu, n, l);
            w.len = __shfl_sync(0xFFFFFFFFu, len, l);
            w.q0 = __shfl_sync(0xFFFFFFFFu, q0, l);
            keys = __shfl_sync(0xFFFFFFFFu, (int)fits, l) != 0;
            // the last tiles of a causal chunk see the most keys: first
            const int t = __shfl_sync(0xFFFFFFFFu, tiles, l), e = __shfl_sync(0xFFFFFFFFu, sum, l);
            at = t - 1 - (tile - (before + e - t));
            found = true;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    bad = __any_sync(0xFFFFFFFFu, wrong) || (found && !keys);
    return found && keys;
}

__device__ __forceinline__ bool key_seen(const Work &w, int k)
{
    return k < w.hi && (k >= w.lo || k < w.sk);
}

// Block id of key k of the block's sequence (anything for keys that no row sees).
// The load roles ask for it well before they use it: the first use waits.
__device__ __forceinline__ int32_t key_block(const AttnParams &p, const Work &w, int k)
{
    const int b = p.by_block.quotient(k);
    return key_seen(w, k) ? __ldg(p.block_tables + (int64_t)w.seq * p.max_blocks + b) : 0;
}

// Slot of key k in block `blk`, or -1: not seen by any row, or (bad) the block
// lies outside the pool.
__device__ __forceinline__ int64_t key_slot(const AttnParams &p, const Work &w, int k, int32_t blk,
                                            bool &bad)
{
    if (!key_seen(w, k))
        return -1;
    if (blk < 0 || blk >= p.num_blocks) {
        bad = true;
        return -1;
    }
    return (int64_t)blk * p.block + (k - p.by_block.quotient(k) * p.block);
}

// ---------------------------------------------------------------------------
// Load roles
// ---------------------------------------------------------------------------

// Query rows of row tile t into their panels, by the tile's 256 softmax threads; rows
// past the end are zeros.  A group of threads takes whole panels of a row, then the
// row `step` further on, so one division finds token and head of the first.
template <class G>
__device__ __forceinline__ void load_queries(const AttnParams &p, const Work &w, uint32_t q_smem,
                                             int t, int tid)
{
    constexpr int LANES = G::MLA ? 8 : 16, step = 256 / LANES;
    const int c = tid & (LANES - 1);
    const int row = w.row0 + t * kRows + tid / LANES;
    int tok = p.by_group.quotient(row), g = row - tok * p.group;
    const int dt = p.by_group.quotient(step), dg = step - dt * p.group;
    const uint32_t dst = q_smem + ((t * G::QPANELS + (c >> 3)) << 14);
    for (int rr = tid / LANES; rr < kRows; rr += step) {
        const uint32_t n = tok < w.n ? 16u : 0u;
        const int h = G::MLA ? g : w.head * p.group + g;
        const char *src = p.q + (n ? (w.q0 + tok) * p.q_ts + h * p.q_hs : 0) + c * 16;
        const uint32_t to = dst + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
        if constexpr (G::MLA) { // the other half's panels, then k_pe's
#pragma unroll
            for (int i = 0; i < 4; ++i)
                copy16(to + (i << 14), src + (1 - w.head) * 512 + i * 128, n);
            copy16(to + (4 << 14), src + 1024, n);
        } else {
            copy16(to, src, n);
        }
        tok += dt;
        g += dg;
        if (g >= p.group) {
            g -= p.group;
            ++tok;
        }
    }
}

// Every key of tile kt is seen by some row: its rows can be copied as they are.
template <int KT>
__device__ __forceinline__ bool tile_whole(const Work &w, int kt)
{
    const int k0 = kt * KT;
    return (k0 >= w.lo && k0 + KT <= w.hi) || k0 + KT <= w.sk;
}

// Waits for the boxes that may be in flight when `filled` tiles went into a ring, also
// when the block gives up early: its shared memory goes after that.
template <int STAGES>
__device__ __forceinline__ void copies_land(uint32_t full, int filled)
{
    int none = 0;
    for (int i = 0; i < STAGES; ++i)
        if (filled > i)
            bar_wait(full + i * 8, ((filled - 1 - i) / STAGES) & 1, &none, 10000000ll);
}

// Stages filled by cp.async: their threads wait for the copies, make them visible to
// the MMAs and signal, one stage behind the one that they are filling.
struct Copies {
    uint32_t full = 0; // barrier of the stage that is not signalled yet

    __device__ void flush()
    {
        if (full) {
            copy_wait<0>();
            async_fence();
            bar_signal(full);
            full = 0;
        }
    }

    __device__ void filled(uint32_t bar)
    {
        copy_commit();
        if (full) {
            copy_wait<1>();
            async_fence();
            bar_signal(full);
        }
        full = bar;
    }

    // before a wait for a stage: nobody waits for this one meanwhile
    __device__ void before_wait(uint32_t empty, uint32_t parity)
    {
        if (full && !__all_sync(0xFFFFFFFFu, bar_try(empty, parity)))
            flush();
    }
};

// A vote over the load warps, also their meeting point.
template <class G>
__device__ __forceinline__ bool load_any(bool x)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 q, %1, 0;\n"
                 "barrier.cta.red.or.pred p, 15, %2, q;\nselp.b32 %0, 1, 0, p;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)x), "n"(G::LOAD_WARPS * 32)
                 : "memory");
    return r != 0;
}

// Head rows into the ring as they are stored.  Whole tiles are boxes of the
// tensor maps that one warp asks for (a box is at most a block of the pool), a run
// of tiles in a loop of few instructions: a tile's boxes have to go out within the
// time of its MMAs.  Tiles that hold keys nobody sees, and pools whose blocks do
// not divide a tile, are copied row by row by all warps with zeros in the place of
// those keys: a lane owns one key row of its warp, 16 lanes copy 256 bytes (8 lanes
// 128).  The warps meet after every run, so none waits for a stage that is more than
// one phase away, which a parity would not show; a warp whose wait ran out goes on to
// the next meeting, where they all give up.
template <class G>
__device__ __forceinline__ void load_heads(const AttnParams &p, const Work &w, uint32_t ring,
                                           uint32_t bars, int warp, int lane,
                                           volatile int *abort, bool &bad)
{
    constexpr int WARPS = G::LOAD_WARPS, ROWS = G::KT / WARPS; // rows of a warp: 32 or 16
    constexpr int PIECES = G::STAGE / G::KT / 16, PER = 32 / PIECES; // of a row; rows at a time
    const int base = warp * ROWS;
    const int c = lane & (PIECES - 1), sub = lane / PIECES;
    const int32_t *const table = p.block_tables + (int64_t)w.seq * p.max_blocks;
    auto whole = [&](int v) { return p.box_rows > 0 && tile_whole<G::KT>(w, real_tile(w, v)); };
    Copies copies;
    int stage = 0, phase = 1, filled = 0;
    bool ok = true;
    auto next = [&] {
        ++filled;
        if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1;
        }
    };
    for (int v = w.beg; v < w.end;) {
        if (whole(v)) {
            int last = v + 1;
            while (last < w.end && whole(last))
                ++last;
            copies.flush();
            if (warp == 0) {
                // a tile is `per` blocks, or a part of one
                const int per = G::KT / p.box_rows, in = p.block / p.box_rows;
                const bool mine = lane < per;
                auto block_of = [&](int kt) { return in == 1 ? kt * per + lane : kt / in; };
                int kt = real_tile(w, v);
                int32_t blk = mine ? __ldg(table + block_of(kt)) : 0;
                for (int u = v; ok && u < last; ++u) {
                    const int row = (in == 1 ? 0 : (kt % in) * G::KT) + blk * p.block;
                    const bool fits = (uint32_t)blk < (uint32_t)p.num_blocks;
                    bad |= !fits;
                    const int y = fits ? row : (int)(p.num_blocks * p.block); // else zeros
                    kt = real_tile(w, u + 1);
                    if (mine && u + 1 < last)
                        blk = __ldg(table + block_of(kt));
#pragma unroll
                    for (int part = 0; part < 2; ++part) { // K, then V
                        const uint32_t full = bars + stage * 8;
                        ok = ok && bar_wait(full + G::STAGES * 8, phase, abort, p.wait_limit_ns);
                        if (!ok)
                            break;
                        if (lane == 0)
                            bar_signal_bulk(full, WARPS * 32, G::STAGE);
                        if (mine) {
                            const CUtensorMap *map = part == 0 ? &p.rot_map : &p.copy_map;
                            const uint32_t at = ring + stage * G::STAGE + lane * p.box_rows * 128;
                            copy_box(at, map, w.head * 128, y, full);
                            if (PIECES == 16) // 64 columns of bf16 to a box
                                copy_box(at + 16384, map, w.head * 128 + 64, y, full);
                        }
                        next();
                    }
                }
            } else { // where warp 0 will be
                filled += 2 * (last - v);
                stage += 2 * (last - v);
                phase ^= (stage / G::STAGES) & 1;
                stage %= G::STAGES;
            }
            v = last;
            if (load_any<G>(!ok))
                break;
            continue;
        }
        const int k = real_tile(w, v) * G::KT + base + (lane & (ROWS - 1));
        const int64_t slot = key_slot(p, w, k, key_block(p, w, k), bad);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const uint32_t full = bars + stage * 8, dst = ring + stage * G::STAGE;
            copies.before_wait(full + G::STAGES * 8, phase);
            ok = ok && bar_wait(full + G::STAGES * 8, phase, abort, p.wait_limit_ns);
            if (ok) {
                const char *src = part == 0 ? p.rot : p.copy;
                const int64_t ss = part == 0 ? p.rot_ss : p.copy_ss;
                const char *col = src + w.head * PIECES * 16 + c * 16;
#pragma unroll
                for (int i = 0; i < ROWS / PER; ++i) {
                    const int r = i * PER + sub;
                    const int64_t s = __shfl_sync(0xFFFFFFFFu, slot, r);
                    const int row = base + r;
                    copy16(dst + ((c >> 3) << 14) + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                           col + (s < 0 ? 0 : s * ss), s < 0 ? 0u : 16u);
                }
                copies.filled(full);
                next();
            }
        }
        ++v;
    }
    copies.flush();
    if (warp == 0)
        copies_land<G::STAGES>(bars, filled);
}

// Head rows in e4m3: copied as they are stored, RAW tiles ahead, then converted
// into the ring.  A thread converts the pieces that it copied itself, so a
// warp waits for nobody else's copies.  8 lanes hold the 128 bytes of a row.
template <class G>
__device__ __forceinline__ void load_heads_e4m3(const AttnParams &p, const Work &w, uint32_t ring,
                                                uint32_t bars, int warp, int lane,
                                                volatile int *abort, bool &bad)
{
    constexpr int WARPS = G::LOAD_WARPS, ROWS = G::KT / WARPS, IT = ROWS / 4;
    const int base = warp * ROWS, own = lane & (ROWS - 1);
    const int c = lane & 7, sub = lane >> 3;
    const uint32_t raw = ring + G::RAW_AT;
    const int items = 2 * (w.end - w.beg); // K, V of each tile
    auto key_at = [&](int v) { return real_tile(w, v) * G::KT + base + own; };
    auto block_at = [&](int v) { return v < w.end ? key_block(p, w, key_at(v)) : 0; };
    const char *const src[2] = {p.rot + w.head * 128 + c * 16, p.copy + w.head * 128 + c * 16};
    const float *const sc[2] = {p.rs + w.head, p.cs + w.head};
    int slot = -1; // of this lane's row in the tile last asked for
    int ask_v = w.beg, ask_stage = 0;
    int32_t blk = block_at(w.beg);
    // asks for item n (K of a tile before its V)
    auto ask = [&](int n) {
        if (n < items) {
            if (!(n & 1)) {
                slot = (int)key_slot(p, w, key_at(ask_v), blk, bad);
                blk = block_at(++ask_v);
            }
            const bool v = n & 1;
            const char *const from = v ? src[1] : src[0];
            const int64_t ss = v ? p.copy_ss : p.rot_ss;
            const uint32_t to = raw + ask_stage * G::RAW_STAGE;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int s = __shfl_sync(0xFFFFFFFFu, slot, i * 4 + sub);
                copy16(to + ((warp * IT + i) * 32 + lane) * 16, from + (s < 0 ? 0 : s * ss),
                       s < 0 ? 0u : 16u);
            }
            if (lane < ROWS)
                copy4(to + G::STAGE / 2 + (base + own) * 4,
                      (v ? sc[1] : sc[0]) + (slot < 0 ? 0 : slot * (v ? p.cs_ss : p.rs_ss)));
            if (++ask_stage == G::RAW)
                ask_stage = 0;
        }
        copy_commit();
    };
    for (int n = 0; n < G::RAW; ++n)
        ask(n);
    // a lane's two pieces of a row: the odd one first in the upper panel, so that
    // the eight lanes of a row meet eight different 16-byte columns
    const int first = c >> 2;
    const int c0 = (2 * c + first) & 7, c1 = (2 * c + 1 - first) & 7;
    int stage = 0, phase = 1, from_stage = 0;
#pragma unroll 1
    for (int n = 0; n < items; ++n) {
        copy_wait<G::RAW - 1>();
        __syncwarp(); // the scales of the warp's rows came through other lanes
        if (!bar_wait(bars + (G::STAGES + stage) * 8, phase, abort, p.wait_limit_ns))
            return;
        const uint32_t from = raw + from_stage * G::RAW_STAGE;
        const uint32_t dst = ring + stage * G::STAGE + (first << 14) + base * 128;
        constexpr int B = 4; // pieces at a time
#pragma unroll 1
        for (int i0 = 0; i0 < IT; i0 += B) {
            uint4 x[B];
            uint32_t mul[B], rare = 0;
#pragma unroll
            for (int i = 0; i < B; ++i) {
                x[i] = lds16(from + ((warp * IT + i0 + i) * 32 + lane) * 16);
                mul[i] = scale_mul(lds4(from + G::STAGE / 2 + (base + (i0 + i) * 4 + sub) * 4));
            }
#pragma unroll
            for (int i = 0; i < B; ++i)
                rare |= rare16(x[i], mul[i]);
            auto store = [&](int r, const uint4 &lo, const uint4 &hi) {
                sts16(dst + r * 128 + ((c0 ^ (r & 7)) << 4), first ? hi : lo);
                sts16(dst + r * 128 + ((c1 ^ (r & 7)) << 4), first ? lo : hi);
            };
            if (!rare) {
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    uint4 lo, hi;
                    convert16<false>(x[i], mul[i], lo, hi);
                    store((i0 + i) * 4 + sub, lo, hi);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < B; ++i) {
                    uint4 lo, hi;
                    const uint32_t at = from + ((warp * IT + i0 + i) * 32 + lane) * 16;
                    convert16<true>(
                        lds16(at),
                        scale_mul(lds4(from + G::STAGE / 2 + (base + (i0 + i) * 4 + sub) * 4)), lo,
                        hi);
                    store((i0 + i) * 4 + sub, lo, hi);
                }
            }
        }
        async_fence();
        bar_signal(bars + stage * 8);
        __syncwarp(); // every lane has read the scales before they are replaced
        ask(n + G::RAW);
        if (++from_stage == G::RAW)
            from_stage = 0;
        if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1;
        }
    }
}

// MLA rows in bf16.  In a run of whole tiles a warp for each part asks for its boxes, so
// that part 0 of the next tile, whose stage is free after the scores, does not wait for
// the others of this one, and a fourth brings this half's columns of a later tile to L2: a
// stage is free little more than a tile ahead, less than HBM takes.  Other tiles are copied row by
// row, with zeros in the place of keys that nobody sees: a warp owns 8 rows, 8 lanes
// copy 128 bytes of a row.  The warps meet after every run (see load_heads).
template <class G>
__device__ __forceinline__ void load_mla_bf16(const AttnParams &p, const Work &w, uint32_t ring,
                                              uint32_t bars, int warp, int lane,
                                              volatile int *abort, bool &bad)
{
    constexpr int AHEAD = 3;
    const int base = warp * 8, c = lane & 7, sub = lane >> 3;
    const int32_t *const table = p.block_tables + (int64_t)w.seq * p.max_blocks;
    auto whole = [&](int v) { return p.box_rows > 0 && tile_whole<G::KT>(w, real_tile(w, v)); };
    Copies copies;
    bool ok = true;
    int v = w.beg;
    while (v < w.end) {
        if (whole(v)) {
            int last = v + 1;
            while (last < w.end && whole(last))
                ++last;
            copies.flush();
            if (warp <= G::PARTS) {
                // a tile is `per` blocks, or a part of one; the last warp is AHEAD of the others
                const int per = G::KT / p.box_rows, in = p.block / p.box_rows;
                const bool before = warp == G::PARTS;
                const int skip = before ? AHEAD : 0, part = before ? G::PARTS - 1 : warp;
                const int col = part == 0 ? (1 - w.head) * 256 : w.head * 256 + (part - 1) * 128;
                const bool mine = lane < per;
                auto ask = [&](int u) {
                    const int kt = real_tile(w, u);
                    return mine && u < last ? __ldg(table + (in == 1 ? kt * per + lane : kt / in)) : 0;
                };
                int32_t blk = ask(v + skip);
                for (int u = v; ok && u < last; ++u) {
                    const int kt = real_tile(w, u + skip);
                    const bool fits = (uint32_t)blk < (uint32_t)p.num_blocks;
                    bad |= !fits;
                    const int y = fits ? (in == 1 ? 0 : (kt % in) * G::KT) + blk * p.block
                                       : (int)(p.num_blocks * p.block); // past the pool: zeros
                    blk = ask(u + 1 + skip);
                    const int ord = u - w.beg, stage = ord & 1, phase = ((ord >> 1) & 1) ^ 1;
                    const uint32_t full = bars + (part * 2 + stage) * 8;
                    ok = bar_wait(full + G::BARS / 2 * 8, phase, abort, p.wait_limit_ns);
                    if (!ok)
                        break;
                    if (before) {
                        if (mine && u + skip < last) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                prefetch_box(&p.copy_map, w.head * 256 + i * 64, y);
                            if (w.head == 0)
                                prefetch_box(&p.rot_map, 0, y);
                        }
                        continue;
                    }
                    if (lane == 0)
                        bar_signal_bulk(full, G::LOAD_WARPS * 32,
                                        part == 0 ? G::OTHER : 2 * G::PANEL);
                    if (mine) {
                        const uint32_t at = G::part(ring, part, stage) + lane * p.box_rows * 128;
                        copy_box(at, &p.copy_map, col, y, full);
                        copy_box(at + G::PANEL, &p.copy_map, col + 64, y, full);
                        if (part == 0) {
                            copy_box(at + 2 * G::PANEL, &p.copy_map, col + 128, y, full);
                            copy_box(at + 3 * G::PANEL, &p.copy_map, col + 192, y, full);
                            copy_box(at + 4 * G::PANEL, &p.rot_map, 0, y, full);
                        }
                    }
                }
            }
            v = last;
            if (load_any<G>(!ok))
                break;
            continue;
        }
        const int k = real_tile(w, v) * G::KT + base + c;
        const int64_t slot = key_slot(p, w, k, key_block(p, w, k), bad);
        const int ord = v - w.beg, stage = ord & 1, phase = ((ord >> 1) & 1) ^ 1;
#pragma unroll
        for (int part = 0; part < G::PARTS; ++part) {
            const uint32_t full = bars + (part * 2 + stage) * 8, dst = G::part(ring, part, stage);
            const int col = part == 0 ? (1 - w.head) * 512 : w.head * 512 + (part - 1) * 256;
            copies.before_wait(full + G::BARS / 2 * 8, phase);
            ok = ok && bar_wait(full + G::BARS / 2 * 8, phase, abort, p.wait_limit_ns);
            if (!ok)
                continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t s = __shfl_sync(0xFFFFFFFFu, slot, i * 4 + sub);
                const int row = base + i * 4 + sub;
                const uint32_t at = dst + row * 128 + ((c ^ (row & 7)) << 4), n = s < 0 ? 0 : 16;
                const char *src = p.copy + (s < 0 ? 0 : s * p.copy_ss) + col + c * 16;
#pragma unroll
                for (int g = 0; g < (part == 0 ? 4 : 2); ++g)
                    copy16(at + g * G::PANEL, src + g * 128, n);
                if (part == 0)
                    copy16(at + 4 * G::PANEL, p.rot + (s < 0 ? 0 : s * p.rot_ss) + c * 16, n);
            }
            copies.filled(full);
        }
        ++v;
    }
    copies.flush();
    if (warp == 0) // the last tiles of each part; after an early end some never come
        for (int part = 0; part < G::PARTS; ++part)
            copies_land<2>(bars + part * 16, v - w.beg);
}

// MLA rows with an e4m3 latent: the next tile waits in registers.
template <class G>
__device__ __forceinline__ void load_mla_e4m3(const AttnParams &p, const Work &w, uint32_t ring,
                                              uint32_t bars, int warp, int lane,
                                              volatile int *abort, bool &bad)
{
    const int base = warp * 4, c = lane & 7, sub = lane >> 3;
    uint4 lat[2][2], pe; // [part][group of 128]
    float scale[2][2];
    auto key_at = [&](int v) { return real_tile(w, v) * G::KT + base + sub; };
    auto block_at = [&](int v) { return v < w.end ? key_block(p, w, key_at(v)) : 0; };
    auto slot_at = [&](int v, int32_t blk) {
        return v < w.end ? key_slot(p, w, key_at(v), blk, bad) : (int64_t)-1;
    };
    auto fetch = [&](int part, int64_t slot) {
        const int half = part == 0 ? 1 - w.head : w.head;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const char *src = p.copy + slot * p.copy_ss + half * 256 + c * 16;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            lat[part][g] = slot < 0 ? zero : __ldg(reinterpret_cast<const uint4 *>(src + g * 128));
            scale[part][g] = slot < 0 ? 1.0f : __ldg(p.cs + slot * p.cs_ss + half * 2 + g);
        }
        if (part == 0)
            pe = slot < 0 ? zero
                          : __ldg(reinterpret_cast<const uint4 *>(p.rot + slot * p.rot_ss + c * 16));
    };
    const int first = c >> 2;
    const int c0 = (2 * c + first) & 7, c1 = (2 * c + 1 - first) & 7;
    const int64_t slot0 = slot_at(w.beg, block_at(w.beg));
    fetch(0, slot0);
    fetch(1, slot0);
    int32_t next = block_at(w.beg + 1);
    for (int v = w.beg; v < w.end; ++v) {
        const int64_t slot = slot_at(v + 1, next);
        next = block_at(v + 2);
        const int ord = v - w.beg, stage = ord & 1, phase = ((ord >> 1) & 1) ^ 1;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const uint32_t full = bars + (part * 2 + stage) * 8, dst = G::part(ring, part, stage);
            if (!bar_wait(full + G::BARS / 2 * 8, phase, abort, p.wait_limit_ns) ||
                (part == 1 && !bar_wait(full + (G::BARS / 2 + 2) * 8, phase, abort, p.wait_limit_ns)))
                return;
            const uint32_t mul[2] = {scale_mul(scale[part][0]), scale_mul(scale[part][1])};
            const uint32_t rare = rare16(lat[part][0], mul[0]) | rare16(lat[part][1], mul[1]);
            const int row = base + sub;
            const uint32_t at = dst + row * 128;
            auto store = [&](auto kind) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint4 x, y;
                    convert16<decltype(kind)::value>(lat[part][g], mul[g], x, y);
                    const uint32_t to = at + (g * 2 + first) * G::PANEL;
                    sts16(to + ((c0 ^ (row & 7)) << 4), first ? y : x);
                    sts16(to + ((c1 ^ (row & 7)) << 4), first ? x : y);
                }
                if (part == 0)
                    sts16(at + 4 * G::PANEL + ((c ^ (row & 7)) << 4), pe);
            };
            if (rare)
                store(std::true_type{});
            else
                store(std::false_type{});
            async_fence();
            bar_signal(full);
            if (part == 1) // both pairs of panels
                bar_signal(full + 16);
            fetch(part, slot);
        }
    }
}

// ---------------------------------------------------------------------------
// MMA role (one warp)
// ---------------------------------------------------------------------------

// S = Q Kᵀ of one row tile over PN panels of Q and K.
template <int N, int PANEL, int PN>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t q, uint32_t k, bool first,
                                             uint32_t lead)
{
    const uint32_t a = operand(q, 16), b = operand(k, 16);
#pragma unroll
    for (int pn = 0; pn < PN; ++pn)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma_smem<N>(d, a + pn * (16384 >> 4) + kk * 2, b + pn * (PANEL >> 4) + kk * 2,
                        !(first && pn == 0 && kk == 0), lead);
}

// O += P V: P in tensor memory, two keys to a column, each half of the keys over its
// half of S; V in panels.
template <int N, int KT>
__device__ __forceinline__ void issue_values(uint32_t d, uint32_t pt, uint32_t v, bool first,
                                             uint32_t lead)
{
    const uint32_t b = operand(v, KT * 128);
#pragma unroll
    for (int kk = 0; kk < KT / 16; ++kk)
        mma_tmem<N, 1>(d, pt + (kk < KT / 32 ? kk * 8 : KT / 2 + (kk - KT / 32) * 8),
                       b + kk * (2048 >> 4), !(first && kk == 0), lead);
}

template <class G>
__device__ __forceinline__ bool run_mma_two(const AttnParams &p, const Work &w, uint32_t tmem,
                                            uint32_t q_smem, uint32_t ring, uint32_t bars,
                                            uint32_t lead, volatile int *abort)
{
    const TileMask mask[2] = {tile_mask(p, w.n, w.len, w.row0),
                              tile_mask(p, w.n, w.len, w.row0 + kRows)};
    const uint32_t full = bars + kBarRing * 8, empty = full + G::STAGES * 8;
    bool pend[2] = {false, false}, begun[2] = {false, false};
    uint32_t pphase[2] = {0, 0};
    int stage = 0, phase = 0;         // of K of tile v
    int vstage = 0;                   // of V of the tile before
    bool v_open = false;              // V of the tile before is still held
    auto values = [&](int t) {
        if (!bar_wait(bars + (kBarP + t) * 8, pphase[t], abort, p.wait_limit_ns))
            return false;
        pphase[t] ^= 1;
        mma_fence_after();
        issue_values<128, 128>(tmem + G::O_COL(t), tmem + G::S_COL(t), ring + vstage * G::STAGE,
                               !begun[t], lead);
        begun[t] = true;
        pend[t] = false;
        return true;
    };
    for (int v = w.beg; v < w.end; ++v) {
        const int kt = real_tile(w, v);
        if (!bar_wait(full + stage * 8, phase, abort, p.wait_limit_ns))
            return false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (pend[t] && !values(t))
                return false;
            if (t == 1 && v_open)
                bar_signal_mma(empty + vstage * 8, lead);
            if (tile_active<G::KT>(mask[t], kt)) {
                issue_scores<128, 16384, 2>(tmem + G::S_COL(t), q_smem + (t << 15),
                                            ring + stage * G::STAGE, true, lead);
                bar_signal_mma(bars + (kBarS + t) * 8, lead);
                pend[t] = true;
            }
        }
        bar_signal_mma(empty + stage * 8, lead);
        if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1;
        }
        // V of this tile is the next stage; the weights come later
        vstage = stage;
        if (!bar_wait(full + stage * 8, phase, abort, p.wait_limit_ns))
            return false;
        v_open = true;
        if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1;
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
        if (pend[t] && !values(t))
            return false;
    bar_signal_mma(bars + kBarDone * 8, lead);
    return true;
}

// One row tile, two buffers of S: the scores of a tile are formed while the
// softmax of the one before runs.
template <class G>
__device__ __forceinline__ bool run_mma_one(const AttnParams &p, const Work &w, uint32_t tmem,
                                            uint32_t q_smem, uint32_t ring, uint32_t bars,
                                            uint32_t lead, volatile int *abort)
{
    const uint32_t full = bars + kBarRing * 8;
    int stage = 0, phase = 0, vstage = 0;
    for (int v = w.beg; v <= w.end; ++v) {
        const int ord = v - w.beg, i = ord & 1, turn = (ord >> 1) & 1;
        const uint32_t s_col = tmem + G::S_COL(i);
        const bool more = v < w.end;
        if (more) {
            if constexpr (G::MLA) {
                if (!bar_wait(full + i * 8, turn, abort, p.wait_limit_ns))
                    return false;
                issue_scores<64, G::PANEL, 5>(s_col, q_smem, G::part(ring, 0, i), true, lead);
                bar_signal_mma(full + (G::BARS / 2 + i) * 8, lead);
#pragma unroll
                for (int pair = 0; pair < 2; ++pair) {
                    if (!bar_wait(full + (2 + 2 * pair + i) * 8, turn, abort, p.wait_limit_ns))
                        return false;
                    const uint32_t k = operand(G::part(ring, 1 + pair, i), 16);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        mma_tmem<64, 0>(s_col, tmem + G::Q_COL + (pair * 8 + j) * 8,
                                        k + (j >> 2) * (G::PANEL >> 4) + (j & 3) * 2, 1u, lead);
                }
                bar_signal_mma(bars + (kBarS + i) * 8, lead);
            } else {
                if (!bar_wait(full + stage * 8, phase, abort, p.wait_limit_ns))
                    return false;
                issue_scores<128, 16384, 2>(s_col, q_smem, ring + stage * G::STAGE, true, lead);
                bar_signal_mma(bars + (kBarS + i) * 8, lead);
                bar_signal_mma(full + (G::STAGES + stage) * 8, lead);
                if (++stage == G::STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (ord > 0) { // weights of the tile before
            const int j = 1 - i;
            if (!bar_wait(bars + (kBarP + j) * 8, ((ord - 1) >> 1) & 1, abort, p.wait_limit_ns))
                return false;
            mma_fence_after();
            if constexpr (G::MLA) {
#pragma unroll
                for (int pair = 0; pair < 2; ++pair) {
                    issue_values<128, 64>(tmem + G::O_COL(0) + pair * 128, tmem + G::S_COL(j),
                                          G::part(ring, 1 + pair, j), ord == 1, lead);
                    bar_signal_mma(full + (G::BARS / 2 + 2 + 2 * pair + j) * 8, lead);
                }
            } else {
                issue_values<128, 128>(tmem + G::O_COL(0), tmem + G::S_COL(j),
                                       ring + vstage * G::STAGE, ord == 1, lead);
                bar_signal_mma(full + (G::STAGES + vstage) * 8, lead);
            }
            bar_signal_mma(bars + kBarO * 8, lead);
        }
        if constexpr (!G::MLA) {
            if (more) {
                vstage = stage;
                if (!bar_wait(full + stage * 8, phase, abort, p.wait_limit_ns))
                    return false;
                if (++stage == G::STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    }
    bar_signal_mma(bars + kBarDone * 8, lead);
    return true;
}

// ---------------------------------------------------------------------------
// Softmax role (a thread per row)
// ---------------------------------------------------------------------------

// The lowest n of 32 bits (none below 0, all above 31).
__device__ __forceinline__ uint32_t below(int n)
{
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

struct RowState {
    float top = -INFINITY; // maximum that the weights and O are taken against
    float sum = 0.0f;      // of this thread's half of the keys
};

// What the two threads of a row exchange.
template <class G>
struct RowPairs {
    float value[2][G::NT * kRows]; // [half][row]
};

// A vote over the two warps that share 32 rows.  Both come to every vote, also when a
// wait of one ran out: they go on or give up together.
__device__ __forceinline__ bool pair_any(int pair, bool x)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 q, %1, 0;\n"
                 "barrier.cta.red.or.pred p, %2, 64, q;\nselp.b32 %0, 1, 0, p;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)x), "r"(1 + pair)
                 : "memory");
    return r != 0;
}

// The other thread's value; the place is free again when both have read.
template <class G>
__device__ __forceinline__ float pair_swap(RowPairs<G> &pairs, int pair, int half, int row, float x)
{
    pairs.value[half][row] = x;
    bar_wait_all(1 + pair, 64);
    const float y = pairs.value[half ^ 1][row];
    bar_wait_all(1 + pair, 64);
    return y;
}

// Value `col` of key slot `s` as an fp32 if it is not finite, else 0.
template <class G>
__device__ __forceinline__ float nonfinite_value(const AttnParams &p, int64_t s, int col)
{
    const char *row = p.copy + s * p.copy_ss;
    if (G::QUANT)
        return (*reinterpret_cast<const uint8_t *>(row + col) & 0x7Fu) == 0x7Fu
                   ? __uint_as_float(0x7FC00000u)
                   : 0.0f;
    const uint32_t b = *reinterpret_cast<const uint16_t *>(row + col * 2);
    return (b & 0x7F80u) == 0x7F80u ? __uint_as_float(b << 16) : 0.0f;
}

// MLA: two of the query panels of this half into tensor memory, a row to a lane.
template <class G>
__device__ __forceinline__ void queries_to_tmem(const AttnParams &p, const Work &w, uint32_t tmem,
                                                int warp, int lane, int rows, int panel)
{
    const int r = warp * 32 + lane, row = w.row0 + r, tok = p.by_group.quotient(row);
    const bool valid = r < rows;
    const char *src =
        p.q + (valid ? (w.q0 + tok) * p.q_ts + (row - tok * p.group) * p.q_hs : 0) + w.head * 512;
    uint32_t x[64]; // both panels' loads in flight at once
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint4 y = valid ? __ldg(reinterpret_cast<const uint4 *>(src + panel * 128) + j)
                              : make_uint4(0, 0, 0, 0);
        x[4 * j] = y.x;
        x[4 * j + 1] = y.y;
        x[4 * j + 2] = y.z;
        x[4 * j + 3] = y.w;
    }
    const uint32_t at = tmem + G::Q_COL + panel * 32 + ((uint32_t)(warp * 32) << 16);
    tmem_st32(at, x);
    tmem_st32(at + 32, x + 32);
    tmem_st_wait();
}

// `warp` (0..3) owns rows 32 * warp ..., `half` says which keys of a tile are this
// thread's; `warps` of the four have rows.
template <class G>
__device__ __forceinline__ void run_softmax(const AttnParams &p, const Work &w, const TileMask &m,
                                            int t, uint32_t tmem, uint32_t ring, uint32_t bars,
                                            int warp, int half, int lane, int warps,
                                            volatile int *abort, volatile int *dirty,
                                            RowPairs<G> &pairs)
{
    constexpr int KT = G::KT, HK = KT / 2, HO = G::OC / 2; // keys, columns of O of a thread
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int pair = t * 4 + warp;
    const int r = warp * 32 + lane;
    const int row = w.row0 + t * kRows + r;
    const int tok = p.by_group.quotient(row), g = row - tok * p.group;
    const bool valid = r < m.rows;
    const int pos = w.len - w.n + tok;
    // keys this row sees: [lo, hi) and [0, sk)
    const int hi = !valid ? 0 : p.causal ? min(w.len, pos + 1) : w.len;
    const int lo = p.window ? max(0, pos - p.window + 1) : 0;
    const int sk = p.window ? min(p.sinks, hi) : 0;
    const bool one_token = G::NT == 1 && m.pos0 == m.pos1;
    const float c = p.scale * 1.4426950408889634f;
    const uint32_t o_col = tmem + G::O_COL(t) + half * HO + lanes;
    RowState st;
    int done = 0; // tiles of this row tile so far
    bool ok = true;
    for (int v = w.beg; v < w.end; ++v) {
        const int kt = real_tile(w, v);
        if (G::NT == 2 && !tile_active<KT>(m, kt))
            continue;
        const int buf = G::NT == 2 ? t : (done & 1);
        const uint32_t s_col = tmem + G::S_COL(buf) + half * HK + lanes;
        const uint32_t parity = G::NT == 2 ? (done & 1) : ((done >> 1) & 1);
        ok = ok && bar_wait(bars + (kBarS + buf) * 8, parity, abort, p.wait_limit_ns);
        mma_fence_after();
        const bool full = tile_full<KT>(p, m, kt);
        // the half row in registers: tensor memory takes some 300 clocks to answer, once
        uint32_t s[HK];
#pragma unroll
        for (int i = 0; i < HK; i += 32)
            tmem_ld32(s_col + i, s + i);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < HK; i += 32)
            tmem_pin32(s + i);
        if (!full) {
#pragma unroll
            for (int i = 0; i < HK; i += 32) { // a bit per key that is seen
                const int k0 = kt * KT + half * HK + i;
                const uint32_t see = below(hi - k0) & (~below(lo - k0) | below(sk - k0));
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    s[i + j] = (see >> j) & 1u ? s[i + j] : 0xFF800000u;
            }
        }
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}; // chains of maxima
#pragma unroll
        for (int j = 0; j < HK / 2; ++j)
            t4[j & 3] = max3(t4[j & 3], __uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
        float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        bool grew = (top - st.top) * c > kLazy; // also from -inf
        if (pair_any(pair, grew || !ok)) {
            if (pair_any(pair, !ok))
                return;
            top = fmaxf(top, pair_swap<G>(pairs, pair, half, t * kRows + r, top));
            grew = (top - st.top) * c > kLazy;
            const float f = grew ? exp2_fast((st.top - top) * c) : 1.0f;
            if (grew) {
                st.top = top;
                st.sum *= f;
            }
            if (done > 0) {
                // O of the tiles before is complete: NT = 2 issues it before these scores
                if (G::NT == 1) {
                    ok = bar_wait(bars + kBarO * 8, (done - 1) & 1, abort, p.wait_limit_ns);
                    mma_fence_after();
                }
#pragma unroll 1
                for (int i = 0; i < HO; i += 16) {
                    uint32_t o[16];
                    tmem_ld16(o_col + i, o);
                    tmem_ld_wait();
                    tmem_pin16(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st16(o_col + i, o);
                }
            }
        }
        const float off = st.top == -INFINITY ? 0.0f : -st.top * c;
        const f2 c2 = f2_of_bits(__float_as_uint(c), __float_as_uint(c));
        const f2 off2 = f2_of_bits(__float_as_uint(off), __float_as_uint(off));
        f2 sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < HK; i += 32) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const f2 x = f2_fma(f2_of_bits(s[i + 2 * j], s[i + 2 * j + 1]), c2, off2);
                float a, b;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
                a = exp2_fast(a);
                b = exp2_fast(b);
                sum2[j & 1] = f2_add(sum2[j & 1], f2_of_bits(__float_as_uint(a), __float_as_uint(b)));
                s[i / 2 + j] = pack_bf16(a, b);
            }
            tmem_st16(s_col + i / 2, s + i / 2); // over scores that have been read
        }
        float s0, s1;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(f2_add(sum2[0], sum2[1])));
        st.sum += s0 + s1;
        tmem_st_wait();
        if (!full && !one_token) {
            // A weight of 0 does not keep an infinite or NaN value out of the
            // product: take such values out of V here; rows that do see them get
            // them back at the end.
            const int ord = v - w.beg;
            uint32_t vbase;
            int pieces;
            if constexpr (G::MLA) {
                for (int part = 1; part < G::PARTS; ++part)
                    ok = ok && bar_wait(bars + (kBarRing + part * 2 + (ord & 1)) * 8,
                                        (ord >> 1) & 1, abort, p.wait_limit_ns);
                vbase = G::part(ring, 1, ord & 1);
                pieces = G::OWN / 16;
            } else {
                const int item = 2 * ord + 1, at = item % G::STAGES;
                ok = ok && bar_wait(bars + (kBarRing + at) * 8, (item / G::STAGES) & 1, abort,
                                    p.wait_limit_ns);
                vbase = ring + at * G::STAGE;
                pieces = G::STAGE / 16;
            }
            const int me = (half * warps + warp) * 32 + lane, all = warps * 64;
            uint32_t bad = 0;
            for (int i = me; i < pieces; i += all * 4) {
                uint4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = lds16(vbase + min(i + j * all, pieces - 1) * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    bad |= nonfinite2(x[j].x) | nonfinite2(x[j].y) | nonfinite2(x[j].z) |
                           nonfinite2(x[j].w);
            }
            if (bad & 0x80008000u) {
                *dirty = 1;
                __threadfence_block();
                for (int i = me; i < pieces; i += all) {
                    const uint4 x = lds16(vbase + i * 16);
                    sts16(vbase + i * 16, make_uint4(finite2(x.x), finite2(x.y), finite2(x.z),
                                                     finite2(x.w)));
                }
                async_fence();
            }
        }
        mma_fence_before();
        bar_signal(bars + (kBarP + buf) * 8);
        ++done;
    }
    // O is complete
    ok = ok && bar_wait(bars + kBarDone * 8, 0, abort, p.wait_limit_ns);
    mma_fence_after();
    if (pair_any(pair, !ok))
        return;
    const float other = pair_swap<G>(pairs, pair, half, t * kRows + r, st.sum);
    const float sum = half == 0 ? st.sum + other : other + st.sum; // the same in both
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int h = G::MLA ? g : w.head * p.group + g;
    const int64_t at = (w.q0 + tok) * p.heads + h;
    const int col0 = (G::MLA ? w.head * 256 : 0) + half * HO;
    const bool parts = w.splits > 1;
    if (valid && half == 0 && (!G::MLA || w.head == 0)) {
        const float lse = sum == 0.0f ? -INFINITY : st.top * p.scale + logf(sum);
        if (parts)
            p.part_lse[w.split * p.total_q * p.heads + at] = lse;
        else if (p.lse)
            p.lse[at] = lse;
    }
    char *out = p.out + (w.q0 + tok) * p.o_ts + h * p.o_hs + col0 * 2;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0; // a row's sectors are whole
    float *part = p.part + (w.split * p.total_q * p.heads + at) * G::DV + col0;
#pragma unroll 1
    for (int i = 0; i < HO; i += 32) {
        uint32_t o[32];
        tmem_ld32(o_col + i, o);
        tmem_ld_wait();
        tmem_pin32(o);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            o[j] = sum == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[j]) * inv);
        if (*dirty) {
            for (int v = w.beg; v < w.end; ++v) {
                const int k0 = real_tile(w, v) * KT;
                for (int k = k0; k < k0 + KT; ++k) {
                    if (!valid || !(k < hi && (k >= lo || k < sk)))
                        continue;
                    bool bad = false;
                    const int64_t s = key_slot(p, w, k, key_block(p, w, k), bad);
                    if (s < 0)
                        continue;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = __float_as_uint(
                            __uint_as_float(o[j]) +
                            nonfinite_value<G>(p, s, (G::MLA ? 0 : w.head * 128) + col0 + i + j));
                }
            }
        }
        if (!valid)
            continue;
        if (parts) {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
                st32(part + i + j, o + j);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                o[j] = pack_bf16(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
            if (wide) {
                st32(out + i * 2, o);
                st32(out + i * 2 + 32, o + 8);
            } else {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<uint4 *>(out + i * 2 + j * 4) =
                        make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------

template <class G>
__global__ void __launch_bounds__(kAttnThreads<G>, 1) attention_kernel(
    const __grid_constant__ AttnParams p)
{
    using S = Smem<G>;
    extern __shared__ unsigned char raw_smem[];
    __shared__ Work s_work;
    __shared__ uint32_t s_tmem, s_status;
    __shared__ int s_go;
    __shared__ volatile int s_abort, s_dirty;
    __shared__ RowPairs<G> s_pairs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const uint32_t q_smem = smem + S::Q, ring = smem + S::RING, bars = smem + S::BAR;

    if (warp == 0) {
        // block -> (row tile, key head or half, split); heads of one row tile and
        // its halves are neighbours, so their rows meet in L2
        const int heads = G::MLA ? 2 : p.kv_heads, x = (int)blockIdx.x;
        const int y = p.by_heads.quotient(x), tile = p.by_splits.quotient(y);
        Work w{};
        w.head = x - y * heads;
        w.split = y - tile * p.max_splits;
        int at = 0;
        bool bad = false;
        bool go = find_tile<kRows * G::NT>(p, tile, lane, w, at, bad);
        if (go) {
            w.row0 = at * kRows * G::NT;
            const int nv = key_tiles<G::KT, G::NT>(p, w);
            go = take_split(p, nv, w);
        }
        if (lane == 0) {
            s_work = w;
            s_go = go;
            s_status = bad ? kStatusOutOfRange : kStatusOk;
            s_abort = 0;
            s_dirty = 0;
            for (int i = 0; i < 2; ++i) { // the warps that have rows signal the weights
                const int rows = tile_mask(p, w.n, w.len, w.row0 + (G::NT == 2 ? i : 0) * kRows).rows;
                bar_init(bars + (kBarP + i) * 8, max(1, (rows + 31) / 32) * 64);
            }
            bar_init_fence();
        }
    } else if (warp == 1 && lane == 0) {
        bar_init(bars + kBarQ * 8, G::SOFT_WARPS * 32);
        bar_init(bars + kBarDone * 8, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(bars + (kBarS + i) * 8, 1);
            bar_init(bars + (kBarO + i) * 8, 1); // the second: drain
        }
        for (int i = 0; i < G::BARS / 2; ++i) {
            bar_init(bars + (kBarRing + i) * 8, G::LOAD_WARPS * 32);
            bar_init(bars + (kBarRing + G::BARS / 2 + i) * 8, 1);
        }
        bar_init_fence();
    } else if (warp == kMmaWarp<G>) {
        tmem_alloc(smem_u32(&s_tmem), 512);
    }
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = s_tmem;

    if (!s_go) {
        // nothing for this block
    } else if (warp < G::SOFT_WARPS) {
        if constexpr (kShares<G>)
            reg_inc<kSoftRegs>();
        const Work w = s_work;
        const int t = warp >> 3, half = (warp >> 2) & 1;
        const TileMask mask = tile_mask(p, w.n, w.len, w.row0 + t * kRows);
        const int wl = warp & 3, warps = (mask.rows + 31) / 32;
        load_queries<G>(p, w, q_smem, t, tid & 255);
        if constexpr (G::MLA)
            queries_to_tmem<G>(p, w, tmem, wl, lane, mask.rows, half * 2);
        copy_commit();
        copy_wait<0>();
        async_fence();
        mma_fence_before();
        bar_signal(bars + kBarQ * 8);
        if (wl < warps)
            run_softmax<G>(p, w, mask, t, tmem, ring, bars, wl, half, lane, warps, &s_abort,
                           &s_dirty, s_pairs);
    } else if (warp < kMmaWarp<G>) {
        if constexpr (kShares<G>)
            reg_dec<kLoadRegs>();
        const Work w = s_work;
        const int lw = warp - G::SOFT_WARPS;
        bool bad = false;
        if constexpr (G::MLA && G::QUANT)
            load_mla_e4m3<G>(p, w, ring, bars + kBarRing * 8, lw, lane, &s_abort, bad);
        else if constexpr (G::MLA)
            load_mla_bf16<G>(p, w, ring, bars + kBarRing * 8, lw, lane, &s_abort, bad);
        else if constexpr (G::QUANT)
            load_heads_e4m3<G>(p, w, ring, bars + kBarRing * 8, lw, lane, &s_abort, bad);
        else
            load_heads<G>(p, w, ring, bars + kBarRing * 8, lw, lane, &s_abort, bad);
        if (bad)
            s_status = kStatusOutOfRange;
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        if constexpr (kShares<G>)
            reg_dec<kMmaRegs>();
    }
    if (s_go && warp == kMmaWarp<G>) {
        const Work w = s_work;
        const uint32_t lead = elect_lane();
        bool ok = bar_wait(bars + kBarQ * 8, 0, &s_abort, p.wait_limit_ns);
        if (ok) {
            mma_fence_after();
            if constexpr (G::NT == 2)
                ok = run_mma_two<G>(p, w, tmem, q_smem, ring, bars, lead, &s_abort);
            else
                ok = run_mma_one<G>(p, w, tmem, q_smem, ring, bars, lead, &s_abort);
        }
        if (!ok) { // let what was issued finish before tensor memory goes
            int none = 0;
            bar_signal_mma(bars + (kBarO + 1) * 8, lead);
            bar_wait(bars + (kBarO + 1) * 8, 0, &none, 1000000000ll);
        }
    }
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    if (warp == kMmaWarp<G>)
        tmem_free(tmem, 512);
    if (tid == 0)
        write_block_status(p.header, s_abort ? kStatusTimeout : s_status, blockIdx.x, p.status_words);
}

// ---------------------------------------------------------------------------
// One new token per sequence, up to 16 query heads to a key head
// ---------------------------------------------------------------------------
//
// With so few rows the products are turned round: keys are the M of the MMA,
//     Sᵀ (128 keys x 16 rows) = K Qᵀ,   Oᵀ (128 x 16) += Vᵀ Pᵀ,
// so a thread has one key and all rows: R exponentials a tile instead of 128, and
// its key's mask is one comparison.  The rows' maxima are references that all
// threads hold; a vote finds a score that passes its reference by more than
// 2^8, and only then are the true maxima formed across the block and O rescaled.
// Sums stay per key until the end.  An MMA with N = 16 takes 40 clocks (the
// operand A is read at 128 bytes a clock), 640 a tile, where the tile's rows take
// 2700 from HBM: the kernel is bound by memory.  Two blocks share an SM, so that
// one's start and end lie under the other's loads.
//
// e4m3 rows go into 8-bit MMAs as they are stored; 1400 clocks of HBM a tile
// leave no time to widen them.  Queries and weights are split instead, x = hi +
// lo / 16 with both parts e4m3: with 4 bits each that is every bit of a bf16
// query, and a weight to 2^-8, as good as bf16 (below 2^-10 of the row's
// reference to 2^-18 of it).  The parts are rows of their own (16 for up to 8
// heads, 32 for up to 16).  A key's scale multiplies its scores, its value's scale
// 2^e its weights: they are 2^(s + e - reference), the references being those of
// s + e, and the sums take 2^-e of them.
template <bool QUANT_, int R_>
struct FewGeo {
    static constexpr bool MLA = false, QUANT = QUANT_;
    static constexpr int R = R_;                    // rows: 8 or 16
    static constexpr int N = QUANT ? 2 * R : 16;    // rows of the MMAs
    static constexpr int NT = 1, KT = 128;
    static constexpr int DV = 128;
    static constexpr int LOAD_WARPS = 4;
    static constexpr int STAGE = (QUANT ? 1 : 2) * 128 * 128, STAGES = QUANT ? 6 : 3;
    static constexpr int RING = STAGES * STAGE;
    // a key's weights: N values of 1 or 2 bytes
    static constexpr int Q_BYTES = N * (QUANT ? 128 : 256), P_BYTES = 128 * N * (QUANT ? 1 : 2);
    static constexpr int P_AT = RING, Q_AT = P_AT + 2 * P_BYTES, BAR_AT = Q_AT + Q_BYTES;
    static constexpr int BYTES = BAR_AT + (kBarRing + 2 * STAGES) * 8 + 1024;
    // tensor memory: two S, O
    static constexpr int O_COL = 2 * N, COLS = 4 * N;
};

constexpr int kFewThreads = 288; // 4 softmax warps, 4 load warps, 1 MMA warp
constexpr int kFewRows = 16;
constexpr float kLazyFew = 4.0f;   // growth of a reference: e4m3 weights start at 2^4, end at 448

// Byte of (key, first of 8 rows) of Pᵀ: core matrices of 8 keys x 8 rows (16 bytes
// a key), the second 8 rows 128 bytes on, the next 8 keys 256 bytes on.
__device__ __forceinline__ uint32_t few_weight(int key) { return (key >> 3) * 256 + (key & 7) * 16; }

// Two values to e4m3 parts x = hi + lo / 16.
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t &hi, uint32_t &lo)
{
    uint16_t h, l;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
    uint32_t w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"(h));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(l)
        : "f"((b - f.y) * 16.0f), "f"((a - f.x) * 16.0f));
    hi = h;
    lo = l;
}

// Eight values to eight bytes of each part.
__device__ __forceinline__ void split8(const float *x, uint2 &hi, uint2 &lo)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        split_e4m3(x[2 * i], x[2 * i + 1], h[i], l[i]);
    hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

// A vote over the four softmax warps.  Each of them comes to every vote, also
// when its own wait ran out: they go on or give up together.
__device__ __forceinline__ bool softmax_any(bool x)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 q, %1, 0;\n"
                 "barrier.cta.red.or.pred p, 1, 128, q;\nselp.b32 %0, 1, 0, p;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}

template <class G>
__device__ __forceinline__ bool few_softmax(const AttnParams &p, const Work &w, uint32_t tmem,
                                            uint32_t smem, uint32_t bars, int tid,
                                            volatile int *abort, float (*red)[kFewRows],
                                            const float *q_scale)
{
    constexpr int R = G::R;
    const int warp = tid >> 5, lane = tid & 31;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float c = p.scale * 1.4426950408889634f;
    float ref[R], sum[R]; // references in units of log2
#pragma unroll
    for (int r = 0; r < R; ++r) {
        ref[r] = -INFINITY;
        sum[r] = 0.0f;
    }
    // e4m3: this thread's key's scales, asked for a tile ahead
    float ks = 1.0f, vs = 1.0f;
    int32_t blk = 0;
    bool none = false;
    auto key_at = [&](int v) { return real_tile(w, v) * G::KT + tid; };
    auto ask = [&](int v, int32_t b) {
        const int64_t slot = v < w.end ? key_slot(p, w, key_at(v), b, none) : -1;
        ks = slot < 0 ? 1.0f : __ldg(p.rs + slot * p.rs_ss + w.head);
        vs = slot < 0 ? 1.0f : __ldg(p.cs + slot * p.cs_ss + w.head);
    };
    if constexpr (G::QUANT) {
        if (w.beg < w.end)
            ask(w.beg, key_block(p, w, key_at(w.beg)));
        if (w.beg + 1 < w.end)
            blk = key_block(p, w, key_at(w.beg + 1));
    }
    for (int v = w.beg; v < w.end; ++v) {
        const int ord = v - w.beg, i = ord & 1;
        const bool see = key_seen(w, key_at(v));
        const float my_ks = ks, my_vs = vs;
        if constexpr (G::QUANT) {
            ask(v + 1, blk);
            if (v + 2 < w.end)
                blk = key_block(p, w, key_at(v + 2));
        }
        bool ok = bar_wait(bars + (kBarS + i) * 8, (ord >> 1) & 1, abort, p.wait_limit_ns);
        mma_fence_after();
        uint32_t raw[G::N];
#pragma unroll
        for (int n = 0; n < G::N; n += 16)
            tmem_ld16(tmem + i * G::N + n + lanes, raw + n);
        tmem_ld_wait();
#pragma unroll
        for (int n = 0; n < G::N; n += 16)
            tmem_pin16(raw + n);
        float x[R], inv = 1.0f;
        if constexpr (G::QUANT) {
            const float e = (float)((int)(__float_as_uint(my_vs) >> 23) - 127);
            inv = __uint_as_float((254u << 23) - __float_as_uint(my_vs)); // 1 / 2^e
            const float cks = c * my_ks;
#pragma unroll
            for (int r = 0; r < R; ++r)
                x[r] = fmaf(fmaf(__uint_as_float(raw[R + r]), 0.0625f, __uint_as_float(raw[r])),
                            cks * q_scale[r], e);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
                x[r] = __uint_as_float(raw[r]) * c;
        }
        bool grew = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = see ? x[r] : -INFINITY;
            grew |= x[r] - ref[r] > kLazyFew;
        }
        if (softmax_any(grew || !ok)) {
            if (softmax_any(!ok))
                return false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float m = x[r];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
                if (lane == 0)
                    red[warp][r] = m;
            }
            bar_wait_all(1, 128);
            float f[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float m = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
                const bool up = m - ref[r] > kLazyFew;
                f[r] = up ? exp2_fast(ref[r] - m) : 1.0f;
                ref[r] = up ? m : ref[r];
                sum[r] *= f[r];
            }
            if (ord > 0) { // a lane of Oᵀ is a value column, its columns are the rows
                ok = bar_wait(bars + kBarO * 8, (ord - 1) & 1, abort, p.wait_limit_ns);
                if (softmax_any(!ok))
                    return false;
                mma_fence_after();
                uint32_t o[G::N];
#pragma unroll
                for (int n = 0; n < G::N; n += 16)
                    tmem_ld16(tmem + G::O_COL + n + lanes, o + n);
                tmem_ld_wait();
#pragma unroll
                for (int n = 0; n < G::N; n += 16)
                    tmem_pin16(o + n);
#pragma unroll
                for (int n = 0; n < G::N; ++n)
                    if (G::QUANT || n < R)
                        o[n] = __float_as_uint(__uint_as_float(o[n]) * f[n % R]);
#pragma unroll
                for (int n = 0; n < G::N; n += 16)
                    tmem_st16(tmem + G::O_COL + n + lanes, o + n);
                tmem_st_wait();
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = exp2_fast(x[r] - (ref[r] == -INFINITY ? 0.0f : ref[r]));
            sum[r] = G::QUANT ? fmaf(x[r], inv, sum[r]) : sum[r] + x[r];
        }
        const uint32_t buf = smem + G::P_AT + i * G::P_BYTES;
        if constexpr (G::QUANT) {
            // 16 bytes a key and 16 rows: the high parts, then the low ones
#pragma unroll
            for (int r = 0; r < R; ++r)
                x[r] *= 16.0f;
            uint2 hi[R / 8], lo[R / 8];
#pragma unroll
            for (int r = 0; r < R; r += 8)
                split8(x + r, hi[r / 8], lo[r / 8]);
            if constexpr (R == 8) {
                sts16(buf + tid * 16, make_uint4(hi[0].x, hi[0].y, lo[0].x, lo[0].y));
            } else {
                sts16(buf + few_weight(tid), make_uint4(hi[0].x, hi[0].y, hi[1].x, hi[1].y));
                sts16(buf + few_weight(tid) + 128, make_uint4(lo[0].x, lo[0].y, lo[1].x, lo[1].y));
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; r += 8)
                sts16(buf + few_weight(tid) + r * 16,
                      make_uint4(pack_bf16(x[r], x[r + 1]), pack_bf16(x[r + 2], x[r + 3]),
                                 pack_bf16(x[r + 4], x[r + 5]), pack_bf16(x[r + 6], x[r + 7])));
        }
        async_fence();
        mma_fence_before();
        bar_signal(bars + (kBarP + i) * 8);
    }
    if (softmax_any(!bar_wait(bars + kBarDone * 8, 0, abort, p.wait_limit_ns)))
        return false;
    mma_fence_after();
    // the sums of the block's keys
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float m = sum[r];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            m += __shfl_xor_sync(0xFFFFFFFFu, m, d);
        if (lane == 0)
            red[warp][r] = m;
    }
    bar_wait_all(1, 128);
    uint32_t o[G::N];
#pragma unroll
    for (int n = 0; n < G::N; n += 16)
        tmem_ld16(tmem + G::O_COL + n + lanes, o + n);
    tmem_ld_wait();
#pragma unroll
    for (int n = 0; n < G::N; n += 16)
        tmem_pin16(o + n);
    const bool parts = w.splits > 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r >= p.group)
            break;
        const float l = (red[0][r] + red[1][r]) + (red[2][r] + red[3][r]);
        float y = __uint_as_float(o[r]);
        if constexpr (G::QUANT)
            y = fmaf(__uint_as_float(o[R + r]), 0.0625f, y) * 0.0625f;
        y = l == 0.0f ? 0.0f : y / l;
        const int h = w.head * p.group + r;
        const int64_t at = w.q0 * p.heads + h;
        if (parts)
            p.part[(w.split * p.total_q * p.heads + at) * G::DV + tid] = y;
        else
            *reinterpret_cast<uint16_t *>(p.out + w.q0 * p.o_ts + h * p.o_hs + tid * 2) =
                (uint16_t)pack_bf16(y, y);
        if (tid == 0) {
            const float lse = l == 0.0f ? -INFINITY : ref[r] * 0.6931471805599453f + logf(l);
            if (parts)
                p.part_lse[w.split * p.total_q * p.heads + at] = lse;
            else if (p.lse)
                p.lse[at] = lse;
        }
    }
    return true;
}

template <class G>
__device__ __forceinline__ bool few_mma(const AttnParams &p, const Work &w, uint32_t tmem,
                                        uint32_t smem, uint32_t bars, uint32_t lead,
                                        volatile int *abort)
{
    const uint32_t full = bars + kBarRing * 8, empty = full + G::STAGES * 8;
    const uint32_t q = operand(smem + G::Q_AT, 16);
    // Pᵀ: no swizzle; core matrices of 8 keys x 16 bytes, 128 bytes to the rows of the
    // next 16 bytes, P_BYTES / 16 to the next 8 keys
    constexpr uint32_t kWeightHigh = (128u >> 4) | (1u << 14);
    constexpr uint32_t kKeys8 = G::P_BYTES / 16;
    int stage = 0, phase = 0, vstage = 0;
    auto next = [&] {
        if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1;
        }
    };
    for (int v = w.beg; v <= w.end; ++v) {
        const int ord = v - w.beg, i = ord & 1;
        const bool more = v < w.end;
        if (more) {
            if (!bar_wait(full + stage * 8, phase, abort, p.wait_limit_ns))
                return false;
            const uint32_t k = operand(smem + stage * G::STAGE, 16);
            if constexpr (G::QUANT) {
#pragma unroll
                for (int j = 0; j < 4; ++j) // 32 columns of 8 bits
                    mma_smem_e4m3<G::N, 0>(tmem + i * G::N, k + j * 2, q + j * 2, j > 0, lead,
                                           kOperandHigh);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mma_smem<G::N>(tmem + i * G::N, k + (j >> 2) * (16384 >> 4) + (j & 3) * 2,
                                   q + (j >> 2) * (2048 >> 4) + (j & 3) * 2, j > 0, lead);
            }
            bar_signal_mma(bars + (kBarS + i) * 8, lead);
            bar_signal_mma(empty + stage * 8, lead);
            next();
        }
        if (ord > 0) {
            const int b = 1 - i;
            if (!bar_wait(bars + (kBarP + b) * 8, ((ord - 1) >> 1) & 1, abort, p.wait_limit_ns))
                return false;
            mma_fence_after();
            const uint32_t a = operand(smem + vstage * G::STAGE, 16384);
            const uint32_t pt = operand(smem + G::P_AT + b * G::P_BYTES, kKeys8);
            if constexpr (G::QUANT) {
#pragma unroll
                for (int j = 0; j < 4; ++j) // 32 keys
                    mma_smem_e4m3<G::N, 1>(tmem + G::O_COL, a + j * (4096 >> 4),
                                           pt + j * (4 * kKeys8 >> 4), ord > 1 || j > 0, lead,
                                           kWeightHigh);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) // 16 keys
                    mma_smem<G::N, 1>(tmem + G::O_COL, a + j * (2048 >> 4),
                                      pt + j * (2 * kKeys8 >> 4), ord > 1 || j > 0, lead,
                                      kWeightHigh);
            }
            bar_signal_mma(empty + vstage * 8, lead);
            bar_signal_mma(bars + kBarO * 8, lead);
        }
        if (more) {
            vstage = stage;
            if (!bar_wait(full + stage * 8, phase, abort, p.wait_limit_ns))
                return false;
            next();
        }
    }
    bar_signal_mma(bars + kBarDone * 8, lead);
    return true;
}

// The queries of a block as e4m3 parts, a row's largest value in [128, 256) after a
// power-of-two scale; rows past the group are 0.  16 threads to a row.
template <class G>
__device__ __forceinline__ void few_queries_e4m3(const AttnParams &p, const Work &w, uint32_t q_smem,
                                                 int lt, float *q_scale)
{
    for (int r = lt >> 4; r < G::R; r += 8) {
        const int c = lt & 15;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < p.group)
            v = __ldg(reinterpret_cast<const uint4 *>(
                    p.q + w.q0 * p.q_ts + (int64_t)(w.head * p.group + r) * p.q_hs) + c);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = u[i] & 0x7FFFu, b = (u[i] >> 16) & 0x7FFFu;
            m = max(m, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        // 2^e of the row's scale: the exponent of its largest value, less 7
        const int e = min(max((int)(m >> 7) - 134, -120), 120);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16) * inv;
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u) * inv;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) // what was infinite is NaN
            x[i] = fabsf(x[i]) < 256.0f ? x[i] : __uint_as_float(0x7FC00000u);
        uint2 hi, lo;
        split8(x, hi, lo);
        const uint32_t at = q_smem + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(hi.x), "r"(hi.y) : "memory");
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + G::R * 128), "r"(lo.x), "r"(lo.y)
                     : "memory");
        if (c == 0)
            q_scale[r] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
}

template <class G>
__global__ void __launch_bounds__(kFewThreads, 2) attention_few_kernel(
    const __grid_constant__ AttnParams p)
{
    extern __shared__ unsigned char raw_smem[];
    __shared__ uint32_t s_tmem, s_status;
    __shared__ volatile int s_abort;
    __shared__ float s_red[4][kFewRows], s_qscale[kFewRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const uint32_t bars = smem + G::BAR_AT;

    const int x = (int)blockIdx.x, y = p.by_heads.quotient(x);
    Work w;
    w.seq = p.by_splits.quotient(y);
    w.head = x - y * p.kv_heads;
    w.split = y - w.seq * p.max_splits;
    w.row0 = 0;
    bool bad = !seq_queries(p, w.seq, w.q0, w.n);
    bool go = w.n > 0;
    if (go && !seq_keys(p, w.seq, w.len)) {
        bad = true;
        go = false;
    }
    if (go) {
        const int nv = key_tiles<G::KT, 1>(p, w);
        go = take_split(p, nv, w);
    }
    if (!go) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (tid == 0)
            write_block_status(p.header, bad ? kStatusOutOfRange : kStatusOk, blockIdx.x,
                               p.status_words);
        return;
    }
    if (tid == 0) {
        s_status = kStatusOk;
        s_abort = 0;
        bar_init(bars + kBarQ * 8, 128);
        bar_init(bars + kBarDone * 8, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(bars + (kBarS + i) * 8, 1);
            bar_init(bars + (kBarP + i) * 8, 128);
            bar_init(bars + (kBarO + i) * 8, 1); // the second: drain
        }
        for (int i = 0; i < G::STAGES; ++i) {
            bar_init(bars + (kBarRing + i) * 8, 128);
            bar_init(bars + (kBarRing + G::STAGES + i) * 8, 1);
        }
        bar_init_fence();
    }
    if (warp == 8)
        tmem_alloc(smem_u32(&s_tmem), G::COLS);
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = s_tmem;

    if (warp < 4) {
        if constexpr (G::QUANT) // the scales of the queries
            bar_wait_all(2, 256);
        few_softmax<G>(p, w, tmem, smem, bars, tid, &s_abort, s_red, s_qscale);
    } else if (warp < 8) {
        const int lt = tid - 128;
        if constexpr (G::QUANT) {
            few_queries_e4m3<G>(p, w, smem + G::Q_AT, lt, s_qscale);
            bar_arrive(2, 256);
            async_fence();
            bar_signal(bars + kBarQ * 8);
        } else {
            for (int i = lt; i < kFewRows * 16; i += 128) { // rows past the group are 0
                const int r = i >> 4, c = i & 15;
                const bool ok = r < p.group;
                const char *src = p.q + w.q0 * p.q_ts +
                                  (int64_t)(w.head * p.group + (ok ? r : 0)) * p.q_hs + c * 16;
                copy16(smem + G::Q_AT + (c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                       src, ok ? 16u : 0u);
            }
            bar_signal_copies(bars + kBarQ * 8);
        }
        bool out = false;
        load_heads<G>(p, w, smem, bars + kBarRing * 8, warp - 4, lane, &s_abort, out);
        if (out)
            s_status = kStatusOutOfRange;
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const uint32_t lead = elect_lane();
        bool ok = bar_wait(bars + kBarQ * 8, 0, &s_abort, p.wait_limit_ns);
        if (ok) {
            async_fence();
            ok = few_mma<G>(p, w, tmem, smem, bars, lead, &s_abort);
        }
        if (!ok) { // let what was issued finish before tensor memory goes
            int none = 0;
            bar_signal_mma(bars + (kBarO + 1) * 8, lead);
            bar_wait(bars + (kBarO + 1) * 8, 0, &none, 1000000000ll);
        }
    }
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    if (warp == 8)
        tmem_free(tmem, G::COLS);
    if (tid == 0)
        write_block_status(p.header, s_abort ? kStatusTimeout : s_status, blockIdx.x, p.status_words);
}

// Joins the parts of rows whose keys were split: a warp per (token, head).
//   lse = log Σ exp(lse_s),  out = Σ exp(lse_s - lse) out_s
template <class G>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ AttnParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t rows = p.total_q * p.heads;
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t tok = at / p.heads;
    const int h = (int)(at - tok * p.heads);
    int splits = 0;
    if (at < rows) {
        int a = 0, b = p.num_seqs; // the last sequence that starts at or before the token
        while (b - a > 1) {
            const int mid = (a + b) / 2;
            if (p.q_off[mid] <= tok)
                a = mid;
            else
                b = mid;
        }
        Work w;
        if (seq_queries(p, a, w.q0, w.n) && seq_keys(p, a, w.len) && tok >= w.q0 &&
            tok < w.q0 + w.n) {
            const int row = (int)(tok - w.q0) * p.group + h % p.group;
            w.row0 = row / (kRows * G::NT) * (kRows * G::NT);
            splits = p.by_run.quotient(key_tiles<G::KT, G::NT>(p, w) + p.split_tiles - 1);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (splits <= 1)
        return; // the row's block wrote it
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32)
        top = fmaxf(top, p.part_lse[s * rows + at]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float ref = top == -INFINITY ? 0.0f : top;
    float acc[G::DV / 32] = {}, sum = 0.0f;
    for (int s = 0; s < splits; ++s) {
        const float wgt = expf(p.part_lse[s * rows + at] - ref);
        sum += wgt;
        const float4 *o = reinterpret_cast<const float4 *>(p.part + (s * rows + at) * G::DV);
#pragma unroll
        for (int i = 0; i < G::DV / 128; ++i) {
            const float4 x = o[i * 32 + lane];
            acc[i * 4] = fmaf(wgt, x.x, acc[i * 4]);
            acc[i * 4 + 1] = fmaf(wgt, x.y, acc[i * 4 + 1]);
            acc[i * 4 + 2] = fmaf(wgt, x.z, acc[i * 4 + 2]);
            acc[i * 4 + 3] = fmaf(wgt, x.w, acc[i * 4 + 3]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    char *out = p.out + tok * p.o_ts + h * p.o_hs;
#pragma unroll
    for (int i = 0; i < G::DV / 128; ++i)
        *reinterpret_cast<uint2 *>(out + (i * 128 + lane * 4) * 2) =
            make_uint2(pack_bf16(acc[i * 4] * inv, acc[i * 4 + 1] * inv),
                       pack_bf16(acc[i * 4 + 2] * inv, acc[i * 4 + 3] * inv));
    if (lane == 0 && p.lse)
        p.lse[at] = sum == 0.0f ? -INFINITY : ref + logf(sum);
}

// Tensor map of one part of the pool's rows (`width` columns of bf16 or bytes): boxes
// of 128 bytes and p.box_rows rows, swizzled as the MMAs read them.
bool encode_map(CUtensorMap *map, const char *base, int64_t row_bytes, int64_t rows, int width,
                int box_rows, bool bytes)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    if (!encode)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {bytes ? 128u : 64u, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return encode(map,
                  bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<char *>(base), dims, strides,
                  box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows are copied as boxes where a block of the pool is a multiple of 8 rows (the
// swizzle's period) and divides a key tile, or the other way round.
template <class G>
void set_boxes(AttnParams &p)
{
    p.box_rows = 0;
    const int b = p.block;
    const int64_t rows = p.num_blocks * b;
    const int heads = p.kv_heads;
    if (b % 8 != 0 || (G::KT % b != 0 && b % G::KT != 0) || rows >= 0x7FFFFFFFll)
        return;
    const int box = std::min(b, G::KT);
    const int copy = G::MLA ? 512 : heads * 128, rot = G::MLA ? 64 : heads * 128;
    if (encode_map(&p.copy_map, p.copy, p.copy_ss, rows, copy, box, G::QUANT) &&
        encode_map(&p.rot_map, p.rot, p.rot_ss, rows, rot, box, G::QUANT))
        p.box_rows = box;
}

// Joins split rows; starts while the last blocks run and waits for them on the
// device.
template <class G>
cudaError_t launch_join(const AttnParams &p, cudaStream_t stream)
{
    if (p.max_splits == 1)
        return cudaSuccess;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.total_q * p.heads + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<G>, p);
}

// The kernel's limit of dynamic shared memory, raised once on each device.
template <auto KERNEL>
cudaError_t allow_smem(int bytes)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev) & 1u))
        return e;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        done.fetch_or(uint64_t(1) << dev);
    return e;
}

template <class G>
cudaError_t launch(AttnParams &p, int64_t blocks, cudaStream_t stream)
{
    constexpr int bytes = Smem<G>::BYTES;
    static_assert(bytes + sizeof(RowPairs<G>) + 256 <= 227 * 1024, "shared memory");
    if (!G::QUANT) // e4m3 rows are converted on their way
        set_boxes<G>(p);
    cudaError_t e = allow_smem<attention_kernel<G>>(bytes);
    if (e != cudaSuccess)
        return e;
    if (kShares<G>) { // the shares come out of what a block starts with, or it would wait
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, attention_kernel<G>)) != cudaSuccess)
            return e;
        if (G::SOFT_WARPS * kSoftRegs + G::LOAD_WARPS * kLoadRegs + 4 * kMmaRegs >
            kAttnThreads<G> / 32 * fa.numRegs)
            return cudaErrorInvalidConfiguration;
    }
    attention_kernel<G><<<(unsigned)blocks, kAttnThreads<G>, bytes, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    return launch_join<G>(p, stream);
}

template <class G>
cudaError_t launch_few(AttnParams &p, int64_t blocks, cudaStream_t stream)
{
    static_assert(G::BYTES <= 113 * 1024, "two blocks to an SM");
    set_boxes<G>(p);
    cudaError_t e = allow_smem<attention_few_kernel<G>>(G::BYTES);
    if (e != cudaSuccess)
        return e;
    attention_few_kernel<G><<<(unsigned)blocks, kFewThreads, G::BYTES, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    return launch_join<G>(p, stream);
}

} // namespace

AttnPlan plan_attention(RowKind kind, const AttnShape &a)
{
    const bool mla = kind == RowKind::Mla;
    const int64_t kt = mla ? 64 : 128;
    AttnPlan pl{};
    const bool few = !mla && a.max_q_len <= 1 && a.group <= kFewRows;
    // More than one row tile to a sequence: e4m3 rows are widened once, in a pass of
    // their own, where the workspace for that stays moderate.  8 chunks of up to 513
    // tokens x 28 heads: 265 us when every tile widened them; an MLA batch 372 us.
    const bool tiles_share = (int64_t)a.max_q_len * a.group > kRows;
    const int64_t rows_bytes = (int64_t)a.num_seqs * a.max_kv_len * (mla ? 1152 : a.kv_heads * 512);
    pl.expand = a.quant && tiles_share && rows_bytes <= kExpandBytes;
    pl.row_tiles = few ? 0 : !mla && tiles_share && (!a.quant || pl.expand) ? 2 : 1;
    const int64_t rows = kRows * std::max(1, pl.row_tiles);
    // row tiles over all sequences: at most one partly filled one each
    const int64_t tiles = few ? a.num_seqs : a.total_q * a.group / rows + a.num_seqs;
    const int64_t units = tiles * (mla ? 2 : a.kv_heads);
    // most key tiles of one row tile
    int64_t nv = (a.max_kv_len + kt - 1) / kt;
    if (a.window > 0) {
        const int64_t toks = (rows + a.group - 1) / a.group + 1;
        const int64_t w = (std::min<int64_t>(a.sinks, a.max_kv_len) + kt - 1) / kt +
                          (a.window + toks + kt - 1) / kt + 1;
        nv = std::min(nv, w);
    }
    nv = std::max<int64_t>(nv, 1);
    // pieces of the key axis: enough blocks for a few on every SM, none shorter
    // than four tiles (a block's start and end cost about as much as two)
    // (whole rows when there are units for two rounds, and their parts need no joining)
    const int64_t slots = few ? 2 * 152 : 152;
    const int64_t want = units >= 2 * slots && !few
                             ? nv
                             : std::max<int64_t>(4, (units * nv + 4 * slots - 1) / (4 * slots));
    pl.split_tiles = (int32_t)std::min(nv, want);
    pl.max_splits = (int32_t)((nv + pl.split_tiles - 1) / pl.split_tiles);
    pl.blocks = units * pl.max_splits;
    return pl;
}

cudaError_t launch_attention(AttnParams &p, RowKind kind, const AttnPlan &pl, cudaStream_t stream)
{
    const bool quant = p.cs != nullptr;
    p.by_group = Divisor((uint32_t)p.group);
    p.by_block = Divisor((uint32_t)p.block);
    p.by_heads = Divisor(kind == RowKind::Mla ? 2u : (uint32_t)p.kv_heads);
    p.by_splits = Divisor((uint32_t)p.max_splits);
    p.by_run = Divisor((uint32_t)p.split_tiles);
    if (kind == RowKind::Mla)
        return quant ? launch<MlaGeo<true>>(p, pl.blocks, stream)
                     : launch<MlaGeo<false>>(p, pl.blocks, stream);
    if (pl.row_tiles == 0 && p.group <= 8)
        return quant ? launch_few<FewGeo<true, 8>>(p, pl.blocks, stream)
                     : launch_few<FewGeo<false, 8>>(p, pl.blocks, stream);
    if (pl.row_tiles == 0)
        return quant ? launch_few<FewGeo<true, 16>>(p, pl.blocks, stream)
                     : launch_few<FewGeo<false, 16>>(p, pl.blocks, stream);
    if (pl.row_tiles == 2)
        return launch<HeadGeo<false, 2>>(p, pl.blocks, stream);
    return quant ? launch<HeadGeo<true, 1>>(p, pl.blocks, stream)
                 : launch<HeadGeo<false, 1>>(p, pl.blocks, stream);
}

} // namespace kvr
