// kv_quant.cu -- rows of the paged cache in 8-bit floating point: written
// with one power-of-two scale per 128 values, and read back.
//
// A group of 128 bf16 values with largest finite magnitude a gets the scale
// 2^e, e the smallest integer with a <= 448 * 2^e, and the values x * 2^-e
// rounded to e4m3.  With a = 2^k * m, 1 <= m < 2, and 448 = 2^8 * 1.75, e is
// k - 8, plus one when m > 1.75: exponent and mantissa bits of the largest
// value decide it exactly, and multiplying by 2^-e is exact too, so the only
// rounding is the one to e4m3.
//
// Both directions are bound by HBM: a value is read once and written once
// (2 + 1 bytes, the scales 4 bytes per 128).  A warp takes a few rows of one layer
// at a time (MLA rows of 576 values two at a time: 1152 rows x 61 layers read back in
// 25 us, one by one in 29, four by four in 27): segments of whole groups, 16 lanes to a
// group, 16-byte accesses on the bf16 side and 8-byte ones on the e4m3 side; a group's
// maximum is four shuffles.  16411 GQA rows x 32 layers written in 511 us, 6.4 TB/s, 0.94
// of the copy bandwidth; 9001 MHA rows x 16 layers read back in 542 to 562 us by the card,
// 6.4 to 6.6 TB/s, 0.94 to 0.97.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "kv_serve.h"

namespace kvr {

namespace {

constexpr int kQuantThreads = 256;
constexpr int64_t kFewRows = 152 * 32; // rows that leave warps without work

// Row shapes: 16-byte bf16 pieces of the copy part (and of the rotary part, where that
// is quantised too: it is as wide); ROWS: rows of a warp's unit.
template <int COPY, int ROT, bool ROTQ_, int ROWS_>
struct QRow {
    static constexpr int CP = COPY / 8;
    static constexpr bool ROTQ = ROTQ_;
    static constexpr int ROWS = ROWS_, SEGS = ROWS * (ROTQ ? 2 : 1);
    static_assert(!ROTQ || COPY == ROT, "segments of one width");
    static_assert(ROTQ || (ROT == 64 && ROWS <= 4), "8 lanes to a k_pe row");
};

// Exponent e of a group's scale from the bits of its largest finite magnitude
// (a non-negative bf16).
__device__ __forceinline__ int scale_exp(uint32_t a)
{
    if (a == 0u)
        return 0;
    const int e = (int)(a >> 7) - 135 + ((a & 127u) > 96u ? 1 : 0);
    return e < -120 ? -120 : e;
}

__device__ __forceinline__ float exp2_int(int e) // -126 <= e <= 127
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Largest magnitudes of a 16-byte piece's even and odd values: the bits of a
// positive bf16 order like the value, those that are not finite above all others.
__device__ __forceinline__ uint32_t piece_max(uint4 v)
{
    const uint32_t m = 0x7FFF7FFFu;
    return max_u16x2(max_u16x2(v.x & m, v.y & m), max_u16x2(v.z & m, v.w & m));
}

// A piece with the values that are not finite set to 0.
__device__ __forceinline__ uint4 finite_piece(uint4 v)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] &= (w[i] & 0x7F80u) == 0x7F80u ? 0xFFFF0000u : ~0u;
        w[i] &= (w[i] & 0x7F800000u) == 0x7F800000u ? 0x0000FFFFu : ~0u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest value over the 16 lanes of a group.
__device__ __forceinline__ uint32_t group_max(uint32_t m)
{
#pragma unroll
    for (int x = 8; x > 0; x >>= 1)
        m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight values times inv to e4m3: at most 448 where they are finite.  RARE: others
// among them, which become NaN.
template <bool RARE>
__device__ __forceinline__ uint2 quant_piece(uint4 v, float inv)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = __uint_as_float(w[i] << 16) * inv, hi = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
        if (RARE) {
            const float nan = __uint_as_float(0x7FC00000u);
            lo = fabsf(lo) <= 448.0f ? lo : nan;
            hi = fabsf(hi) <= 448.0f ? hi : nan;
        }
        h[i] = e4m3x2(lo, hi);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ uint4 value_piece(uint2 v, float s)
{
    const uint32_t w[2] = {v.x, v.y};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i >> 1] >> ((i & 1) * 16))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(f.y * s), "f"(f.x * s));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// A run of values of one row: bf16 at `rows` (NULL: skipped), e4m3 at `pool` (NULL, read
// back only: zeros) with its scales.
struct Segment {
    char *rows, *pool;
    float *scale;
};

// Quantise N segments of NP 16-byte pieces (16 to a group).
template <int NP, int N>
__device__ __forceinline__ void quantise(const Segment (&seg)[N], int lane)
{
    constexpr int IT = NP / 32, B = IT * N > 8 ? 8 / N : IT;
    static_assert(NP % 32 == 0 && IT % B == 0, "whole groups");
#pragma unroll 1
    for (int b = 0; b < IT; b += B) {
        uint4 v[N][B] = {}; // a skipped segment counts as zeros
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (seg[n].rows)
                    v[n][i] = ld_stream(seg[n].rows + ((b + i) * 32 + lane) * 16);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < B; ++i) {
                uint32_t m = group_max(piece_max(v[n][i]));
                const bool rare = __any_sync(0xFFFFFFFFu, m >= 0x7F80u);
                if (rare)
                    m = group_max(piece_max(finite_piece(v[n][i])));
                const int e = scale_exp(m), at = (b + i) * 32 + lane;
                if (seg[n].rows) {
                    *reinterpret_cast<uint2 *>(seg[n].pool + at * 8) =
                        rare ? quant_piece<true>(v[n][i], exp2_int(-e))
                             : quant_piece<false>(v[n][i], exp2_int(-e));
                    if ((lane & 15) == 0)
                        seg[n].scale[at >> 4] = exp2_int(e);
                }
            }
    }
}

// Read N segments back; KEEP: into rows that are read again soon.
template <int NP, int N, bool KEEP>
__device__ __forceinline__ void dequantise(const Segment (&seg)[N], int lane)
{
    constexpr int IT = NP / 32, B = IT * N > 8 ? 8 / N : IT;
#pragma unroll 1
    for (int b = 0; b < IT; b += B) {
        uint2 v[N][B] = {};
        float s[N][B] = {};
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int at = (b + i) * 32 + lane;
                if (seg[n].rows && seg[n].pool) {
                    v[n][i] = __ldcs(reinterpret_cast<const uint2 *>(seg[n].pool + at * 8));
                    s[n][i] = __ldg(seg[n].scale + (at >> 4));
                }
            }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (seg[n].rows) {
                    char *const to = seg[n].rows + ((b + i) * 32 + lane) * 16;
                    if (KEEP)
                        *reinterpret_cast<uint4 *>(to) = value_piece(v[n][i], s[n][i]);
                    else
                        st_stream(to, value_piece(v[n][i], s[n][i]));
                }
    }
}

// What to do with a unit of rows: write them into the pool, read them back, or read
// them back for kernels that follow.
enum class Move { Write, Read, Keep };

// One unit of R::ROWS rows of layer l: row lane % ROWS has slot rs of `rows` (-1:
// skipped) and ps of `pool` (-1, reading: zeros).
template <class R, Move M>
__device__ __forceinline__ void move_unit(const PoolView &rows, const QuantView &pool, int64_t l,
                                          int64_t rs, int64_t ps, int lane)
{
    constexpr int ROWS = R::ROWS;
    char *const rc = rows.copy + l * rows.copy_ls, *const rr = rows.rot + l * rows.rot_ls;
    char *const pc = pool.copy + l * pool.copy_ls, *const pr = pool.rot + l * pool.rot_ls;
    Segment seg[R::SEGS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t a = __shfl_sync(0xFFFFFFFFu, rs, r), b = __shfl_sync(0xFFFFFFFFu, ps, r);
        const bool row = a >= 0, old = b >= 0;
        seg[r] = {row ? rc + a * rows.copy_ss : nullptr, old ? pc + b * pool.copy_ss : nullptr,
                  pool.cs + l * pool.cs_ls + b * pool.cs_ss};
        if constexpr (R::ROTQ)
            seg[ROWS + r] = {row ? rr + a * rows.rot_ss : nullptr,
                             old ? pr + b * pool.rot_ss : nullptr,
                             pool.rs + l * pool.rs_ls + b * pool.rs_ss};
    }
    // MLA: 8 lanes to the k_pe of a row
    const int64_t ka = __shfl_sync(0xFFFFFFFFu, rs, lane >> 3);
    const int64_t kb = __shfl_sync(0xFFFFFFFFu, ps, lane >> 3);
    const bool has_pe = !R::ROTQ && lane < ROWS * 8 && ka >= 0;
    char *const kr = rr + ka * rows.rot_ss + (lane & 7) * 16;
    char *const kp = pr + kb * pool.rot_ss + (lane & 7) * 16;
    uint4 pe = make_uint4(0, 0, 0, 0);
    if (has_pe && (M == Move::Write || kb >= 0))
        pe = ld_stream(M == Move::Write ? kr : kp);
    if constexpr (M == Move::Write)
        quantise<R::CP>(seg, lane);
    else
        dequantise<R::CP, R::SEGS, M == Move::Keep>(seg, lane);
    if (has_pe) {
        if (M == Move::Read)
            st_stream(kr, pe);
        else
            *reinterpret_cast<uint4 *>(M == Move::Write ? kp : kr) = pe;
    }
}

// A warp takes units of R::ROWS rows of a layer; READ: pool -> rows, else rows ->
// pool.
template <class R, bool READ>
__global__ void __launch_bounds__(kQuantThreads) quant_kernel(const __grid_constant__ QuantParams p)
{
    constexpr int ROWS = R::ROWS;
    const int lane = threadIdx.x & 31;
    const int64_t per_layer = (p.num_rows + ROWS - 1) / ROWS, total = per_layer * p.layers;
    const int64_t step = (int64_t)gridDim.x * (kQuantThreads / 32);
    int bad = 0;
    for (int64_t u = (int64_t)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5); u < total;
         u += step) {
        const int64_t l = u / per_layer, i = (u - l * per_layer) * ROWS + (lane & (ROWS - 1));
        int64_t rs = -1, ps = -1; // slots of row lane % ROWS of the unit
        if (i < p.num_rows) {
            rs = p.row_slot ? p.row_slot[i] : i;
            ps = p.pool_slot[i];
            if (rs < 0 || rs >= p.rows.num_slots || ps < 0 || ps >= p.pool.num_slots) {
                bad = 1;
                rs = -1;
            }
        }
        move_unit<R, READ ? Move::Read : Move::Write>(p.rows, p.pool, l, rs, ps, lane);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
        write_block_status(p.header, bad ? kStatusOutOfRange : kStatusOk, blockIdx.x, gridDim.x);
}

// The cached rows of a batch that its queries see, as bf16 rows: key k of sequence s
// goes to row s * p.pad + k.  Rows of a bad block become zeros, and so do the others of a
// block of kExpandBlock rows with some that are seen.  Also writes the block table of those
// rows.
template <class R>
__global__ void __launch_bounds__(kQuantThreads) expand_kernel(const __grid_constant__ ExpandParams p)
{
    constexpr int ROWS = R::ROWS;
    const int lane = threadIdx.x & 31;
    const int64_t total = (int64_t)p.num_seqs * p.pad / ROWS;
    const int64_t step = (int64_t)gridDim.x * (kQuantThreads / 32);
    int bad = 0;
    for (int64_t i = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x;
         i < (int64_t)p.num_seqs * (p.pad / kExpandBlock); i += (int64_t)gridDim.x * kQuantThreads)
        p.table[i] = (int32_t)i;
    for (int64_t u = (int64_t)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5); u < total;
         u += step) {
        const int64_t row = u * ROWS + (lane & (ROWS - 1));
        const int s = (int)(u * ROWS / p.pad), k = (int)(row - (int64_t)s * p.pad);
        const int n = p.q_off[s + 1] - p.q_off[s], len = p.kv_len[s];
        // sequences whose lengths do not fit are left to the attention kernel
        const bool fits = n > 0 && len >= 0 && len <= p.max_kv_len &&
                          (int64_t)len <= (int64_t)p.max_blocks * p.block;
        const int lo = p.window ? len - n - p.window + 1 : 0;
        const bool seen = fits && k < len && (k >= lo || k < p.sinks);
        const int k0 = k / kExpandBlock * kExpandBlock;
        const bool block_seen = fits && k0 < len && (k0 + kExpandBlock > lo || k0 < p.sinks);
        if (!__any_sync(0xFFFFFFFFu, block_seen))
            continue;
        int64_t ps = -1;
        if (seen) {
            const int b = (int)((uint32_t)k / (uint32_t)p.block);
            const int32_t blk = p.block_tables[(int64_t)s * p.max_blocks + b];
            if (blk < 0 || blk >= p.num_blocks)
                bad = 1;
            else
                ps = (int64_t)blk * p.block + (k - b * p.block);
        }
        move_unit<R, Move::Keep>(p.rows, p.pool, 0, block_seen ? row : -1, ps, lane);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
        p.status[blockIdx.x] = bad ? kStatusOutOfRange : kStatusOk;
}

template <class R>
cudaError_t launch_expand_row(const ExpandParams &p, cudaStream_t stream)
{
    expand_kernel<R><<<p.blocks, kQuantThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <class R, bool READ>
cudaError_t launch_row(const QuantParams &p, cudaStream_t stream)
{
    constexpr int WARPS = kQuantThreads / 32;
    const int64_t units = (p.num_rows + R::ROWS - 1) / R::ROWS * p.layers;
    const int64_t want = (units + WARPS - 1) / WARPS;
    const int blocks = (int)(want < kQuantMaxBlocks ? want : kQuantMaxBlocks);
    quant_kernel<R, READ><<<blocks, kQuantThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <bool READ>
cudaError_t launch(const QuantParams &p, RowKind kind, cudaStream_t stream)
{
    // few rows (a decode step): one to a warp, more of them at work at once
    const bool few = p.num_rows * p.layers <= kFewRows;
    switch (kind) {
    case RowKind::Mla:
        return few ? launch_row<QRow<512, 64, false, 1>, READ>(p, stream)
                   : launch_row<QRow<512, 64, false, 2>, READ>(p, stream);
    case RowKind::Gqa:
        return launch_row<QRow<1024, 1024, true, 1>, READ>(p, stream);
    case RowKind::Gqa4:
        if (few)
            return launch_row<QRow<512, 512, true, 1>, READ>(p, stream);
        return launch_row<QRow<512, 512, true, 2>, READ>(p, stream);
    case RowKind::Mha:
        return launch_row<QRow<4096, 4096, true, 1>, READ>(p, stream);
    }
    return cudaErrorInvalidValue;
}

} // namespace

cudaError_t launch_quantize(const QuantParams &p, RowKind kind, cudaStream_t stream)
{
    return launch<false>(p, kind, stream);
}

cudaError_t launch_dequantize(const QuantParams &p, RowKind kind, cudaStream_t stream)
{
    return launch<true>(p, kind, stream);
}

int expand_blocks(int64_t rows)
{
    const int64_t want = (rows + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    return (int)(want < kQuantMaxBlocks ? want : kQuantMaxBlocks);
}

cudaError_t launch_expand(const ExpandParams &p, RowKind kind, cudaStream_t stream)
{
    switch (kind) {
    case RowKind::Mla:
        return launch_expand_row<QRow<512, 64, false, 2>>(p, stream);
    case RowKind::Gqa:
        return launch_expand_row<QRow<1024, 1024, true, 1>>(p, stream);
    case RowKind::Gqa4:
        return launch_expand_row<QRow<512, 512, true, 2>>(p, stream);
    case RowKind::Mha:
        return launch_expand_row<QRow<4096, 4096, true, 1>>(p, stream);
    }
    return cudaErrorInvalidValue;
}

} // namespace kvr
