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
// (2 + 1 bytes, the scales 4 bytes per 128).  A warp takes one row of one
// layer at a time, 16 lanes to a group: 16-byte accesses on the bf16 side,
// 8-byte ones on the e4m3 side, up to eight in flight per lane; the group's
// maximum is four shuffles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "kv_serve.h"

namespace kvr {

namespace {

constexpr int kQuantThreads = 256;

// Row shapes: 16-byte bf16 pieces of the copy and rotary part; ROTQ: the
// rotary part is quantised too.
template <int COPY, int ROT, bool ROTQ_>
struct QRow {
    static constexpr int CP = COPY / 8, RP = ROT / 8;
    static constexpr bool ROTQ = ROTQ_;
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

// Largest finite magnitude of a 16-byte piece, as bf16 bits.
__device__ __forceinline__ uint32_t piece_max(uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i] & 0x7FFFu, b = (w[i] >> 16) & 0x7FFFu;
        m = max(m, a < 0x7F80u ? a : 0u);
        m = max(m, b < 0x7F80u ? b : 0u);
    }
    return m;
}

// Two values to e4m3; finite values are at most 448 here, so anything above
// was infinite and becomes NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    const float nan = __uint_as_float(0x7FC00000u);
    lo = fabsf(lo) <= 448.0f ? lo : nan;
    hi = fabsf(hi) <= 448.0f ? hi : nan;
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint2 quant_piece(uint4 v, float inv)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = e4m3x2(__uint_as_float(w[i] << 16) * inv,
                      __uint_as_float(w[i] & 0xFFFF0000u) * inv);
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

// Quantise NP 16-byte pieces (16 to a group) of one row.
template <int NP>
__device__ __forceinline__ void quant_part(const char *src, char *dst, float *scale, int lane)
{
    constexpr int IT = NP / 32, B = IT < 8 ? IT : 8;
    static_assert(NP % 32 == 0 && IT % B == 0, "whole groups");
#pragma unroll 1
    for (int b = 0; b < IT; b += B) {
        uint4 v[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
            v[i] = ld_stream(src + ((b + i) * 32 + lane) * 16);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            uint32_t m = piece_max(v[i]);
#pragma unroll
            for (int x = 8; x > 0; x >>= 1)
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
            const int e = scale_exp(m), at = (b + i) * 32 + lane;
            *reinterpret_cast<uint2 *>(dst + at * 8) = quant_piece(v[i], exp2_int(-e));
            if ((lane & 15) == 0)
                scale[at >> 4] = exp2_int(e);
        }
    }
}

template <int NP>
__device__ __forceinline__ void value_part(const char *src, char *dst, const float *scale, int lane)
{
    constexpr int IT = NP / 32, B = IT < 8 ? IT : 8;
#pragma unroll 1
    for (int b = 0; b < IT; b += B) {
        uint2 v[B];
        float s[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int at = (b + i) * 32 + lane;
            v[i] = __ldcs(reinterpret_cast<const uint2 *>(src + at * 8));
            s[i] = __ldg(scale + (at >> 4));
        }
#pragma unroll
        for (int i = 0; i < B; ++i)
            st_stream(dst + ((b + i) * 32 + lane) * 16, value_piece(v[i], s[i]));
    }
}

// One warp per (layer, row); READ: pool -> rows, else rows -> pool.
template <class R, bool READ>
__global__ void __launch_bounds__(kQuantThreads) quant_kernel(const __grid_constant__ QuantParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t total = p.num_rows * p.layers;
    const int64_t step = (int64_t)gridDim.x * (kQuantThreads / 32);
    int bad = 0;
    for (int64_t w = (int64_t)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5); w < total;
         w += step) {
        const int64_t l = w / p.num_rows, i = w - l * p.num_rows;
        const int64_t rs = p.row_slot ? p.row_slot[i] : i, ps = p.pool_slot[i];
        if (rs < 0 || rs >= p.rows.num_slots || ps < 0 || ps >= p.pool.num_slots) {
            bad = 1;
            continue;
        }
        char *rc = p.rows.copy + l * p.rows.copy_ls + rs * p.rows.copy_ss;
        char *rr = p.rows.rot + l * p.rows.rot_ls + rs * p.rows.rot_ss;
        char *pc = p.pool.copy + l * p.pool.copy_ls + ps * p.pool.copy_ss;
        char *pr = p.pool.rot + l * p.pool.rot_ls + ps * p.pool.rot_ss;
        float *cs = p.pool.cs + l * p.pool.cs_ls + ps * p.pool.cs_ss;
        float *xs = R::ROTQ ? p.pool.rs + l * p.pool.rs_ls + ps * p.pool.rs_ss : nullptr;
        if constexpr (READ) {
            value_part<R::CP>(pc, rc, cs, lane);
            if constexpr (R::ROTQ)
                value_part<R::RP>(pr, rr, xs, lane);
            else if (lane < R::RP)
                st_stream(rr + lane * 16, ld_stream(pr + lane * 16));
        } else {
            quant_part<R::CP>(rc, pc, cs, lane);
            if constexpr (R::ROTQ)
                quant_part<R::RP>(rr, pr, xs, lane);
            else if (lane < R::RP)
                *reinterpret_cast<uint4 *>(pr + lane * 16) = ld_stream(rr + lane * 16);
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
        write_block_status(p.header, bad ? kStatusOutOfRange : kStatusOk, blockIdx.x, gridDim.x);
}

template <bool READ>
cudaError_t launch(const QuantParams &p, RowKind kind, cudaStream_t stream)
{
    const int64_t warps = p.num_rows * p.layers;
    const int64_t want = (warps + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    const int blocks = (int)(want < kQuantMaxBlocks ? want : kQuantMaxBlocks);
    switch (kind) {
    case RowKind::Mla:
        quant_kernel<QRow<512, 64, false>, READ><<<blocks, kQuantThreads, 0, stream>>>(p);
        break;
    case RowKind::Gqa:
        quant_kernel<QRow<1024, 1024, true>, READ><<<blocks, kQuantThreads, 0, stream>>>(p);
        break;
    case RowKind::Gqa4:
        quant_kernel<QRow<512, 512, true>, READ><<<blocks, kQuantThreads, 0, stream>>>(p);
        break;
    case RowKind::Mha:
        quant_kernel<QRow<4096, 4096, true>, READ><<<blocks, kQuantThreads, 0, stream>>>(p);
        break;
    }
    return cudaGetLastError();
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

} // namespace kvr
