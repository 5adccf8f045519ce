// kv_attention.cu -- attention of new tokens over the paged cache.
//
// The plainest form: a block per (query token, head), a warp per key, the
// running maximum and sum of the softmax in registers, the four warps' parts
// joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "kv_serve.h"

namespace kvr {

namespace {

constexpr int kSimpleThreads = 128;

// N values at element `at` of a row: bf16, or e4m3 times the group's scale.
template <int N>
__device__ __forceinline__ void load_row(const char *row, const float *scale, int at, float *v)
{
    if (scale) {
        const float s = scale[at / kGroup];
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(*reinterpret_cast<const uint16_t *>(row + at + i)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            v[i] = f.x * s;
            v[i + 1] = f.y * s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(row + (at + i) * 2);
            v[i] = __uint_as_float(w << 16);
            v[i + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
    }
}

template <bool MLA>
__global__ void __launch_bounds__(kSimpleThreads) attention_simple_kernel(
    const __grid_constant__ AttnParams p)
{
    constexpr int DK = MLA ? 576 : 128, DV = MLA ? 512 : 128;
    constexpr int VL = DV / 32, KL = DK / 32; // values per lane
    __shared__ float s_max[4], s_sum[4], s_acc[4][DV];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, hk = h / p.group;
    int lo = 0, hi = p.num_seqs; // the last sequence that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (p.q_off[mid] <= t ? lo : hi) = mid;
    }
    const int n = p.q_off[lo + 1] - p.q_off[lo], len = p.kv_len[lo];
    if (n < 0 || n > p.max_q_len || len < 0 || len > p.max_kv_len ||
        (int64_t)len > (int64_t)p.max_blocks * p.block || t >= p.q_off[lo + 1]) {
        if (threadIdx.x == 0)
            set_status(p.header, kStatusOutOfRange);
        return;
    }
    const int pos = len - n + (int)(t - p.q_off[lo]);
    float q[KL], acc[VL], top = -INFINITY, sum = 0.0f;
    const char *qr = p.q + t * p.q_ts + h * p.q_hs;
    load_row<VL>(qr, nullptr, lane * VL, q);
    if (MLA)
        load_row<2>(qr, nullptr, 512 + lane * 2, q + VL);
    for (int i = 0; i < VL; ++i)
        acc[i] = 0.0f;
    const int end = p.causal ? min(len, pos + 1) : len;
    const int first = p.window ? max(0, pos - p.window + 1) : 0;
    const int nsink = p.window ? max(0, min(min(p.sinks, first), end)) : 0;
    for (int j = warp; j < nsink + max(0, end - first); j += 4) {
        const int k = j < nsink ? j : first + (j - nsink);
        const int32_t blk = p.block_tables[(int64_t)lo * p.max_blocks + k / p.block];
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0)
                set_status(p.header, kStatusOutOfRange);
            continue;
        }
        const int64_t slot = (int64_t)blk * p.block + k % p.block;
        const char *cr = p.copy + slot * p.copy_ss, *rr = p.rot + slot * p.rot_ss;
        const float *cs = p.cs ? p.cs + slot * p.cs_ss : nullptr;
        const float *rs = p.rs ? p.rs + slot * p.rs_ss : nullptr;
        float key[KL], val[VL], dot = 0.0f;
        if (MLA) {
            load_row<VL>(cr, cs, lane * VL, val);
            for (int i = 0; i < VL; ++i)
                key[i] = val[i];
            load_row<2>(rr, nullptr, lane * 2, key + VL);
        } else {
            load_row<VL>(cr, cs, hk * 128 + lane * VL, val);
            load_row<KL>(rr, rs, hk * 128 + lane * KL, key);
        }
#pragma unroll
        for (int i = 0; i < KL; ++i)
            dot = fmaf(q[i], key[i], dot);
        for (int x = 16; x > 0; x >>= 1)
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, x);
        dot *= p.scale;
        const float m = fmaxf(top, dot);
        const float f = m == -INFINITY ? 1.0f : __expf(top - m);
        const float e = dot == -INFINITY ? 0.0f : __expf(dot - m);
        sum = sum * f + e;
        for (int i = 0; i < VL; ++i)
            acc[i] = acc[i] * f + e * val[i];
        top = m;
    }
    if (lane == 0) {
        s_max[warp] = top;
        s_sum[warp] = sum;
    }
    for (int i = 0; i < VL; ++i)
        s_acc[warp][lane * VL + i] = acc[i];
    __syncthreads();
    const float m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    float f[4], total = 0.0f;
    for (int w = 0; w < 4; ++w) {
        f[w] = s_max[w] == -INFINITY ? 0.0f : __expf(s_max[w] - m);
        total += f[w] * s_sum[w];
    }
    for (int d = threadIdx.x; d < DV; d += kSimpleThreads) {
        float o = 0.0f;
        for (int w = 0; w < 4; ++w)
            o += f[w] * s_acc[w][d];
        reinterpret_cast<__nv_bfloat16 *>(p.out + t * p.o_ts + h * p.o_hs)[d] =
            __float2bfloat16_rn(total == 0.0f ? 0.0f : o / total);
    }
    if (threadIdx.x == 0 && p.lse)
        p.lse[t * p.heads + h] = total == 0.0f ? -INFINITY : m + logf(total);
}

} // namespace

cudaError_t launch_attention(const AttnParams &p, RowKind kind, cudaStream_t stream)
{
    const dim3 grid((unsigned)p.total_q, (unsigned)p.heads);
    if (kind == RowKind::Mla)
        attention_simple_kernel<true><<<grid, kSimpleThreads, 0, stream>>>(p);
    else
        attention_simple_kernel<false><<<grid, kSimpleThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace kvr
