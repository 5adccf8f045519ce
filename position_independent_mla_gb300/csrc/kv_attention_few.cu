// kv_attention_few.cu -- attention of one new token per sequence with up to 16 query
// heads to a key head, the usual decode step.
//
// With so few rows the products are turned round: keys are the M of the MMA,
//     Sᵀ (128 keys x 16 rows) = K Qᵀ,   Oᵀ (128 x 16) += Vᵀ Pᵀ,
// so a thread has one key and all rows: R exponentials a tile instead of 128, and
// its key's mask is one comparison.  The rows' maxima are references that all
// threads hold; a vote finds a score that passes its reference by more than
// 2^4, and only then are the true maxima formed across the block and O rescaled.
// Sums stay per key until the end.  An MMA with N = 16 takes 40 clocks (the
// operand A is read at 128 bytes a clock), 640 a tile, where the tile's rows take
// 2700 from HBM: the kernel is bound by memory.  Two blocks share an SM, so that
// one's start and end lie under the other's loads.
//
// e4m3 rows go into 8-bit MMAs as they are stored; 1400 clocks of HBM a tile
// leave no time to widen them.  Queries and weights are split instead into three e5m2
// parts of 3 bits each, x = a + b / 8 + c / 64: every bit of a bf16 query down to 2^-29 of
// its head's largest value (to 2^-37 of it below), and a weight to 2^-9, better than bf16, down
// to 2^-25 of the row's reference (to 2^-34 of it below).  The exponents' range is what
// counts: two e4m3 parts have the bits too, but end at 2^-18 of a reference, and the sum
// of ten thousand weights that small may be a few per cent of the result (64 ragged
// sequences 187 us with those, 190 to 193 with three).  The parts are rows of their own
// (24 of 32 for up to 8 heads, 48 for up to 16).  Weights over bf16 rows are rounded to
// bf16, the type of the rows that they are multiplied with: 2^-8 of each, as out itself.
//
// A key's scale multiplies its scores, its value's scale 2^e its weights: they are
// 2^(s + e - reference), the references being those of s + e.  The sums are of
// 2^(s - reference) with references of the scores alone, so that they (and lse) do not
// depend on the values: 2^(s + e) of keys whose scales lie 2^120 apart has no place in
// one fp32 sum.  A value row without values other than 0 (and NaN) has the scale 1, which
// says nothing of its size: it raises no reference of the weights.  Rows at that scale are
// looked at for it, in the shared memory that the MMA reads them from, only when a
// reference is about to grow.
//
// Short contexts of few sequences leave most of the SMs idle and are a matter of
// latency: their runs of keys become the blocks of a cluster, which join their parts
// through shared memory instead of a second kernel (one token over 577 keys, 32
// heads over 8: 10.2 us a call, 11.4 with the second kernel).
//
// 64 ragged sequences over e4m3 rows: 190 us, 6.0 TB/s, 0.89 of the copy bandwidth; 8
// sequences under a window of 4096, 32 heads of their own, bf16: 98 us, 5.5 TB/s, 0.81.
// With 16 heads to a key head instead of 4: 336 us over bf16 rows, 0.94; 334 over e4m3
// rows, 0.51, where two blocks' softmax warps split twice 16 weights a key and are the bound.
#include "kv_attn_tile.cuh"

namespace kvr {

namespace {

template <bool QUANT_, int R_>
struct FewGeo {
    static constexpr bool MLA = false, QUANT = QUANT_;
    static constexpr int R = R_;                    // rows: 8 or 16
    // rows of the MMAs; e4m3: R for each of three parts, to whole 16 (others: 16)
    static constexpr int N = QUANT ? (3 * R + 15) / 16 * 16 : 16;
    static constexpr int KT = 128;
    static constexpr int DV = 128;
    static constexpr int LOAD_WARPS = 4;
    static constexpr int STAGE = (QUANT ? 1 : 2) * 128 * 128;
    static constexpr int STAGES = !QUANT ? 3 : R == 8 ? 6 : 5;
    static constexpr int RING = STAGES * STAGE;
    // a key's weights: N values of 1 or 2 bytes
    static constexpr int Q_BYTES = N * (QUANT ? 128 : 256), P_BYTES = 128 * N * (QUANT ? 1 : 2);
    static constexpr int P_AT = RING, Q_AT = P_AT + 2 * P_BYTES, BAR_AT = Q_AT + Q_BYTES;
    static constexpr int BYTES = BAR_AT + (kBarRing + 2 * STAGES) * 8 + 1024;
    // tensor memory: two S, O
    static constexpr int O_COL = 2 * N, COLS = N == 48 ? 256 : 4 * N;
};

constexpr int kFewThreads = 288; // 4 softmax warps, 4 load warps, 1 MMA warp
constexpr float kLazyFew = 4.0f;   // growth of a reference
constexpr float kWeightUnit = 2048.0f; // of e5m2 weights, which grow to 2^15 then; e5m2 ends at 57344

// Byte of a key's first 16 bytes of Pᵀ: core matrices of 8 keys x 16 bytes, the next 16 bytes
// of a key 128 on, the next 8 keys behind all rows of these.
template <class G>
__device__ __forceinline__ uint32_t few_weight(int key)
{
    return (key >> 3) * (G::P_BYTES / 16) + (key & 7) * 16;
}

// What the softmax warps share: maxima of a tile, and the references (in units of log2) with
// the factors of their last growth; of the scores, and (e4m3) of the weights.
struct FewRefs {
    float top[2][4][kFewRows], ref[2][kFewRows], grow[2][kFewRows];
};

// This thread's values of the R rows in tensor memory.  16 rows in three parts come in two
// steps, half of the registers at a time.
template <class G>
__device__ __forceinline__ void few_rows(uint32_t at, float (&x)[G::R])
{
    constexpr int R = G::R, FIRST = G::N == 48 ? 16 : 0;
    uint32_t raw[G::N];
#pragma unroll
    for (int n = FIRST; n < G::N; n += 16)
        tmem_ld16(at + n, raw + n);
    tmem_ld_wait();
#pragma unroll
    for (int n = FIRST; n < G::N; n += 16)
        tmem_pin16(raw + n);
    if constexpr (!G::QUANT) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            x[r] = __uint_as_float(raw[r]);
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
            x[r] = fmaf(__uint_as_float(raw[2 * R + r]), 0.125f, __uint_as_float(raw[R + r]));
        if (FIRST) {
            tmem_ld16(at, raw);
            tmem_ld_wait();
            tmem_pin16(raw);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
            x[r] = fmaf(x[r], 0.125f, __uint_as_float(raw[r]));
    }
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

// An e4m3 row of 128 bytes, swizzled, holds a value that is neither 0 nor NaN.
__device__ __forceinline__ bool few_has_values(uint32_t row, int key)
{
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 v = lds16(row + ((j ^ (key & 7)) << 4));
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) // 0x7F in the bytes that are NaN
            any |= x[i] & 0x7F7F7F7Fu & ~((e4m3_nan(x[i]) >> 7) * 0x7Fu);
    }
    return any != 0;
}

template <class G>
__device__ __forceinline__ bool few_softmax(const AttnParams &p, const Work &w, uint32_t tmem,
                                            uint32_t smem, uint32_t bars, int tid,
                                            volatile int *abort, FewRefs &refs,
                                            const float *q_scale)
{
    constexpr int R = G::R;
    constexpr int KINDS = G::QUANT ? 2 : 1, WEIGHTS = KINDS - 1; // of references; the weights'
    const int warp = tid >> 5, lane = tid & 31;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float c = p.scale * 1.4426950408889634f;
    float sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        sum[r] = 0.0f;
    if (tid < 2 * kFewRows)
        refs.ref[tid / kFewRows][tid % kFewRows] = -INFINITY;
    bar_wait_all(1, 128);
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
        float x[R], e = 0.0f; // scores; exponent of the value's scale
        few_rows<G>(tmem + i * G::N + lanes, x);
        if constexpr (G::QUANT)
            e = (float)((int)(__float_as_uint(my_vs) >> 23) - 127);
        const float cks = G::QUANT ? c * my_ks : c;
#pragma unroll
        for (int r = 0; r < R; ++r)
            x[r] *= G::QUANT ? cks * q_scale[r] : cks;
        bool grew = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = see ? x[r] : -INFINITY;
            grew |= x[r] - refs.ref[0][r] > kLazyFew;
            if (G::QUANT)
                grew |= x[r] + e - refs.ref[WEIGHTS][r] > kLazyFew;
        }
        if (softmax_any(grew || !ok)) {
            bool sized = see; // the value's scale tells its size
            if constexpr (G::QUANT) {
                const bool look = see && my_vs == 1.0f;
                if (ok && __any_sync(0xFFFFFFFFu, look)) { // V of this tile stays until its weights
                    const int item = 2 * ord + 1, at = item % G::STAGES;
                    ok = bar_wait(bars + (kBarRing + at) * 8, (item / G::STAGES) & 1, abort,
                                  p.wait_limit_ns);
                    if (ok && look)
                        sized = few_has_values(smem + at * G::STAGE + tid * 128, tid);
                }
            }
            if (softmax_any(!ok))
                return false;
#pragma unroll
            for (int k = 0; k < KINDS; ++k)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float m = k == 0 ? x[r] : sized ? x[r] + e : -INFINITY;
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1)
                        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
                    if (lane == 0)
                        refs.top[k][warp][r] = m;
                }
            bar_wait_all(1, 128);
            if (tid < KINDS * R) {
                const int k = tid / R, r = tid % R;
                const float(&top)[4][kFewRows] = refs.top[k];
                const float m = fmaxf(fmaxf(top[0][r], top[1][r]), fmaxf(top[2][r], top[3][r]));
                const float ref = refs.ref[k][r];
                const bool up = m - ref > kLazyFew;
                refs.grow[k][r] = up ? exp2_fast(ref - m) : 1.0f;
                refs.ref[k][r] = up ? m : ref;
            }
            bar_wait_all(1, 128);
#pragma unroll
            for (int r = 0; r < R; ++r)
                sum[r] *= refs.grow[0][r];
            if (ord > 0) { // a lane of Oᵀ is a value column, its columns are the rows
                ok = bar_wait(bars + kBarO * 8, (ord - 1) & 1, abort, p.wait_limit_ns);
                if (softmax_any(!ok))
                    return false;
                mma_fence_after();
#pragma unroll
                for (int n = 0; n < G::N; n += 16) {
                    uint32_t o[16];
                    tmem_ld16(tmem + G::O_COL + n + lanes, o);
                    tmem_ld_wait();
                    tmem_pin16(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) *
                                               refs.grow[WEIGHTS][(n + j) % R]);
                    tmem_st16(tmem + G::O_COL + n + lanes, o);
                }
                tmem_st_wait();
            }
        }
        auto against = [&](int k, int r) {
            const float ref = refs.ref[k][r];
            return ref == -INFINITY ? 0.0f : ref;
        };
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float s = x[r];
            x[r] = exp2_fast(s - against(0, r));
            sum[r] += x[r];
            if (G::QUANT)
                x[r] = exp2_fast(s + e - against(WEIGHTS, r));
        }
        const uint32_t buf = smem + G::P_AT + i * G::P_BYTES;
        if constexpr (G::QUANT) {
            // 16 bytes a key and 16 rows of the MMA
#pragma unroll
            for (int r = 0; r < R; ++r)
                x[r] *= kWeightUnit;
            uint2 y[G::N / 8] = {}; // rows past the parts are 0
#pragma unroll
            for (int r = 0; r < R; r += 8) {
                uint2 part[3];
                split8(x + r, part);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    y[(k * R + r) / 8] = part[k];
            }
#pragma unroll
            for (int n = 0; n < G::N / 16; ++n)
                sts16(buf + few_weight<G>(tid) + n * 128,
                      make_uint4(y[2 * n].x, y[2 * n].y, y[2 * n + 1].x, y[2 * n + 1].y));
        } else {
#pragma unroll
            for (int r = 0; r < R; r += 8)
                sts16(buf + few_weight<G>(tid) + r * 16,
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
            refs.top[0][warp][r] = m;
    }
    bar_wait_all(1, 128);
    float o[R];
    few_rows<G>(tmem + G::O_COL + lanes, o);
    const bool parts = w.splits > 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r >= p.group)
            break;
        const float(&part)[4][kFewRows] = refs.top[0];
        const float l = (part[0][r] + part[1][r]) + (part[2][r] + part[3][r]);
        float y = o[r];
        if constexpr (G::QUANT) // from the references of the weights to those of the scores
            y *= (1.0f / kWeightUnit) * exp2f(refs.ref[WEIGHTS][r] - refs.ref[0][r]);
        y = l == 0.0f ? 0.0f : y / l;
        const int h = w.head * p.group + r;
        const int64_t at = w.q0 * p.heads + h;
        if (p.cluster) // the ring is free now
            sts4(smem + r * 512 + tid * 4, y);
        else if (parts)
            p.part[(w.split * p.total_q * p.heads + at) * G::DV + tid] = y;
        else
            *reinterpret_cast<uint16_t *>(p.out + w.q0 * p.o_ts + h * p.o_hs + tid * 2) =
                (uint16_t)pack_bf16(y, y);
        if (tid == 0) {
            const float lse = l == 0.0f ? -INFINITY : refs.ref[0][r] * 0.6931471805599453f + logf(l);
            if (p.cluster)
                sts4(smem + G::R * 512 + r * 4, lse);
            else if (parts)
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
                    mma_smem_8bit<G::N, 0>(tmem + i * G::N, k + j * 2, q + j * 2, j > 0, lead,
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
                    mma_smem_8bit<G::N, 1>(tmem + G::O_COL, a + j * (4096 >> 4),
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

// The queries of a block as e5m2 parts, a row's largest value in [2^14, 2^15) after a
// power-of-two scale; rows past the group (and past the parts) are 0.  16 threads to a row.
template <class G>
__device__ __forceinline__ void few_queries_e5m2(const AttnParams &p, const Work &w, uint32_t q_smem,
                                                 int lt, float *q_scale)
{
    const int c = lt & 15;
    auto store = [&](int row, uint2 v) {
        const uint32_t at = q_smem + row * 128 + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(v.x), "r"(v.y) : "memory");
    };
    if (G::N > 3 * G::R)
        store(3 * G::R + (lt >> 4), make_uint2(0, 0));
    for (int r = lt >> 4; r < G::R; r += 8) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < p.group)
            v = __ldg(reinterpret_cast<const uint4 *>(
                    p.q + w.q0 * p.q_ts + (int64_t)(w.head * p.group + r) * p.q_hs) + c);
        uint2 part[3];
        const float scale = query_e5m2(v, part);
#pragma unroll
        for (int k = 0; k < 3; ++k)
            store(k * G::R + r, part[k]);
        if (c == 0)
            q_scale[r] = scale;
    }
}

// The blocks of a cluster hold the parts of one (sequence, key head): each joins some of
// its rows.  `idle`: this block has no part (or gave up).
template <class G>
__device__ __forceinline__ void few_join(const AttnParams &p, const Work &w, uint32_t smem, int tid,
                                         bool idle)
{
    const uint32_t lse_at = smem + G::R * 512;
    if (idle && tid < G::R)
        sts4(lse_at + tid * 4, -INFINITY);
    __syncwarp();
    cluster_sync();
    for (int r = w.split; tid < 128 && r < p.group; r += p.max_splits) {
        float top = -INFINITY, sum = 0.0f, acc = 0.0f;
        for (int s = 0; s < p.max_splits; ++s)
            top = fmaxf(top, lds4_of(lse_at + r * 4, s));
        const float ref = top == -INFINITY ? 0.0f : top;
        for (int s = 0; s < p.max_splits; ++s) {
            const float lse = lds4_of(lse_at + r * 4, s);
            if (lse == -INFINITY)
                continue; // no part, or one that saw nothing
            const float wgt = expf(lse - ref);
            sum += wgt;
            acc = fmaf(wgt, lds4_of(smem + r * 512 + tid * 4, s), acc);
        }
        const int h = w.head * p.group + r;
        const float y = sum == 0.0f ? 0.0f : acc / sum;
        *reinterpret_cast<uint16_t *>(p.out + w.q0 * p.o_ts + h * p.o_hs + tid * 2) =
            (uint16_t)pack_bf16(y, y);
        if (tid == 0 && p.lse)
            p.lse[w.q0 * p.heads + h] = sum == 0.0f ? -INFINITY : ref + logf(sum);
    }
    __syncwarp();
    cluster_sync(); // no block leaves while another reads it
}

template <class G>
__global__ void __launch_bounds__(kFewThreads, 2) attention_few_kernel(
    const __grid_constant__ AttnParams p)
{
    extern __shared__ unsigned char raw_smem[];
    __shared__ uint32_t s_tmem, s_status;
    __shared__ volatile int s_abort;
    __shared__ FewRefs s_refs;
    __shared__ float s_qscale[kFewRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const uint32_t bars = smem + G::BAR_AT;

    // in a cluster the splits of a (sequence, key head) are neighbours; otherwise the
    // heads, whose values lie side by side
    const int x = (int)blockIdx.x;
    const int y = p.cluster ? p.by_splits.quotient(x) : p.by_heads.quotient(x);
    Work w;
    w.seq = p.cluster ? p.by_heads.quotient(y) : p.by_splits.quotient(y);
    w.split = p.cluster ? x - y * p.max_splits : y - w.seq * p.max_splits;
    w.head = p.cluster ? y - w.seq * p.kv_heads : x - y * p.kv_heads;
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
        if (p.cluster && w.n > 0 && !bad) // the other blocks of the cluster wait
            few_join<G>(p, w, smem, tid, true);
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
        few_softmax<G>(p, w, tmem, smem, bars, tid, &s_abort, s_refs, s_qscale);
    } else if (warp < 8) {
        const int lt = tid - 128;
        if constexpr (G::QUANT) {
            few_queries_e5m2<G>(p, w, smem + G::Q_AT, lt, s_qscale);
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
        load_heads<G>(p, w, smem, bars + kBarRing * 8, warp - 4, lane, true, &s_abort, out);
        if (out)
            s_status = kStatusOutOfRange;
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const uint32_t lead = elect_lane();
        bool ok = blockIdx.x != p.skip_block &&
                  bar_wait(bars + kBarQ * 8, 0, &s_abort, p.wait_limit_ns);
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
    if (p.cluster)
        few_join<G>(p, w, smem, tid, s_abort != 0);
    if (tid == 0)
        write_block_status(p.header, s_abort ? kStatusTimeout : s_status, blockIdx.x, p.status_words);
}

// Joins the parts of rows whose keys were split: a warp per (token, head).
__global__ void __launch_bounds__(256) few_join_kernel(const __grid_constant__ AttnParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t rows = p.total_q * p.heads;
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t tok = at / p.heads;
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
        Work w{};
        if (seq_queries(p, a, w.q0, w.n) && seq_keys(p, a, w.len) && w.n > 0 && tok == w.q0)
            splits = p.by_run.quotient(key_tiles<128, 1>(p, w) + p.split_tiles - 1);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (splits <= 1)
        return; // the row's block wrote it
    const int h = (int)(at - tok * p.heads);
    join_row<1>(
        splits, lane, p.out + tok * p.o_ts + h * p.o_hs, p.lse ? p.lse + at : nullptr,
        [&](int k, int) {
            return reinterpret_cast<const float4 *>(p.part + (k * rows + at) * 128);
        },
        [&](int k) { return p.part_lse + k * rows + at; });
}

template <class G>
cudaError_t launch_few(AttnParams &p, int64_t blocks, cudaStream_t stream)
{
    static_assert(G::BYTES <= 113 * 1024, "two blocks to an SM");
    set_boxes<G>(p);
    cudaError_t e = allow_smem<attention_few_kernel<G>>(G::BYTES);
    if (e != cudaSuccess)
        return e;
    if (p.cluster) {
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)p.max_splits;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(kFewThreads);
        cfg.dynamicSmemBytes = G::BYTES;
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, attention_few_kernel<G>, p);
    }
    attention_few_kernel<G><<<(unsigned)blocks, kFewThreads, G::BYTES, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    return p.max_splits == 1
               ? cudaSuccess
               : launch_join(few_join_kernel, p, (p.total_q * p.heads + 7) / 8, stream);
}

} // namespace

cudaError_t launch_attention_few(AttnParams &p, int64_t blocks, cudaStream_t stream)
{
    const bool quant = p.cs != nullptr;
    if (p.group <= 8)
        return quant ? launch_few<FewGeo<true, 8>>(p, blocks, stream)
                     : launch_few<FewGeo<false, 8>>(p, blocks, stream);
    return quant ? launch_few<FewGeo<true, 16>>(p, blocks, stream)
                 : launch_few<FewGeo<false, 16>>(p, blocks, stream);
}

} // namespace kvr
