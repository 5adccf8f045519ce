// kv_weights.cu -- what each cached key receives of the queries' attention:
//
//     w_k = keep * w_k + Σ_{i, h} exp(scale * q_ih . key_k - lse_ih)
//
// over the queries that see the key and all heads.  The products are turned round: keys
// are the M of the MMA, rows of queries its N, Sᵀ (128 keys x rows) = K Qᵀ, so that a thread
// has one key and sums its own row of tensor memory; nothing is exchanged until the end,
// and what a key row holds has no part in another key's sum.
//
// A block owns 128 keys of a sequence (two such tiles where there are many queries) and
// takes steps: a row tile (the tokens that fill 128 rows with the query heads of one key
// head) of one key head.  The steps of a key tile are divided among the blocks of a
// cluster, which add their sums up in the order of the blocks: equal calls give equal bits.
//
// Roles of a block's warps:
//   sum    8 a key tile, two threads to a key, one for each half of the columns: read S
//          from tensor memory, 2^(s * scale * log2 e - lse * log2 e), add up;
//   load   bring K and Q (boxes of tensor maps by one thread; e4m3 rows, and pools and
//          queries that boxes do not fit, by all of them);
//   lse    one warp brings the queries' lse, a step ahead;
//   mma    one warp issues every MMA.
#include <algorithm>

#include "kv_attn_tile.cuh"

namespace kvr {

namespace {

template <bool MLA_, bool QUANT_, bool HOLD_>
struct SumGeo {
    static constexpr bool MLA = MLA_, QUANT = QUANT_;
    static constexpr bool HOLD = HOLD_; // K of the block's head stays, Q passes
    static constexpr int KT = 128;
    static constexpr int NT = HOLD ? 2 : 1;       // key tiles of a block
    static constexpr int CHUNKS = MLA ? 9 : 1;    // of a step, and
    static constexpr int PANELS = MLA ? 1 : 2;    // panels of 64 columns of each
    static constexpr int K_CHUNK = NT * PANELS * 128 * 128; // bytes
    static constexpr int SUM_WARPS = 8 * NT, LOAD_WARPS = 4;
    static constexpr int LSE_WARP = SUM_WARPS + LOAD_WARPS, MMA_WARP = LSE_WARP + 1;
    static constexpr int THREADS = (MMA_WARP + 1) * 32;
    static constexpr int BLOCKS = HOLD ? 1 : 2;   // to an SM
    static constexpr int HELD = HOLD ? K_CHUNK : 0;
    static int stage_bytes(int n) { return (HOLD ? 0 : K_CHUNK) + PANELS * n * 128; }
};

constexpr int kSumMaxStages = 6;
constexpr int kSumSmem = 104 * 1024, kSumSmemAlone = 200 * 1024; // two blocks to an SM, one

// Barriers: K held, and free again; S of two buffers, and free again; lse likewise; then the
// ring's, full and empty.
enum { kBarK = 0, kBarKFree = 1, kBarSum = 2, kBarSumFree = 4, kBarLse = 6, kBarEnd = 8, kBarStage = 9 };

struct SumWork {
    int seq, n, len, base; // new tokens, cached ones, those before the new ones
    int q0;                // first query token
    int k0;                // first key
    int ra;                // first row tile, and
    int tiles;             // row tiles that see a key of the block
    int step0, step1;      // this block's steps: step s is row tile ra + s % tiles of head s / tiles
};

__device__ __forceinline__ void copy_box3(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                          uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// D (128 x n) of A (128 rows) and B (n rows), both along K.
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t desc,
                                         uint32_t acc, uint32_t lead)
{
    asm volatile("{\n.reg .pred p, q;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\n"
                 "setp.ne.b32 q, %6, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d),
                 "r"(a), "r"(b), "r"(desc), "r"(acc), "r"(kOperandHigh), "r"(lead)
                 : "memory");
}

__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// Keys of the block that some query sees exist; their tokens [i0, i1) of the block.
template <class G>
__device__ __forceinline__ void find_steps(const WeightsParams &p, SumWork &w, int rank)
{
    const AttnParams &a = p.a;
    const int k1 = min(w.len, w.k0 + G::NT * 128) - 1; // last key
    int i0 = 0, i1 = w.n;
    if (a.causal)
        i0 = max(0, w.k0 - w.base);
    if (a.window && w.k0 >= a.sinks)
        i1 = (int)min((int64_t)w.n, max((int64_t)0, (int64_t)k1 + a.window - w.base));
    w.ra = p.by_toks.quotient(i0);
    w.tiles = i1 <= i0 ? 0 : p.by_toks.quotient(i1 + p.toks - 1) - w.ra;
    const int64_t steps = (int64_t)w.tiles * a.kv_heads;
    w.step0 = (int)(steps * rank / p.parts);
    w.step1 = (int)(steps * (rank + 1) / p.parts);
}

// A step after another, without divisions.
struct Step {
    int head, tile; // of the sequence's row tiles

    __device__ Step(const SumWork &w, int s) : head(s / max(1, w.tiles)), tile(w.ra + s % max(1, w.tiles)) {}
    __device__ void next(const SumWork &w)
    {
        if (++tile == w.ra + w.tiles) {
            tile = w.ra;
            ++head;
        }
    }
};

// 16-byte pieces of a chunk of K by the load warps' threads: PER rows' worth to a thread at
// a time.  Asked for a chunk ahead, converted and stored when its stage is free.
template <class G>
struct HandKeys {
    static constexpr int TH = G::LOAD_WARPS * 32;
    // e4m3: 64 columns of a latent row are 4 pieces, a head's row 8; bf16: 8 and 16
    static constexpr int PIECES = G::QUANT ? (G::MLA ? 4 : 8) : (G::MLA ? 8 : 16);
    static constexpr int PER = 128 * PIECES / TH; // of a key tile

    // piece j of a thread: key row and piece of it
    __device__ static void at(int tid, int j, int &row, int &c)
    {
        const int i = tid + j * TH;
        row = i / PIECES;
        c = i % PIECES;
    }

    // `pe`: the chunk of k_pe, bf16 in both pools (two rounds of pieces in a quantised one)
    __device__ static uint4 load(const AttnParams &a, int64_t slot, int head, int chunk, int c)
    {
        if (slot < 0)
            return make_uint4(0, 0, 0, 0);
        const char *src;
        if (G::MLA)
            src = a.copy + slot * a.copy_ss + chunk * (G::QUANT ? 64 : 128);
        else
            src = a.rot + slot * a.rot_ss + head * (G::QUANT ? 128 : 256);
        return ld_stream(src + c * 16);
    }

    __device__ static float scale(const AttnParams &a, int64_t slot, int head, int chunk)
    {
        if (!G::QUANT || slot < 0)
            return 1.0f;
        return __ldg(G::MLA ? a.cs + slot * a.cs_ss + (chunk >> 1) : a.rs + slot * a.rs_ss + head);
    }

    __device__ static void store(uint32_t dst, int row, int c, uint4 v, float scale)
    {
        const uint32_t at = dst + row * 128, sw = row & 7;
        if (!G::QUANT) {
            sts16(at + ((c >> 3) << 14) + (((c & 7) ^ sw) << 4), v);
            return;
        }
        uint4 lo, hi;
        const uint32_t mul = scale_mul(scale);
        if (rare16(v, mul))
            convert16<true>(v, mul, lo, hi);
        else
            convert16<false>(v, mul, lo, hi);
        const int c2 = 2 * c;
        sts16(at + ((c2 >> 3) << 14) + (((c2 & 7) ^ sw) << 4), lo);
        sts16(at + ((c2 >> 3) << 14) + ((((c2 + 1) & 7) ^ sw) << 4), hi);
    }
};

template <class G>
__global__ void __launch_bounds__(G::THREADS, G::BLOCKS) weights_kernel(
    const __grid_constant__ WeightsParams p)
{
    const AttnParams &a = p.a;
    extern __shared__ unsigned char raw_smem[];
    __shared__ __align__(8) uint64_t s_bars[kBarStage + 2 * kSumMaxStages];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ int s_bad;
    __shared__ int64_t s_slot[G::NT * 128]; // of the block's keys; -1: none
    __shared__ __align__(16) float s_off[2][128];
    __shared__ float s_sum[2][G::NT * 128];
    __shared__ float s_part[G::NT * 128 + 1]; // and whether the block gave up
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)blockIdx.x % p.parts, unit = (int)blockIdx.x / p.parts;
    const int tile = unit / a.num_seqs, seq = unit - tile * a.num_seqs;
    auto leave = [&](uint32_t code) {
        if (tid == 0)
            write_block_status(a.header, code, blockIdx.x, gridDim.x);
    };
    SumWork w{};
    w.seq = seq;
    int64_t q0;
    const bool fits = seq_queries(a, seq, q0, w.n) && seq_keys(a, seq, w.len);
    w.q0 = (int)q0;
    w.base = w.len - w.n;
    w.k0 = tile * G::NT * 128;
    if (!fits || w.k0 >= w.len) { // the same for the whole cluster
        leave(fits || tile > 0 ? kStatusOk : kStatusOutOfRange);
        return;
    }
    find_steps<G>(p, w, rank);

    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const uint32_t ring = smem + G::HELD;
    const uint32_t stage_bytes = (G::HOLD ? 0 : G::K_CHUNK) + G::PANELS * p.n * 128;
    const uint32_t q_in_stage = G::HOLD ? 0 : G::K_CHUNK;
    const uint32_t bars = smem_u32(s_bars);
    const uint32_t full = bars + kBarStage * 8, empty = full + kSumMaxStages * 8;
    const bool k_boxes = !G::QUANT && a.box_rows > 0;
    const bool hand = !k_boxes || !p.q_boxes;
    const uint32_t columns = G::NT * p.n * 2 <= 32 ? 32 : G::NT * p.n * 2 <= 64 ? 64
                           : G::NT * p.n * 2 <= 128 ? 128 : G::NT * p.n * 2 <= 256 ? 256 : 512;
    if (warp == G::MMA_WARP) {
        tmem_alloc(smem_u32(&s_tmem), columns);
    } else if (tid == 0) {
        s_abort = 0;
        s_bad = 0;
        const uint32_t fill = hand ? 1 + G::LOAD_WARPS * 32 : 1;
        bar_init(bars + kBarK * 8, fill);
        bar_init(bars + kBarKFree * 8, 1);
        bar_init(bars + kBarEnd * 8, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(bars + (kBarSum + i) * 8, 1);
            bar_init(bars + (kBarSumFree + i) * 8, G::SUM_WARPS * 32);
            bar_init(bars + (kBarLse + i) * 8, 32);
        }
        for (int i = 0; i < p.stages; ++i) {
            bar_init(full + i * 8, fill);
            bar_init(empty + i * 8, 1);
        }
        bar_init_fence();
    }
    // rows that pad Q, and the slots of the keys
    for (int i = tid; i < p.stages * G::PANELS * (p.n - p.rows) * 8; i += G::THREADS) {
        const int c = i & 7, r = i >> 3, pad = p.n - p.rows;
        const int panel = r / pad % G::PANELS, st = r / pad / G::PANELS;
        sts16(ring + st * stage_bytes + q_in_stage + (panel * p.n + p.rows + r % pad) * 128 + c * 16,
              make_uint4(0, 0, 0, 0));
    }
    for (int i = tid; i < G::NT * 128; i += G::THREADS) {
        const int k = w.k0 + i;
        int64_t s = -1;
        if (k < w.len) {
            const int b = a.by_block.quotient(k);
            const int32_t blk = __ldg(a.block_tables + (int64_t)seq * a.max_blocks + b);
            if (blk >= 0 && blk < a.num_blocks)
                s = (int64_t)blk * a.block + (k - b * a.block);
        }
        s_slot[i] = s;
    }
    async_fence();
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    const int64_t limit = a.wait_limit_ns;

    if (warp < G::SUM_WARPS) {
        const int t = warp >> 3, half = (warp >> 2) & 1;
        const int key = t * 128 + (warp & 3) * 32 + lane, k = w.k0 + key;
        const bool mine = s_slot[key] >= 0;
        if (k < w.len && !mine && half == 0)
            s_bad = 1;
        const float c = a.scale * 1.4426950408889634f;
        const f2 c2 = f2_of_bits(__float_as_uint(c), __float_as_uint(c));
        // tokens that see this key: [lo, hi)
        const int lo = a.causal ? max(0, k - w.base) : 0;
        const int hi = !mine ? 0
                     : a.window && k >= a.sinks
                         ? (int)max((int64_t)0, min((int64_t)w.n, (int64_t)k + a.window - w.base))
                         : w.n;
        // and those that see every key of this tile
        const int k1 = w.k0 + t * 128 + 127;
        const int all_lo = a.causal ? max(0, k1 - w.base) : 0;
        const int all_hi = a.window && k1 >= a.sinks
                               ? (int)max((int64_t)0, min((int64_t)w.n, (int64_t)w.k0 + t * 128 +
                                                                            a.window - w.base))
                               : w.n;
        f2 sum = 0ull;
        Step st(w, w.step0);
        for (int s = w.step0; s < w.step1; ++s, st.next(w)) {
            const int i = s - w.step0, buf = i & 1;
            if (!bar_wait(bars + (kBarLse + buf) * 8, (i >> 1) & 1, &s_abort, limit) ||
                !bar_wait(bars + (kBarSum + buf) * 8, (i >> 1) & 1, &s_abort, limit))
                break;
            mma_fence_after();
            const int tok0 = st.tile * p.toks;
            const bool whole = mine && tok0 >= all_lo && tok0 + p.toks <= all_hi;
            // columns of the tokens that see this key
            const int c_lo = (max(lo, tok0) - tok0) * a.group;
            const int c_hi = (min(hi, tok0 + p.toks) - tok0) * a.group;
            f2 part[2] = {0ull, 0ull};
            for (int at = half * 32; at < p.n; at += 64) {
                uint32_t x[32];
                tmem_ld32(s_tmem + (buf * G::NT + t) * p.n + at + ((uint32_t)((warp & 3) * 32) << 16), x);
                tmem_ld_wait();
                tmem_pin32(x);
                const float *off = s_off[buf] + at;
                if (__all_sync(0xFFFFFFFFu, whole)) {
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float4 o = *reinterpret_cast<const float4 *>(off + 2 * j);
                        const f2 y0 = f2_fma(f2_of_bits(x[2 * j], x[2 * j + 1]), c2,
                                             f2_of_bits(__float_as_uint(o.x), __float_as_uint(o.y)));
                        const f2 y1 = f2_fma(f2_of_bits(x[2 * j + 2], x[2 * j + 3]), c2,
                                             f2_of_bits(__float_as_uint(o.z), __float_as_uint(o.w)));
                        float e0, e1, e2, e3;
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(e0), "=f"(e1) : "l"(y0));
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(e2), "=f"(e3) : "l"(y1));
                        part[0] = f2_add(part[0], f2_of_bits(__float_as_uint(exp2_fast(e0)),
                                                             __float_as_uint(exp2_fast(e1))));
                        part[1] = f2_add(part[1], f2_of_bits(__float_as_uint(exp2_fast(e2)),
                                                             __float_as_uint(exp2_fast(e3))));
                    }
                } else {
                    const uint32_t see = low_bits(c_hi - at) & ~low_bits(c_lo - at);
                    float add[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float e = exp2_fast(fmaf(__uint_as_float(x[j]), c, off[j]));
                        add[j & 1] += (see >> j) & 1u ? e : 0.0f;
                    }
                    part[0] = f2_add(part[0], f2_of_bits(__float_as_uint(add[0]), __float_as_uint(add[1])));
                }
            }
            sum = f2_add(sum, f2_add(part[0], part[1]));
            mma_fence_before();
            bar_signal(bars + (kBarSumFree + buf) * 8);
        }
        float s0, s1;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(sum));
        s_sum[half][key] = s0 + s1;
    } else if (warp < G::LSE_WARP) {
        const int lt = tid - G::SUM_WARPS * 32;
        if (hand || lt < 32) {
            using H = HandKeys<G>;
            int stage = 0, phase = 1, filled = 0;
            bool ok = true;
            Step st(w, w.step0);
            int held = -1, heads = 0; // HOLD: the head whose K is held; how many there were
            // K by boxes: a lane's box of a key tile
            const int per = k_boxes ? 128 / a.box_rows : 0;
            auto boxes = [&](uint32_t dst, uint32_t bar, int head, int chunk, bool ask) {
                uint32_t bytes = 0;
#pragma unroll
                for (int t = 0; t < G::NT; ++t) {
                    const int64_t slot = lane < per ? s_slot[t * 128 + lane * a.box_rows] : -1;
                    const uint32_t who = __ballot_sync(0xFFFFFFFFu, slot >= 0);
                    bytes += __popc(who) * a.box_rows * 128 * G::PANELS;
                    if (!ask || slot < 0)
                        continue;
                    const uint32_t to = dst + t * (G::PANELS << 14) + lane * a.box_rows * 128;
                    if (G::MLA) {
                        if (chunk < 8)
                            copy_box(to, &a.copy_map, chunk * 64, (int)slot, bar);
                        else
                            copy_box(to, &a.rot_map, 0, (int)slot, bar);
                    } else {
                        copy_box(to, &a.rot_map, head * 128, (int)slot, bar);
                        copy_box(to + 16384, &a.rot_map, head * 128 + 64, (int)slot, bar);
                    }
                }
                return bytes;
            };
            auto by_hand = [&](uint32_t dst, int head, int chunk) {
#pragma unroll 1
                for (int t = 0; t < G::NT; ++t) {
                    const uint32_t to = dst + t * (G::PANELS << 14);
                    if (G::MLA && chunk == 8) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int i = lt + j * H::TH, row = i >> 3, c = i & 7;
                            const int64_t s = s_slot[t * 128 + row];
                            const uint4 v = s < 0 ? make_uint4(0, 0, 0, 0)
                                                  : ld_stream(a.rot + s * a.rot_ss + c * 16);
                            sts16(to + row * 128 + ((c ^ (row & 7)) << 4), v);
                        }
                        continue;
                    }
                    constexpr int B = H::PER < 8 ? H::PER : 8;
#pragma unroll 1
                    for (int j0 = 0; j0 < H::PER; j0 += B) {
                        uint4 v[B];
                        float sc[B];
#pragma unroll
                        for (int j = 0; j < B; ++j) {
                            int row, c;
                            H::at(lt, j0 + j, row, c);
                            const int64_t s = s_slot[t * 128 + row];
                            v[j] = H::load(a, s, head, chunk, c);
                            sc[j] = H::scale(a, s, head, chunk);
                        }
#pragma unroll
                        for (int j = 0; j < B; ++j) {
                            int row, c;
                            H::at(lt, j0 + j, row, c);
                            H::store(to, row, c, v[j], sc[j]);
                        }
                    }
                }
            };
            auto queries = [&](uint32_t dst, int chunk) { // by hand
                for (int i = lt; i < p.rows * G::PANELS * 8; i += H::TH) {
                    const int c = i % (G::PANELS * 8), r = i / (G::PANELS * 8);
                    const int tok = a.by_group.quotient(r), g = r - tok * a.group;
                    const int at = st.tile * p.toks + tok;
                    const uint4 v =
                        at >= w.n ? make_uint4(0, 0, 0, 0)
                                  : __ldg(reinterpret_cast<const uint4 *>(
                                        a.q + (int64_t)(w.q0 + at) * a.q_ts +
                                        (int64_t)(st.head * a.group + g) * a.q_hs + chunk * 128 + c * 16));
                    sts16(dst + ((c >> 3) * p.n + r) * 128 + (((c & 7) ^ (r & 7)) << 4), v);
                }
            };
            for (int s = w.step0; ok && s < w.step1; ++s, st.next(w)) {
                if (G::HOLD && st.head != held) {
                    // the MMAs of the head before are done with K
                    ok = heads == 0 || bar_wait(bars + kBarKFree * 8, (heads - 1) & 1, &s_abort, limit);
                    if (!ok)
                        break;
                    held = st.head;
                    ++heads;
                    const uint32_t bar = bars + kBarK * 8;
                    if (lt < 32) {
                        const uint32_t bytes = k_boxes ? boxes(smem, bar, held, 0, false) : 0;
                        if (lane == 0)
                            bar_signal_bulk(bar, 1, bytes);
                        __syncwarp();
                        if (k_boxes)
                            boxes(smem, bar, held, 0, true);
                    }
                    if (hand) {
                        if (!k_boxes)
                            by_hand(smem, held, 0);
                        async_fence();
                        bar_signal(bar);
                    }
                }
                for (int chunk = 0; chunk < G::CHUNKS; ++chunk) {
                    ok = bar_wait(empty + stage * 8, phase, &s_abort, limit);
                    if (!ok)
                        break;
                    const uint32_t at = ring + stage * stage_bytes, bar = full + stage * 8;
                    if (lt < 32) {
                        uint32_t bytes = p.q_boxes ? p.rows * G::PANELS * 128 : 0;
                        if (!G::HOLD && k_boxes)
                            bytes += boxes(at, bar, st.head, chunk, false);
                        if (lane == 0) {
                            bar_signal_bulk(bar, 1, bytes);
                            if (p.q_boxes)
#pragma unroll
                                for (int i = 0; i < G::PANELS; ++i)
                                    copy_box3(at + q_in_stage + i * p.n * 128, &p.q_map,
                                              (chunk * G::PANELS + i) * 64, st.head * a.group,
                                              w.q0 + st.tile * p.toks, bar);
                        }
                        __syncwarp();
                        if (!G::HOLD && k_boxes)
                            boxes(at, bar, st.head, chunk, true);
                    }
                    if (hand) {
                        if (!G::HOLD && !k_boxes)
                            by_hand(at, st.head, chunk);
                        if (!p.q_boxes)
                            queries(at + q_in_stage, chunk);
                        async_fence();
                        bar_signal(bar);
                    }
                    ++filled;
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // boxes in flight land before the block's memory goes, also after an early end
            if (lt < 32) {
                int none = 0;
                if (G::HOLD && heads > 0)
                    bar_wait(bars + kBarK * 8, (heads - 1) & 1, &none, 10000000ll);
                for (int i = 0; i < p.stages; ++i)
                    if (filled > i)
                        bar_wait(full + i * 8, ((filled - 1 - i) / p.stages) & 1, &none, 10000000ll);
            }
        }
    } else if (warp == G::LSE_WARP) {
        // -lse * log2 e of a step's rows, four to a lane; -inf: the row counts nothing
        auto fetch = [&](const Step &st) {
            float4 r;
            float *v = &r.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = lane * 4 + j;
                const int tok = a.by_group.quotient(col), at = st.tile * p.toks + tok;
                float x = -INFINITY;
                if (col < p.rows && at < w.n)
                    x = __ldg(p.lse + (int64_t)(w.q0 + at) * a.heads + st.head * a.group +
                              (col - tok * a.group));
                v[j] = x == -INFINITY ? -INFINITY : -x * 1.4426950408889634f;
            }
            return r;
        };
        if (w.step0 < w.step1) {
            Step st(w, w.step0);
            float4 next = fetch(st);
            for (int s = w.step0; s < w.step1; ++s) {
                const int i = s - w.step0, buf = i & 1;
                const float4 now = next;
                if (s + 1 < w.step1) {
                    st.next(w);
                    next = fetch(st);
                }
                if (i >= 2 && !bar_wait(bars + (kBarSumFree + buf) * 8, ((i >> 1) - 1) & 1, &s_abort, limit))
                    break;
                *reinterpret_cast<float4 *>(&s_off[buf][lane * 4]) = now;
                bar_signal(bars + (kBarLse + buf) * 8);
            }
        }
    } else {
        const uint32_t lead = elect_lane(), tmem = s_tmem;
        const uint32_t desc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(p.n >> 3) << 17) |
                              ((uint32_t)(kRows >> 4) << 24);
        int stage = 0, phase = 0, held = -1, heads = 0;
        bool ok = blockIdx.x != a.skip_block;
        Step st(w, w.step0);
        for (int s = w.step0; ok && s < w.step1; ++s) {
            const int i = s - w.step0, buf = i & 1;
            if (i >= 2)
                ok = bar_wait(bars + (kBarSumFree + buf) * 8, ((i >> 1) - 1) & 1, &s_abort, limit);
            if (G::HOLD && ok && st.head != held) {
                held = st.head;
                ok = bar_wait(bars + kBarK * 8, heads & 1, &s_abort, limit);
                ++heads;
            }
            mma_fence_after();
            for (int chunk = 0; ok && chunk < G::CHUNKS; ++chunk) {
                ok = bar_wait(full + stage * 8, phase, &s_abort, limit);
                if (!ok)
                    break;
                async_fence();
                const uint32_t at = ring + stage * stage_bytes;
                const uint32_t q = operand(at + q_in_stage, 16);
#pragma unroll
                for (int t = 0; t < G::NT; ++t) {
                    const uint32_t d = tmem + (buf * G::NT + t) * p.n;
                    const uint32_t k = operand((G::HOLD ? smem : at) + t * (G::PANELS << 14), 16);
#pragma unroll
                    for (int pn = 0; pn < G::PANELS; ++pn)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_rows(d, k + pn * (16384 >> 4) + kk * 2, q + pn * (p.n * 128 >> 4) + kk * 2,
                                     desc, chunk > 0 || pn > 0 || kk > 0, lead);
                }
                bar_signal_mma(empty + stage * 8, lead);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok)
                break;
            bar_signal_mma(bars + (kBarSum + buf) * 8, lead);
            st.next(w);
            if (G::HOLD && (s + 1 == w.step1 || st.head != held))
                bar_signal_mma(bars + kBarKFree * 8, lead);
        }
        // every MMA is done before tensor memory goes
        int none = 0;
        if (blockIdx.x == a.skip_block)
            s_abort = 1;
        bar_signal_mma(bars + kBarEnd * 8, lead);
        bar_wait(bars + kBarEnd * 8, 0, &none, 1000000000ll);
        __syncwarp();
    }
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    if (warp == G::MMA_WARP)
        tmem_free(s_tmem, columns);
    if (tid < G::NT * 128)
        s_part[tid] = s_sum[0][tid] + s_sum[1][tid];
    if (tid == 0)
        s_part[G::NT * 128] = s_abort ? 1.0f : 0.0f;
    cluster_sync();
    if (rank == 0 && tid < G::NT * 128 && w.k0 + tid < w.len) {
        float sum = 0.0f, gave_up = 0.0f;
        for (int r = 0; r < p.parts; ++r) {
            sum += lds4_of(smem_u32(&s_part[tid]), r);
            gave_up += lds4_of(smem_u32(&s_part[G::NT * 128]), r);
        }
        float *const to = p.weights + seq * p.weight_stride + w.k0 + tid;
        if (gave_up == 0.0f)
            *to = p.keep == 0.0f ? sum : fmaf(p.keep, *to, sum);
    }
    cluster_sync(); // the others' sums have been read
    leave(s_abort ? kStatusTimeout : s_bad ? kStatusOutOfRange : kStatusOk);
}

template <class G>
cudaError_t launch(WeightsParams &p, const WeightsPlan &pl, cudaStream_t stream)
{
    p.a.box_rows = 0;
    if (!G::QUANT)
        set_boxes<G>(p.a);
    cudaError_t e = allow_smem<weights_kernel<G>>(kSumSmemAlone + 1024);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)pl.parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)pl.blocks);
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = (size_t)pl.smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_kernel<G>, p);
}

// Query rows as boxes: `toks` tokens of the heads of one key head, 64 columns.
bool encode_queries(WeightsParams &p, int width)
{
    const auto encode = map_encoder();
    const AttnParams &a = p.a;
    if (!encode)
        return false;
    const int64_t row = width * 2, hs = a.heads > 1 ? a.q_hs : row;
    const int64_t ts = a.total_q > 1 ? a.q_ts : std::max(hs * a.heads, row);
    if (hs <= 0 || ts <= 0)
        return false; // queries that share their memory
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)a.heads, (cuuint64_t)a.total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)hs, (cuuint64_t)ts};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)p.toks}, step[3] = {1, 1, 1};
    return encode(&p.q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<char *>(a.q), dims,
                  strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace

WeightsPlan plan_weights(RowKind kind, const AttnShape &a)
{
    const bool mla = kind == RowKind::Mla;
    WeightsPlan pl{};
    const int32_t group = a.group;
    pl.toks = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kRows / group, a.max_q_len));
    pl.rows = pl.toks * group;
    pl.n = (pl.rows + 31) / 32 * 32;
    const int64_t row_tiles = std::max<int64_t>(1, (a.max_q_len + pl.toks - 1) / pl.toks);
    pl.hold = !mla && row_tiles > 1;
    const int64_t keys = pl.hold ? 256 : 128;
    const int64_t units = a.num_seqs * std::max<int64_t>(1, (a.max_kv_len + keys - 1) / keys);
    const int64_t steps = row_tiles * a.kv_heads;
    pl.parts = 1; // enough blocks for a few rounds
    while (pl.parts < 8 && units * pl.parts < 4 * kSms && steps >= 2 * pl.parts)
        pl.parts *= 2;
    pl.blocks = units * pl.parts;
    const int held = pl.hold ? 2 * 2 * 128 * 128 : 0;
    const int stage = (pl.hold ? 0 : (mla ? 1 : 2) * 128 * 128) + (mla ? 1 : 2) * pl.n * 128;
    const int room = pl.hold || 2 * stage > kSumSmem ? kSumSmemAlone : kSumSmem;
    pl.stages = std::min(kSumMaxStages, (room - held) / stage);
    pl.smem = held + pl.stages * stage + 1024;
    return pl;
}

cudaError_t launch_weights(WeightsParams &p, RowKind kind, const WeightsPlan &pl,
                           cudaStream_t stream)
{
    const bool quant = p.a.cs != nullptr;
    p.toks = pl.toks;
    p.rows = pl.rows;
    p.n = pl.n;
    p.parts = pl.parts;
    p.stages = pl.stages;
    p.by_toks = Divisor((uint32_t)pl.toks);
    p.a.by_group = Divisor((uint32_t)p.a.group);
    p.a.by_block = Divisor((uint32_t)p.a.block);
    p.q_boxes = encode_queries(p, kind == RowKind::Mla ? 576 : 128);
    if (kind == RowKind::Mla)
        return quant ? launch<SumGeo<true, true, false>>(p, pl, stream)
                     : launch<SumGeo<true, false, false>>(p, pl, stream);
    if (pl.hold)
        return quant ? launch<SumGeo<false, true, true>>(p, pl, stream)
                     : launch<SumGeo<false, false, true>>(p, pl, stream);
    return quant ? launch<SumGeo<false, true, false>>(p, pl, stream)
                 : launch<SumGeo<false, false, false>>(p, pl, stream);
}

} // namespace kvr
