// kv_attn_tile.cuh -- what the attention kernels share: a block's work (rows, key tiles,
// masks), head rows on their way into the ring, and the join of split rows.
#pragma once

#include <algorithm>
#include <atomic>

#include "kv_attn_ptx.cuh"

namespace kvr {

// Barriers of a block: queries there; O complete; per row tile or buffer: S ready, P
// ready; a step of O and (its neighbour) what was issued has finished; then the ring's,
// full and empty.
enum { kBarQ = 0, kBarDone = 1, kBarS = 2, kBarP = 4, kBarO = 6, kBarRing = 8 };

constexpr int kFewRows = 16; // rows of attention_few_kernel

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

// Keys [k, k + 32) that new token `tok` of a sequence's tree sees, a bit each: those before
// the new tokens (from `base` on) and what its mask says.
__device__ __forceinline__ uint32_t tree_bits(const AttnParams &p, int64_t tok, int base, int k)
{
    const int64_t b = (int64_t)k - base; // the mask's bit of key k
    if (b <= -32)
        return ~0u;
    const uint32_t *const words = p.tree + tok * p.tree_stride;
    auto word = [&](int64_t i) { return i < p.tree_words ? __ldg(words + i) : 0u; };
    if (b < 0)
        return word(0) << (uint32_t)-b | ((1u << (uint32_t)-b) - 1u);
    return __funnelshift_r(word(b >> 5), word((b >> 5) + 1), (uint32_t)b & 31u);
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

// Queries [a, b) of a sequence, n of them; false (and none) when they do not fit what the
// call stated.  Likewise its keys.
__device__ __forceinline__ bool queries_fit(const AttnParams &p, int a, int b, int &n)
{
    const bool fit = a >= 0 && b >= a && b <= p.total_q && b - a <= p.max_q_len;
    n = fit ? b - a : 0;
    return fit;
}

__device__ __forceinline__ bool keys_fit(const AttnParams &p, int len)
{
    return len >= 0 && len <= p.max_kv_len && (int64_t)len <= p.max_keys;
}

__device__ __forceinline__ bool seq_queries(const AttnParams &p, int s, int64_t &q0, int &n)
{
    q0 = p.q_off[s];
    return queries_fit(p, (int)q0, p.q_off[s + 1], n);
}

__device__ __forceinline__ bool seq_keys(const AttnParams &p, int s, int &len)
{
    len = p.kv_len[s];
    return keys_fit(p, len);
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
// Queries in three e5m2 parts
// ---------------------------------------------------------------------------

// Two values to e5m2 parts x = a + b / 8 + c / 64.
__device__ __forceinline__ void split_e5m2(float x, float y, uint32_t (&part)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint16_t h;
        uint32_t w;
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y), "f"(x));
        part[i] = h;
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(w) : "h"(h));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        x = (x - f.x) * 8.0f;
        y = (y - f.y) * 8.0f;
    }
}

// Eight values to eight bytes of each part.
__device__ __forceinline__ void split8(const float *x, uint2 (&to)[3])
{
    uint32_t h[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        split_e5m2(x[2 * i], x[2 * i + 1], h[i]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
        to[k] = make_uint2(h[0][k] | (h[1][k] << 16), h[2][k] | (h[3][k] << 16));
}

// Eight values of a query row to e5m2 parts, 16 threads to a row: its largest value in [2^14,
// 2^15) after the power-of-two scale that is returned.  What was infinite is NaN.
__device__ __forceinline__ float query_e5m2(uint4 v, uint2 (&part)[3])
{
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
    // 2^e of the row's scale: the exponent of its largest value, less 14
    const int e = max((int)(m >> 7) - 141, -120);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16) * inv;
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u) * inv;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) // what was infinite is NaN
        x[i] = fabsf(x[i]) < 32768.0f ? x[i] : __uint_as_float(0x7FC00000u);
    split8(x, part);
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// ---------------------------------------------------------------------------
// Copies into the ring
// ---------------------------------------------------------------------------

// Every key of tile kt is seen by some row: its rows can be copied as they are.
template <int KT>
__device__ __forceinline__ bool tile_whole(const Work &w, int kt)
{
    const int k0 = kt * KT;
    return (k0 >= w.lo && k0 + KT <= w.hi) || k0 + KT <= w.sk;
}

// Some key of [k, k + n) is seen by some row.
__device__ __forceinline__ bool keys_seen(const Work &w, int k, int n)
{
    return (k < w.hi && k + n > w.lo) || k < w.sk;
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
// time of its MMAs.  Tiles that hold keys nobody sees (`careful`: otherwise they are
// boxes too, with zeros only for boxes of which nobody sees a key), and pools whose
// blocks do not divide a tile, are copied row by row by all warps with zeros in the
// place of those keys: a lane owns one key row of its warp, 16 lanes copy 256 bytes (8
// lanes 128); that takes 4000 clocks a tile, where its MMAs take 2100.  The warps meet after every run, so none waits for a stage that is more than
// one phase away, which a parity would not show; a warp whose wait ran out goes on to
// the next meeting, where they all give up.
template <class G>
__device__ __forceinline__ void load_heads(const AttnParams &p, const Work &w, uint32_t ring,
                                           uint32_t bars, int warp, int lane, bool careful,
                                           volatile int *abort, bool &bad)
{
    constexpr int WARPS = G::LOAD_WARPS, ROWS = G::KT / WARPS; // rows of a warp: 32 or 16
    constexpr int PIECES = G::STAGE / G::KT / 16, PER = 32 / PIECES; // of a row; rows at a time
    const int base = warp * ROWS;
    const int c = lane & (PIECES - 1), sub = lane / PIECES;
    const int32_t *const table = p.block_tables + (int64_t)w.seq * p.max_blocks;
    auto whole = [&](int v) {
        return p.box_rows > 0 && (!careful || tile_whole<G::KT>(w, real_tile(w, v)));
    };
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
                auto seen = [&](int kt) { // this lane's box
                    return mine && keys_seen(w, kt * G::KT + lane * p.box_rows, p.box_rows);
                };
                int kt = real_tile(w, v);
                bool see = seen(kt);
                int32_t blk = see ? __ldg(table + block_of(kt)) : 0;
                for (int u = v; ok && u < last; ++u) {
                    const int row = (in == 1 ? 0 : (kt % in) * G::KT) + blk * p.block;
                    const bool fits = (uint32_t)blk < (uint32_t)p.num_blocks;
                    bad |= !fits;
                    const int y = see && fits ? row : (int)(p.num_blocks * p.block); // else zeros
                    kt = real_tile(w, u + 1);
                    see = u + 1 < last && seen(kt);
                    blk = see ? __ldg(table + block_of(kt)) : 0;
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

// ---------------------------------------------------------------------------
// Split rows, launches
// ---------------------------------------------------------------------------

// One row's parts into its result, by a warp:
//   lse = log Σ exp(lse_s),  out = Σ exp(lse_s - lse) out_s
// V float4 to a lane; part(s, v) and lse(s) say where they lie.  The first parts are asked
// for before their weights are known.
template <int V, class PartAt, class LseAt>
__device__ __forceinline__ void join_row(int splits, int lane, char *out, float *out_lse,
                                         PartAt part, LseAt lse)
{
    constexpr int AHEAD = 2;
    float4 x[AHEAD][V];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v)
            x[k][v] = part(k, v)[lane];
    const float my = lane < splits ? *lse(lane) : -INFINITY;
    float top = my;
    for (int k = 32 + lane; k < splits; k += 32)
        top = fmaxf(top, *lse(k));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float ref = top == -INFINITY ? 0.0f : top;
    float acc[V][4] = {}, sum = 0.0f;
    auto add = [&](int k, const float4 (&y)[V]) {
        const float wgt = expf((k < 32 ? __shfl_sync(0xFFFFFFFFu, my, k) : *lse(k)) - ref);
        sum += wgt;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            acc[v][0] = fmaf(wgt, y[v].x, acc[v][0]);
            acc[v][1] = fmaf(wgt, y[v].y, acc[v][1]);
            acc[v][2] = fmaf(wgt, y[v].z, acc[v][2]);
            acc[v][3] = fmaf(wgt, y[v].w, acc[v][3]);
        }
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        add(k, x[k]);
#pragma unroll 2
    for (int k = AHEAD; k < splits; ++k) {
        float4 y[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            y[v] = part(k, v)[lane];
        add(k, y);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v)
        *reinterpret_cast<uint2 *>(out + (v * 128 + lane * 4) * 2) =
            make_uint2(pack_bf16(acc[v][0] * inv, acc[v][1] * inv),
                       pack_bf16(acc[v][2] * inv, acc[v][3] * inv));
    if (lane == 0 && out_lse)
        *out_lse = sum == 0.0f ? -INFINITY : ref + logf(sum);
}

// The driver's function that makes tensor maps (nullptr: there is none).
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
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
    return encode;
}

// Tensor map of one part of the pool's rows (`width` columns of bf16 or bytes): boxes
// of 128 bytes and p.box_rows rows, swizzled as the MMAs read them.
inline bool encode_map(CUtensorMap *map, const char *base, int64_t row_bytes, int64_t rows, int width,
                int box_rows, bool bytes)
{
    const auto encode = map_encoder();
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

// A kernel that joins the parts of the one before: it starts while the last blocks of that
// one run and waits for them on the device.
inline cudaError_t launch_join(void (*kernel)(AttnParams), const AttnParams &p, int64_t blocks,
                               cudaStream_t stream)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
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

// One new token per sequence, up to kFewRows query heads to a key head
// (kv_attention_few.cu).
cudaError_t launch_attention_few(AttnParams &p, int64_t blocks, cudaStream_t stream);

} // namespace kvr
