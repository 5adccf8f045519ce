// kv_attention.cu -- attention of new tokens over the paged cache on the
// 5th-generation tensor cores (tcgen05).
//
//     S = scale * Q Kᵀ,  O = softmax(S) V,  lse = log Σ exp(S)
//
// for one layer of a paged pool, with one pass over the keys: for a tile of
// keys the running maximum m and sum l of every query row are updated, the
// weights 2^((s - m) * scale * log2 e) are rounded to bf16 and multiplied with
// V onto the accumulator O, which is rescaled when m moves.  bf16 because an MMA takes
// both operands in one type and V is bf16; it is 2^-8 of each weight, as much as the
// rounding of out, and l sums the unrounded ones.
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
//   mma      one warp issues every MMA;
//   find     one warp finds the next unit of work and sets its barriers up.
// O stays in tensor memory.  It is rescaled only when some row's maximum grew by
// more than 2^8 since it was last fixed: until then the weights stay below 2^8,
// which fp32 sums and bf16 weights hold without loss.
//
// The keys of a call are divided evenly over the SMs (Slices, below); a (row tile, head)
// that is cut is written as normalised fp32 parts with their lse, which a second kernel
// joins.  The cuts follow from the call's lengths, so results repeat bit for bit.
//
// Bound: the tensor cores and the softmax beside them.  4096 tokens over 16384, 32 heads
// over 8: 690 us, 1390 TFLOP/s, 0.74 of the rate of a large matrix product; of a tile's
// 2700 clocks the MMAs take 2100.  MLA (32 ragged sequences of up to 16384, 128 heads: 123
// us): 2600 clocks a 64-key tile, 2070 of MMAs; the operands that they read from shared
// memory and the copies into it share its 128 bytes a clock.
//
// Every wait is bounded; a block whose wait runs out reports KV_ERR_TIMEOUT.
#include <algorithm>
#include <type_traits>

#include "kv_attn_tile.cuh"

namespace kvr {

namespace {

constexpr int64_t kExpandBytes = int64_t(2) << 30; // largest workspace for widened rows
constexpr int64_t kPrefetchWait = 20000; // ns that a warp waits before it prefetches anyway
constexpr float kLazy = 8.0f;      // log2 of the growth of a maximum that O tolerates

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
    static constexpr int HALVES = 1, JOIN_BLOCKS = 4, UNIT_COST = NT == 2 ? 4 : 6; // see Slices
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
    static constexpr int HALVES = 2, JOIN_BLOCKS = 8, UNIT_COST = 6;
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

constexpr int kSoftRegs = 96, kLoadRegs = 48, kMmaRegs = 48;

template <class G>
constexpr int kAttnThreads = (kMmaWarp<G> + (kShares<G> ? 4 : 2)) * 32;

template <class G>
struct Smem {
    static constexpr int Q = 0;                                  // [NT][QPANELS][128 rows][128 B]
    static constexpr int RING = G::NT * G::QPANELS * 128 * 128;  // K and V
    static constexpr int BAR = RING + G::RING;                   // barriers
    // two sets, one for a unit and one for the next
    static constexpr int NBARS = kBarRing + G::BARS;
    static constexpr int BYTES = BAR + 2 * NBARS * 8 + 1024;     // + alignment of the base
};

// ---------------------------------------------------------------------------
// Slices of the key tiles
// ---------------------------------------------------------------------------

// Blocks of one (sequence, row tile, head) unit or one run of its keys leave SMs idle at the
// end.  So the keys of all units of a call are counted in a row and cut into equal slices,
// one to each SM (MLA: one to a pair of SMs, the two halves of the value columns, so that
// they read the same rows at the same time).  A block works off its slice unit by unit; a
// unit that a cut goes through is joined from parts.  Places are counted in keys times the
// group: a row tile of a causal sequence is kRows * NT places longer than the one before,
// which holds for every group.  A unit takes UNIT_COST tiles besides (its queries, first
// loads and results), unless slices are short.
// 32 ragged MLA sequences: 126 us a call, 139 with runs of equal length in two rounds of
// blocks (123 now, with the next unit found and loaded meanwhile).
constexpr int kMinRun = 4;      // fewest tiles of a slice
// With so many units to an SM blocks of one unit each even out by themselves (two prompts of
// 6000 tokens under a window, 2900 units: 520 us, 532 in slices of whole units, 541 cut)
constexpr int kManyUnits = 16;
// Most sequences: a block walks over them.  Beyond that no unit is cut, and a long context
// among many short ones is one block's work: 160 MLA sequences of 1000 tokens and one of
// them of 65536 take 117 us, 161 take 1144.
constexpr int kSliceSeqs = 160;

// What one warp knows of the slices.
template <class G>
struct Slices {
    static constexpr int64_t COUNT = G::MLA ? kSms / 2 : kSms;
    static constexpr int ROWS = kRows * G::NT;
    int64_t size, total; // places of a slice, of the call
    int64_t tile, cost;  // of a key tile, of a unit besides its tiles
    // of the unit that was asked for
    int seq, q0, n, len, row_tile, head, tiles;
    int64_t start, next; // places of its first tile and of the next unit
    bool bad;      // some sequence does not fit what the call stated

    // Finds the unit of place `pos`; a negative one is the start of slice -1 - pos.  False
    // past the last.
    __device__ __forceinline__ bool find(const AttnParams &p, int lane, int64_t &pos)
    {
        const int heads = G::MLA ? 1 : p.kv_heads;
        tile = (int64_t)G::KT * p.group;
        const int64_t grow = p.causal && p.window == 0 ? ROWS : 0;
        // sequence s: queries and keys, row tiles, places of the first one's unit
        struct Seq {
            int from, n, len, many;
            int64_t first;
            bool fits;
        };
        auto look = [&](int s) {
            Seq x{0, 0, 0, 0, 0, true};
            if (s >= p.num_seqs)
                return x;
            x.from = __ldg(p.q_off + s);
            const int to = __ldg(p.q_off + s + 1);
            x.len = __ldg(p.kv_len + s);
            x.fits = queries_fit(p, x.from, to, x.n) && (x.n == 0 || keys_fit(p, x.len));
            if (!x.fits || x.n == 0)
                return x;
            x.many = p.by_rows.quotient(x.n * p.group + ROWS - 1);
            if (grow) {
                x.first = (int64_t)max(0, x.len - x.n) * p.group + ROWS + p.group - 1;
            } else if (p.window == 0) {
                x.first = max(1, x.len) * (int64_t)p.group;
            } else { // at most
                const int span = p.window + min(x.n, p.by_group.quotient(ROWS - 1) + 2) - 1;
                const int most = min((x.len + G::KT - 1) / G::KT,
                                     (min(p.sinks, x.len) + G::KT - 1) / G::KT +
                                         (span + G::KT - 2) / G::KT + 1);
                x.first = max(1, most) * tile;
            }
            return x;
        };
        auto places = [&](const Seq &x) {
            return heads * (x.many * x.first + grow * (((int64_t)x.many * (x.many - 1)) >> 1));
        };
        bool wrong = false;
        int64_t units = 0;
        total = 0;
#pragma unroll 1
        for (int s = lane; s < p.num_seqs; s += 32) {
            const Seq x = look(s);
            wrong |= !x.fits;
            units += (int64_t)x.many * heads;
            total += places(x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            units += __shfl_xor_sync(0xFFFFFFFFu, units, d);
            total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
        }
        bad = __any_sync(0xFFFFFFFFu, wrong);
        cost = total >= COUNT * 2 * kMinRun * tile ? G::UNIT_COST * tile : 0;
        total += units * cost;
        size = max(kMinRun * tile, (total + COUNT - 1) / COUNT);
        if (pos < 0)
            pos = (-1 - pos) * size;
        bool found = false;
        int64_t before = 0, base = 0, unit = 0;
        int count = 0;
#pragma unroll 1
        for (int s = 0; s < p.num_seqs && !found; s += 32) {
            Seq x = look(s + lane);
            x.first += cost;
            const int64_t all = places(x);
            int64_t sum = all;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d)
                    sum += o;
            }
            const int64_t at = before + sum - all;
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, pos >= at && pos < at + all);
            if (who) {
                const int l = __ffs((int)who) - 1;
                seq = s + l;
                q0 = __shfl_sync(0xFFFFFFFFu, x.from, l);
                n = __shfl_sync(0xFFFFFFFFu, x.n, l);
                len = __shfl_sync(0xFFFFFFFFu, x.len, l);
                count = __shfl_sync(0xFFFFFFFFu, x.many, l);
                unit = __shfl_sync(0xFFFFFFFFu, x.first, l);
                base = __shfl_sync(0xFFFFFFFFu, at, l);
                found = true;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (!found)
            return false;
        // the row tile: the last whose units start at or before pos
        auto start_of = [&](int t) {
            return base + heads * (t * unit + grow * (((int64_t)t * (t - 1)) >> 1));
        };
        int lo = 0, hi = count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (start_of(mid) <= pos)
                lo = mid;
            else
                hi = mid;
        }
        row_tile = lo;
        const int64_t places_of_unit = unit + lo * grow;
        head = 0;
        while (head + 1 < heads && start_of(lo) + (head + 1) * places_of_unit <= pos)
            ++head;
        start = start_of(lo) + head * places_of_unit + cost;
        next = start - cost + places_of_unit;
        tiles = (int)((places_of_unit - cost + tile - 1) / tile);
        return true;
    }

    // slice of the unit's tile v
    __device__ __forceinline__ int slice_of(int v) const { return (int)((start + v * tile) / size); }
};

// The next piece of this block's slice, from `pos` on (-1 - slice: from its start); false
// past its end.  w.split is the place of its part: a slice begins and ends inside a unit
// at most once each.
template <class G>
__device__ __forceinline__ bool find_slice(const AttnParams &p, int lane, int64_t &pos, Work &w,
                                           bool &bad)
{
    const int slice = (int)blockIdx.x / G::HALVES, half = (int)blockIdx.x % G::HALVES;
    Slices<G> s;
    while (s.find(p, lane, pos)) {
        bad = s.bad;
        const int64_t end = min(s.total, (slice + 1) * s.size);
        if (pos >= end)
            return false;
        // its tiles whose places are this slice's
        const int v0 = pos <= s.start ? 0 : (int)((pos - s.start + s.tile - 1) / s.tile);
        const int v1 = end <= s.start ? 0
                                      : (int)min((int64_t)s.tiles, (end - s.start + s.tile - 1) / s.tile);
        pos = s.next; // a unit that goes on goes on in the next slice
        if (v0 >= v1)
            continue;
        w.seq = s.seq;
        w.q0 = s.q0;
        w.n = s.n;
        w.len = s.len;
        w.row0 = s.row_tile * Slices<G>::ROWS;
        w.head = G::MLA ? half : s.head;
        w.splits = v0 > 0 || v1 < s.tiles ? 2 : 1; // more than one
        w.split = (2 * slice + (v0 == 0)) * G::HALVES + half;
        const int real = key_tiles<G::KT, G::NT>(p, w);
        w.beg = min(real, v0);
        w.end = min(real, v1);
        return true;
    }
    bad = s.bad;
    return false;
}

// Joins the units that the ends of slices cut.  Where they lie is found before the wait for
// the kernel that writes their parts.  Bound by latency: 11 to 13 us by itself for 40 MB of
// parts, 29 to 50 when every row of the call looked for its parts.  JOIN_BLOCKS blocks to a slice: they join the unit whose first
// cut is the slice's start, a warp for a row.
template <class G>
__global__ void __launch_bounds__(256) slice_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int ROWS = kRows * G::NT;
    __shared__ int s_splits, s_rows, s_row0, s_head, s_q0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slice = (int)blockIdx.x / G::JOIN_BLOCKS + 1; // the first start is no cut
    if (warp == 0) {
        Slices<G> s;
        int64_t pos = -1 - slice;
        int splits = 0;
        if (s.find(p, lane, pos)) {
            if (s.slice_of(0) == slice - 1)
                splits = s.slice_of(s.tiles - 1) - slice + 2;
            s_row0 = s.row_tile * ROWS;
            s_rows = min(ROWS, s.n * p.group - s.row_tile * ROWS);
            s_head = s.head;
            s_q0 = s.q0;
        }
        s_splits = splits;
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (s_splits <= 1)
        return;
    const int rows = s_rows;
    for (int r = (int)blockIdx.x % G::JOIN_BLOCKS * 8 + warp; r < rows; r += G::JOIN_BLOCKS * 8) {
        const int row = s_row0 + r, i = p.by_group.quotient(row);
        const int64_t tok = (int64_t)s_q0 + i;
        const int h = s_head * p.group + row - i * p.group;
        // the first part lies in the second place of its slice, the others in the first ones
        auto at = [&](int k) {
            return (int64_t)(2 * (slice - 1 + k) + (k == 0)) * G::HALVES * ROWS + r;
        };
        join_row<G::DV / 128>(
            s_splits, lane, p.out + tok * p.o_ts + h * p.o_hs,
            p.lse ? p.lse + tok * p.heads + h : nullptr,
            [&](int k, int v) {
                constexpr int PER = G::OC / 128; // the halves of MLA columns are parts of their own
                return reinterpret_cast<const float4 *>(
                    p.part + (at(k) + v / PER * ROWS) * G::OC + v % PER * 128);
            },
            [&](int k) { return p.part_lse + at(k); });
    }
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
                                              uint32_t bars, int warp, int lane, bool careful,
                                              volatile int *abort, bool &bad)
{
    constexpr int AHEAD = 3;
    const int base = warp * 8, c = lane & 7, sub = lane >> 3;
    const int32_t *const table = p.block_tables + (int64_t)w.seq * p.max_blocks;
    auto whole = [&](int v) { // as in load_heads
        return p.box_rows > 0 && (!careful || tile_whole<G::KT>(w, real_tile(w, v)));
    };
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
                auto seen = [&](int u) { // this lane's box
                    return mine && u < last &&
                           keys_seen(w, real_tile(w, u) * G::KT + lane * p.box_rows, p.box_rows);
                };
                auto ask = [&](int u) {
                    const int kt = real_tile(w, u);
                    return seen(u) ? __ldg(table + (in == 1 ? kt * per + lane : kt / in)) : 0;
                };
                int32_t blk = ask(v + skip);
                for (int u = v; ok && u < last; ++u) {
                    const int kt = real_tile(w, u + skip);
                    const bool fits = (uint32_t)blk < (uint32_t)p.num_blocks;
                    bad |= !fits;
                    const int y = fits && seen(u + skip) ? (in == 1 ? 0 : (kt % in) * G::KT) + blk * p.block
                                       : (int)(p.num_blocks * p.block); // past the pool: zeros
                    blk = ask(u + 1 + skip);
                    const int ord = u - w.beg, stage = ord & 1, phase = ((ord >> 1) & 1) ^ 1;
                    const uint32_t full = bars + (part * 2 + stage) * 8;
                    if (before) { // keeps step with the others, who do not wait for it
                        int late = 0;
                        bar_wait(full + G::BARS / 2 * 8, phase, &late, kPrefetchWait);
                        if (*abort)
                            break;
                        if (mine && u + skip < last) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                prefetch_box(&p.copy_map, w.head * 256 + i * 64, y);
                            if (w.head == 0)
                                prefetch_box(&p.rot_map, 0, y);
                        }
                        continue;
                    }
                    ok = bar_wait(full + G::BARS / 2 * 8, phase, abort, p.wait_limit_ns);
                    if (!ok)
                        break;
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
            if (more) // the last one is kBarDone's
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
//
// A weight of 0 does not keep an infinite or NaN value of a key that the row does not see
// out of the products.  `finite`: O shows none of that; if it does, the unit is done again,
// `careful`: keys that no row sees are zeros, and such values of others are taken out of V
// before they are used and given back at the end to the rows that do see them.
template <class G>
__device__ __forceinline__ bool run_softmax(const AttnParams &p, const Work &w, const TileMask &m,
                                            int t, uint32_t tmem, uint32_t ring, uint32_t bars,
                                            int warp, int half, int lane, int warps,
                                            bool careful, volatile int *abort, volatile int *dirty,
                                            RowPairs<G> &pairs, RowState &st, bool &finite)
{
    constexpr int KT = G::KT, HK = KT / 2, HO = G::OC / 2; // keys, columns of O of a thread
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int pair = t * 4 + warp;
    const int r = warp * 32 + lane;
    const int row = w.row0 + t * kRows + r;
    const int tok = p.by_group.quotient(row);
    const bool valid = r < m.rows;
    const int pos = w.len - w.n + tok;
    // keys this row sees: [lo, hi) and [0, sk)
    const int hi = !valid ? 0 : p.causal ? min(w.len, pos + 1) : w.len;
    const int lo = p.window ? max(0, pos - p.window + 1) : 0;
    const int sk = p.window ? min(p.sinks, hi) : 0;
    const bool one_token = G::NT == 1 && m.pos0 == m.pos1;
    const float c = p.scale * 1.4426950408889634f;
    const uint32_t o_col = tmem + G::O_COL(t) + half * HO + lanes;
    bool partial = false;
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
                return false;
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
        partial |= !full && (!one_token || p.box_rows > 0);
        if (careful && !full && !one_token) {
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
        return false;
    const float other = pair_swap<G>(pairs, pair, half, t * kRows + r, st.sum);
    st.sum = half == 0 ? st.sum + other : other + st.sum; // the same in both
    finite = true;
    if (partial && !careful) {
        float x = 0.0f; // NaN once a value is not finite
#pragma unroll 1
        for (int i = 0; i < HO; i += 32) {
            uint32_t o[32];
            tmem_ld32(o_col + i, o);
            tmem_ld_wait();
            tmem_pin32(o);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x = fmaf(__uint_as_float(o[j]), 0.0f, x);
        }
        finite = !valid || x == 0.0f;
    }
    return true;
}

// The results of run_softmax's rows, or their parts.
template <class G>
__device__ __forceinline__ void store_rows(const AttnParams &p, const Work &w, const TileMask &m,
                                           int t, uint32_t tmem, int warp, int half, int lane,
                                           bool dirty, const RowState &st)
{
    constexpr int KT = G::KT, HO = G::OC / 2;
    const int r = warp * 32 + lane;
    const int row = w.row0 + t * kRows + r;
    const int tok = p.by_group.quotient(row), g = row - tok * p.group;
    const bool valid = r < m.rows;
    const int pos = w.len - w.n + tok;
    const int hi = !valid ? 0 : p.causal ? min(w.len, pos + 1) : w.len;
    const int lo = p.window ? max(0, pos - p.window + 1) : 0;
    const int sk = p.window ? min(p.sinks, hi) : 0;
    const uint32_t o_col = tmem + G::O_COL(t) + half * HO + ((uint32_t)(warp * 32) << 16);
    const float sum = st.sum, inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int h = G::MLA ? g : w.head * p.group + g;
    const int64_t at = (w.q0 + tok) * p.heads + h;
    const int col0 = (G::MLA ? w.head * 256 : 0) + half * HO;
    const bool parts = w.splits > 1;
    if (valid && half == 0 && (!G::MLA || w.head == 0)) {
        const float lse = sum == 0.0f ? -INFINITY : st.top * p.scale + logf(sum);
        if (parts)
            p.part_lse[(int64_t)w.split * (kRows * G::NT) + t * kRows + r] = lse;
        else if (p.lse)
            p.lse[at] = lse;
    }
    char *out = p.out + (w.q0 + tok) * p.o_ts + h * p.o_hs + col0 * 2;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0; // a row's sectors are whole
    float *part =
        p.part + ((int64_t)w.split * (kRows * G::NT) + t * kRows + r) * G::OC + half * HO;
#pragma unroll 1
    for (int i = 0; i < HO; i += 32) {
        uint32_t o[32];
        tmem_ld32(o_col + i, o);
        tmem_ld_wait();
        tmem_pin32(o);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            o[j] = sum == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[j]) * inv);
        if (dirty) {
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

// All commits of a unit of `tiles` key tiles have arrived: its barriers can be made anew.
// A parity shows the last phase of a barrier when the one before is known to be over.  It is
// for the stages (their copies waited for it) and for O: what came before the scores of the
// last tile, whose weights were waited for, leaves one commit of O, that of the tile before
// the last.
template <class G>
__device__ __forceinline__ void drain(uint32_t bars, int tiles, volatile int *abort, int64_t limit)
{
    auto last = [&](uint32_t bar, int count) {
        if (count > 0)
            bar_wait(bar, (count - 1) & 1, abort, limit);
    };
    const uint32_t empty = bars + (kBarRing + G::BARS / 2) * 8;
    if (G::NT == 1)
        last(bars + kBarO * 8, tiles - 1);
    if constexpr (G::MLA) {
        for (int i = 0; i < G::BARS / 2; ++i)
            last(empty + i * 8, (tiles + 1 - (i & 1)) / 2);
    } else { // two row tiles do not give the last V back
        const int items = 2 * tiles - (G::NT == 2 ? 1 : 0);
        for (int i = 0; i < G::STAGES; ++i)
            last(empty + i * 8, (items - i + G::STAGES - 1) / G::STAGES);
    }
}

// A block works off its slice of the call's key tiles, or its one unit.  The roles meet once
// a unit, when its MMAs are done; the rows' results are stored after that, while the next
// unit's rows and queries are on their way.  One warp finds the next unit and sets its
// barriers up meanwhile (two sets take turns), which takes 6500 clocks.  Chunks of several
// units to a block: 181 us when all that was done in turn, 177 so (8 ragged, 28 heads over
// 4), MLA 222 and 214, 4096 tokens over 16384 729 and 690.
template <class G>
__global__ void __launch_bounds__(kAttnThreads<G>, 1) attention_kernel(
    const __grid_constant__ AttnParams p)
{
    using S = Smem<G>;
    extern __shared__ unsigned char raw_smem[];
    __shared__ Work s_work[3]; // of units k % 3: one to store, one to do, one to come
    __shared__ uint32_t s_tmem, s_status;
    __shared__ int s_go[2];
    __shared__ volatile int s_abort, s_dirty[2];
    __shared__ RowPairs<G> s_pairs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const uint32_t q_smem = smem + S::Q, ring = smem + S::RING;
    auto bars_of = [&](int k) { return smem + S::BAR + (k & 1) * S::NBARS * 8; };
    // All threads; true where a wait of some ran out in the unit before.
    auto meet = [&](bool gave_up) {
        mma_fence_before();
        const bool any = __syncthreads_or(gave_up) != 0;
        mma_fence_after();
        return any;
    };

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < G::SOFT_WARPS) {
        if constexpr (kShares<G>)
            reg_inc<kSoftRegs>();
        meet(false);
        const int t = warp >> 3, half = (warp >> 2) & 1, wl = warp & 3;
        const uint32_t tmem = s_tmem;
        // Queries of a unit on their way; its MMAs may start when every thread has signalled.
        // A warp without rows there does so when the results that the MMAs write over are out.
        auto signal = [&](int k) {
            mma_fence_before();
            bar_signal_copies(bars_of(k) + kBarQ * 8);
        };
        auto ask = [&](int k) {
            const Work w = s_work[k % 3];
            const int rows = tile_mask(p, w.n, w.len, w.row0 + t * kRows).rows;
            load_queries<G>(p, w, q_smem, t, tid & 255);
            if constexpr (G::MLA)
                queries_to_tmem<G>(p, w, tmem, wl, lane, rows, half * 2);
            if (wl * 32 < rows)
                signal(k);
            return wl * 32 < rows;
        };
        bool mine = false;
        if (s_go[0]) {
            mine = ask(0);
            if (!mine)
                signal(0);
        }
        for (int k = 0; s_go[k & 1]; ++k) {
            RowState st;
            bool store = false, stop, dirty;
            for (bool careful = false;; careful = true) {
                bool finite = true;
                st = RowState{};
                if (mine) {
                    const Work w = s_work[k % 3];
                    const TileMask mask = tile_mask(p, w.n, w.len, w.row0 + t * kRows);
                    store = run_softmax<G>(p, w, mask, t, tmem, ring, bars_of(k), wl, half, lane,
                                           (mask.rows + 31) / 32, careful, &s_abort, &s_dirty[k & 1],
                                           s_pairs, st, finite);
                }
                __syncwarp();
                dirty = s_dirty[k & 1] != 0;
                stop = meet(s_abort != 0);
                if (!meet(!finite) || stop)
                    break;
                meet(false);
                mma_fence_before();
                bar_signal(bars_of(k) + kBarQ * 8); // the queries are there
            }
            const bool more = !stop && s_go[(k + 1) & 1];
            if (more)
                mine = ask(k + 1);
            if (store) {
                const Work w = s_work[k % 3];
                store_rows<G>(p, w, tile_mask(p, w.n, w.len, w.row0 + t * kRows), t, tmem, wl, half,
                              lane, dirty, st);
            }
            if (more && !mine)
                signal(k + 1);
            if (stop)
                break;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < kMmaWarp<G>) {
        if constexpr (kShares<G>)
            reg_dec<kLoadRegs>();
        meet(false);
        const int lw = warp - G::SOFT_WARPS;
        for (int k = 0; s_go[k & 1]; ++k) {
            const Work w = s_work[k % 3];
            const uint32_t bars = bars_of(k) + kBarRing * 8;
            bool stop;
            for (bool careful = false;; careful = true) {
                bool bad = false;
                if constexpr (G::MLA && G::QUANT)
                    load_mla_e4m3<G>(p, w, ring, bars, lw, lane, &s_abort, bad);
                else if constexpr (G::MLA)
                    load_mla_bf16<G>(p, w, ring, bars, lw, lane, careful, &s_abort, bad);
                else if constexpr (G::QUANT)
                    load_heads_e4m3<G>(p, w, ring, bars, lw, lane, &s_abort, bad);
                else
                    load_heads<G>(p, w, ring, bars, lw, lane, careful, &s_abort, bad);
                if (bad)
                    s_status = kStatusOutOfRange;
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                stop = meet(s_abort != 0);
                if (!meet(false) || stop)
                    break;
                meet(false);
            }
            if (stop)
                break;
        }
    } else {
        if constexpr (kShares<G>)
            reg_dec<kMmaRegs>();
        const bool finder = warp == kMmaWarp<G> + 1;
        int64_t pos = -1 - (int64_t)(blockIdx.x / G::HALVES);
        // the finder: barriers of unit k; `old`: they have been used
        auto set_up = [&](int k, const Work &w, bool old) {
            for (int i = lane; i < S::NBARS; i += 32) {
                int count = 1; // commits
                if (i == kBarQ)
                    count = G::SOFT_WARPS * 32;
                else if (i == kBarP || i == kBarP + 1) // the warps that have rows signal the weights
                    count = max(1, (tile_mask(p, w.n, w.len,
                                              w.row0 + (G::NT == 2 ? i - kBarP : 0) * kRows).rows +
                                    31) / 32) * 64;
                else if (i >= kBarRing && i < kBarRing + G::BARS / 2)
                    count = G::LOAD_WARPS * 32;
                if (old)
                    bar_drop(bars_of(k) + i * 8);
                bar_init(bars_of(k) + i * 8, count);
            }
            bar_init_fence();
            __syncwarp();
        };
        auto next = [&](int k) { // the finder: work of unit k
            Work w{};
            bool bad = false, go = false;
            if (p.slices) {
                go = find_slice<G>(p, lane, pos, w, bad);
            } else if (k == 0) {
                // block -> (row tile, key head or half); heads of one row tile and its halves
                // are neighbours, so their rows meet in L2
                const int heads = G::MLA ? 2 : p.kv_heads, tile = p.by_heads.quotient(blockIdx.x);
                int at = 0;
                go = find_tile<kRows * G::NT>(p, tile, lane, w, at, bad);
                w.head = (int)blockIdx.x - tile * heads;
                w.row0 = at * kRows * G::NT;
                if (go)
                    w.end = key_tiles<G::KT, G::NT>(p, w);
                w.splits = 1;
            }
            if (lane == 0) {
                s_work[k % 3] = w;
                s_go[k & 1] = go;
                s_dirty[k & 1] = 0;
                if (bad)
                    s_status = kStatusOutOfRange;
            }
            set_up(k, w, k >= 2);
        };
        if (finder) {
            if (lane == 0) {
                s_status = kStatusOk;
                s_abort = 0;
            }
            __syncwarp();
            next(0);
        } else if (warp == kMmaWarp<G>) {
            tmem_alloc(smem_u32(&s_tmem), 512);
        }
        meet(false);
        for (int k = 0; s_go[k & 1]; ++k) {
            bool stop;
            for (bool again = false;; again = true) {
                if (finder && !again) {
                    next(k + 1);
                } else if (warp == kMmaWarp<G>) {
                    const Work w = s_work[k % 3];
                    const uint32_t lead = elect_lane(), tmem = s_tmem, bars = bars_of(k);
                    bool ok = blockIdx.x != p.skip_block &&
                              bar_wait(bars + kBarQ * 8, 0, &s_abort, p.wait_limit_ns);
                    if (ok) {
                        async_fence(); // the queries came by copies of other threads
                        mma_fence_after();
                        if constexpr (G::NT == 2)
                            ok = run_mma_two<G>(p, w, tmem, q_smem, ring, bars, lead, &s_abort);
                        else
                            ok = run_mma_one<G>(p, w, tmem, q_smem, ring, bars, lead, &s_abort);
                    }
                    if (ok) {
                        drain<G>(bars, w.end - w.beg, &s_abort, p.wait_limit_ns);
                    } else { // let what was issued finish before tensor memory goes
                        int none = 0;
                        bar_signal_mma(bars + (kBarO + 1) * 8, lead);
                        bar_wait(bars + (kBarO + 1) * 8, 0, &none, 1000000000ll);
                    }
                    __syncwarp();
                }
                stop = meet(s_abort != 0);
                if (!meet(false) || stop)
                    break;
                if (finder)
                    set_up(k, s_work[k % 3], true);
                meet(false);
            }
            if (stop)
                break;
        }
    }
    meet(false); // all results are out
    if (warp == kMmaWarp<G>)
        tmem_free(s_tmem, 512);
    if (tid == 0)
        write_block_status(p.header, s_abort ? kStatusTimeout : s_status, blockIdx.x, p.status_words);
}

template <class G>
cudaError_t launch(AttnParams &p, int64_t blocks, cudaStream_t stream)
{
    constexpr int bytes = Smem<G>::BYTES;
    static_assert(bytes + sizeof(RowPairs<G>) + 3 * sizeof(Work) + 64 <= 227 * 1024, "shared memory");
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
    if (!p.slices)
        return cudaSuccess;
    constexpr int cuts = (int)Slices<G>::COUNT - 1;
    return launch_join(slice_join_kernel<G>, p, cuts * G::JOIN_BLOCKS, stream);
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
    // (and no sequence has more than its longest chunk would)
    const int64_t most = (std::min<int64_t>(a.total_q, a.max_q_len) * a.group + rows - 1) / rows;
    const int64_t tiles = few || !tiles_share
                              ? a.num_seqs
                              : std::min(a.total_q * a.group / rows + a.num_seqs, a.num_seqs * most);
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
    pl.max_splits = 1;
    pl.blocks = units;
    if (!few) {
        // Slices, or a block to a unit: what each takes, in key tiles, if every unit were as
        // long as the longest may be.  A unit starts and ends in the time of `around` tiles,
        // a join takes `join`.  1024 tokens over themselves, 32 heads over 8: 23 us with a
        // block to a unit, 80 in slices; 16 tokens over 1024: 14 and 19, over 2048 both 20,
        // over 8192: 28 in slices, some 65 otherwise.  A ragged batch has more to gain than
        // that shows.
        const int64_t around = mla ? 6 : pl.row_tiles == 2 ? 4 : 9;
        const int64_t join = mla ? 7 : pl.row_tiles == 2 ? 5 : 12;
        const int64_t u = mla ? units / 2 : units, at_once = mla ? kSms / 2 : kSms;
        const int64_t whole = (u + at_once - 1) / at_once * (nv + around);
        const int64_t cut = std::max<int64_t>(kMinRun, u * nv / at_once) + around +
                            u * around / at_once + join;
        pl.slices = a.num_seqs <= kSliceSeqs && units < kManyUnits * kSms &&
                    (a.num_seqs > 1 ? cut * 10 <= whole * 11 : cut <= whole);
        if (pl.slices)
            pl.blocks = kSms;
        return pl;
    }
    // pieces of the key axis: enough blocks for a few on every SM, none shorter
    // than four tiles (a block's start and end cost about as much as two)
    const int64_t slots = 2 * kSms;
    const int64_t want = std::max<int64_t>(4, (units * nv + 4 * slots - 1) / (4 * slots));
    pl.split_tiles = (int32_t)std::min(nv, want);
    // one round of blocks and short rows: up to 8 runs in a cluster
    const int64_t run = (nv + 7) / 8;
    pl.cluster = nv > 1 && run <= 4 && units * ((nv + run - 1) / run) <= slots;
    if (pl.cluster)
        pl.split_tiles = (int32_t)run;
    pl.max_splits = (int32_t)((nv + pl.split_tiles - 1) / pl.split_tiles);
    pl.blocks = units * pl.max_splits;
    return pl;
}

cudaError_t launch_attention(AttnParams &p, RowKind kind, const AttnPlan &pl, cudaStream_t stream)
{
    const bool quant = p.cs != nullptr;
    p.cluster = pl.cluster ? 1 : 0;
    p.slices = pl.slices ? 1 : 0;
    p.by_group = Divisor((uint32_t)p.group);
    p.by_rows = Divisor((uint32_t)(kRows * std::max(1, pl.row_tiles)));
    p.by_block = Divisor((uint32_t)p.block);
    p.by_heads = Divisor(kind == RowKind::Mla ? 2u : (uint32_t)p.kv_heads);
    p.by_splits = Divisor((uint32_t)p.max_splits);
    p.by_run = Divisor((uint32_t)std::max(1, p.split_tiles));
    if (kind == RowKind::Mla)
        return quant ? launch<MlaGeo<true>>(p, pl.blocks, stream)
                     : launch<MlaGeo<false>>(p, pl.blocks, stream);
    if (pl.row_tiles == 0)
        return launch_attention_few(p, pl.blocks, stream);
    if (pl.row_tiles == 2)
        return launch<HeadGeo<false, 2>>(p, pl.blocks, stream);
    return quant ? launch<HeadGeo<true, 1>>(p, pl.blocks, stream)
                 : launch<HeadGeo<false, 1>>(p, pl.blocks, stream);
}

} // namespace kvr
