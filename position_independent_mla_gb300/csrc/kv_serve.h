// kv_serve.h -- parameters and launchers of the serving operators: quantised
// cache rows (kv_quant.cu) and attention over the paged cache (kv_attention.cu).
#pragma once

#include <cuda.h>

#include "kv_launch.h"

namespace kvr {

constexpr int kGroup = 128; // values that share one scale of a quantised row

// Status of a call without a clearing launch: every block of the call's main
// kernel writes its own word after the workspace header (0 or an error code)
// and block 0 writes the header, so nothing needs to be zero beforehand;
// kv_get_device_status scans the words.  The count is followed by its complement.
constexpr int kHeaderCountWord = 8; // header word: number of block words (0: word 0 holds all)

__device__ __forceinline__ void write_block_status(uint32_t *header, uint32_t code,
                                                   uint32_t block, uint32_t blocks)
{
    header[kHeaderBytes / 4 + block] = code;
    if (block == 0) {
        header[0] = kStatusOk;
        header[kHeaderCountWord] = blocks;
        header[kHeaderCountWord + 1] = ~blocks;
    }
}

// A quantised pool as the kernels see it: byte addresses and byte strides,
// scales in floats.
struct QuantView {
    char *copy;
    int64_t copy_ls, copy_ss;
    float *cs;
    int64_t cs_ls, cs_ss;
    char *rot;
    int64_t rot_ls, rot_ss;
    float *rs; // nullptr: rot is bf16
    int64_t rs_ls, rs_ss;
    int64_t num_slots;
};

struct QuantParams {
    PoolView rows;           // the bf16 side
    QuantView pool;          // at its first layer of the call
    const int32_t *row_slot; // bf16 side: slot of row i (nullptr: i)
    const int32_t *pool_slot;
    int64_t num_rows;
    int32_t layers;
    uint32_t *header;
};

cudaError_t launch_quantize(const QuantParams &p, RowKind kind, cudaStream_t stream);
cudaError_t launch_dequantize(const QuantParams &p, RowKind kind, cudaStream_t stream);
constexpr int kQuantMaxBlocks = 152 * 8; // persistent grid of both

// Rows of a quantised pool that a batch attends to, widened once into bf16 rows of
// the workspace for row tiles that would each convert them again.
constexpr int kExpandBlock = 64; // block size of the rows it writes

struct ExpandParams {
    PoolView rows;  // written: [num_seqs][pad] rows
    QuantView pool; // at the layer of the call
    int64_t pad;    // rows of a sequence: a multiple of kExpandBlock
    int64_t num_blocks;
    int32_t block, num_seqs, max_kv_len, max_blocks, window, sinks;
    const int32_t *q_off, *kv_len, *block_tables;
    int32_t *table;   // written: [num_seqs][pad / kExpandBlock]
    uint32_t *status; // a word per block
    int32_t blocks;
};

int expand_blocks(int64_t rows); // blocks of a launch over so many rows
cudaError_t launch_expand(const ExpandParams &p, RowKind kind, cudaStream_t stream);

// Quotients by a number that only the host knows, for 0 <= n < 2^31 (Granlund and
// Montgomery, Division by invariant integers using multiplication, 1994): with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n) >> l.
struct Divisor {
    uint32_t mul = 1, shift = 0;

    Divisor() = default;
    explicit Divisor(uint32_t d)
    {
        while ((uint64_t(1) << shift) < d)
            ++shift;
        mul = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d)) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int quotient(int n) const
    {
        return (int)((__umulhi(mul, (uint32_t)n) + (uint32_t)n) >> shift);
    }
#endif
};

// Rows and keys of a sequence are 32-bit numbers in the kernels, with room for a tile past
// the end.
constexpr int kRows = 128; // rows of a tile: the M of an MMA
constexpr int kSms = 152;
constexpr int64_t kMaxRows = 0x40000000, kMaxKeys = 0x7FFFFF00;

struct AttnParams {
    // one layer of the pool: bf16 rows, or e4m3 rows with scales (cs != nullptr)
    const char *copy, *rot;
    int64_t copy_ss, rot_ss; // bytes
    const float *cs, *rs;    // scales (floats per slot: cs_ss, rs_ss)
    int64_t cs_ss, rs_ss;
    int64_t num_blocks;
    int32_t block;
    // queries and results, byte strides
    const char *q;
    int64_t q_ts, q_hs;
    char *out;
    int64_t o_ts, o_hs;
    float *lse;
    int64_t total_q;
    int32_t heads, group, kv_heads; // query heads; of them to a key head; key heads
    int32_t num_seqs, max_q_len, max_kv_len, max_blocks;
    int64_t max_keys; // that a block-table row of the caller holds
    const int32_t *q_off, *kv_len, *block_tables;
    int32_t causal, window, sinks;
    // drafted trees (causal and window are 0): bit j of a query's words: it sees new token j
    const uint32_t *tree; // nullptr: none
    int64_t tree_stride;  // words
    int32_t tree_words;
    float scale;
    // split of the key axis, and the parts that are joined afterwards: of few rows
    // [max_splits][total_q][heads][value width], lse [..][heads]
    int32_t split_tiles, max_splits, cluster;
    float *part, *part_lse;
    // of others, where blocks take equal slices of all keys of the call: [2 * kSms][rows of
    // a block][columns of a block]
    int32_t slices;
    int32_t side; // trees: key heads whose blocks read the same keys side by side
    int64_t wait_limit_ns;
    int64_t skip_block; // test hook: this block issues no MMA (-1: none)
    uint32_t *header;
    uint32_t status_words; // of the call: this kernel's blocks, and those of an expansion
    // filled in by launch_attention: quotients by group, rows of a row tile, block, key heads (MLA: halves),
    // max_splits and split_tiles
    Divisor by_group, by_rows, by_block, by_heads, by_splits, by_run;
    // bf16 pools, likewise: rows of a box (0: no boxes)
    int32_t box_rows;
    CUtensorMap copy_map, rot_map;
};

// Sizes of a call that the host knows, and the launch they lead to.
struct AttnShape {
    bool quant, tree;
    int64_t total_q;
    int32_t num_seqs, max_q_len, max_kv_len, window, sinks;
    int32_t group, kv_heads;
};

struct AttnPlan {
    bool expand;         // e4m3 rows are widened first
    int32_t row_tiles;   // 128-row tiles of a block; 0: the kernel for few rows
    int32_t split_tiles; // few rows: key tiles of a block
    int32_t max_splits;
    bool cluster;        // the splits of a row are a cluster that joins them itself
    bool slices;         // the split is made on the device (Slices)
    int32_t side;        // its blocks that take the same keys, for heads of their own
    int64_t blocks;

    bool joins() const { return slices || (max_splits > 1 && !cluster); }
};

// Rows that close up in place (kv_compact.cu).
struct CompactParams {
    PoolView pool; // bytes of either kind of pool
    float *cs, *rs; // scales of a quantised pool (cs == nullptr: bf16)
    int64_t cs_ls, cs_ss, rs_ls, rs_ss;
    const int32_t *block_tables;
    int32_t max_blocks, num_seqs;
    const int32_t *first; // nullptr: 0
    const int32_t *keep;  // [num_seqs][max_count], keep_stride apart
    int64_t keep_stride;
    const int32_t *count;
    int32_t max_count;
    int32_t layer_groups, group_layers; // a tile's layers are cut into this many units
    const float4 *turn_lo, *turn_hi;    // cos / sin tables (nullptr: rows are not turned)
    int32_t turn_bits, turn_half;
    uint32_t *status, *ticket, *flags; // flags: [tiles][num_seqs][layer_groups]
    int64_t wait_limit_ns;
    int64_t skip_publish; // test hook: this ticket does not publish its reads (-1: none)
};

struct TurnParams {
    double base;
    int32_t half, bits, lo_rows, hi_rows;
    float4 *table; // lo_rows of turn_lo, then hi_rows of turn_hi
};

// Rows of a tile; `one`: where every list fits one.
int compact_tile_rows(RowKind kind, bool quant, bool one);
cudaError_t launch_turn_table(const TurnParams &p, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams &p, RowKind kind, bool one, int64_t units,
                           cudaStream_t stream);

// Which tokens stay (kv_select.cu).
struct SelectParams {
    const float *weights; // [num_seqs][max_kv_len], weight_stride apart
    int64_t weight_stride;
    const int32_t *kv_len, *budget;
    int32_t num_seqs, max_kv_len, sinks, recent;
    int32_t *keep;        // [num_seqs][max_keep], keep_stride apart
    int64_t keep_stride;
    int32_t max_keep;
    int32_t *count;
    float *kept;          // nullptr: not wanted
    int64_t kept_stride;
    int32_t cluster;      // blocks of a sequence
    uint32_t *header;
};

int select_cluster(int32_t num_seqs, int32_t max_kv_len);
cudaError_t launch_select(const SelectParams &p, cudaStream_t stream);

// What each key receives of the queries' attention (kv_weights.cu, kv_weights_few.cu,
// kv_weights_many.cu).
struct WeightsParams {
    AttnParams a; // the batch, its pool and its queries; out and the split have no part
    const float *lse;
    float *weights;
    int64_t weight_stride;
    float keep;
    int32_t toks, rows, n; // of a row tile: tokens; rows; rows with those that pad it
    int32_t parts;         // that the row tiles and heads over some keys are divided into
    int64_t total_parts;   // many row tiles: of the call; a.part holds 256 sums of each
    int32_t stages;
    int32_t q_boxes;       // query rows come as boxes of q_map
    int32_t run, slices;   // few rows: key tiles of a block, or equal slices of all of them;
    int32_t row_pad;       // rows of a head, to a power of two
    Divisor by_toks;
    CUtensorMap q_map;
};

struct WeightsPlan {
    bool many;         // head rows under more than one row tile
    int32_t toks, rows, n, parts, stages;
    int64_t blocks, units;
    int32_t smem;
    size_t part_bytes; // of the workspace, for sums of parts
    // few rows, where the pool's rows come as boxes
    bool few, few_slices;
    int32_t few_parts, few_stages, run, row_pad, few_smem;
    int64_t few_blocks;

    int64_t most_blocks() const { return few && few_blocks > blocks ? few_blocks : blocks; }

    int launches() const { return many && parts > 1 ? 2 : 1; }
};

WeightsPlan plan_weights(RowKind kind, const AttnShape &a);
cudaError_t launch_weights(WeightsParams &p, RowKind kind, const WeightsPlan &pl,
                           cudaStream_t stream);

AttnPlan plan_attention(RowKind kind, const AttnShape &a);
cudaError_t launch_attention(AttnParams &p, RowKind kind, const AttnPlan &pl, cudaStream_t stream);

} // namespace kvr
