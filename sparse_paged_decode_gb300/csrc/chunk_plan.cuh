// chunk_plan.cuh -- the work plan of the tensor-core prefill attention, built
// on the device from the batch's lengths (the host reads nothing, so the call
// stays graph safe), and its layout inside the caller's workspace.
//
//   pair   up to 2 * tt consecutive query tokens of one sequence, tt = 128 / G:
//          two tiles of 128 query rows (row = token * G + head) that share
//          every K/V page a CTA loads
//   unit   (pair, kv head, piece): a contiguous piece of the pair's key
//          blocks, the work item of one CTA.  A pair in one piece writes its
//          rows at once; the pieces of a split pair leave fp32 partials
//          (running max, sum, unnormalised output) that a kernel behind the
//          attention kernel joins, in piece order
//
// Units are numbered sequence by sequence, the longest first, and within a
// sequence head by head: CTAs claim them in that order, so the units that are
// claimed last are short ones, and the pairs that run at one time read the
// same pages, so a page comes from HBM once per head and from L2 for the
// other pairs.
#pragma once

#include <stdint.h>

#include "serve.cuh"

namespace spd {

struct ChunkHeader {
    int32_t status;     // bit 0: a wait timed out (the place spd_workspace_status reads)
    int32_t next_unit;  // units claimed beyond the first one of each CTA
    int32_t n_pairs;
    int32_t n_units;    // of all heads
    int32_t head_parts; // partial slots of one head
    int32_t n_splits;   // pairs in more than one piece
    int32_t reserved[58];
};
static_assert(sizeof(ChunkHeader) == 256, "header is one 256-byte line");

// What a search over the pairs and the unit's place need first, in one load.
struct ChunkKey {
    int32_t unit0;   // first unit within a head, over all sequences
    int32_t seq0;    // unit0 of the sequence's first pair
    int32_t seq_units;  // units of the sequence within a head
    int32_t pieces;
};

struct ChunkPair {
    ChunkKey key;
    int32_t b;       // sequence
    int32_t i0;      // first token of the pair within its chunk
    int32_t nt;      // tokens
    int32_t tok0;    // first query token
    int32_t part0;   // first partial slot within a head (split pairs)
    int32_t row;     // page-table row of the sequence (any, where cap is 0)
    int32_t pre;     // cached keys
    int32_t cap;     // keys in all, at most what the table holds
};
static_assert(sizeof(ChunkPair) == 48, "pair record is 48 bytes");

// A pair in more than one piece, for the join.
struct ChunkSplit {
    int32_t tok0, nt, pieces, part0;
};

constexpr int kChunkMaxParts = 608;  // partial slots: four pieces per SM of a 152-SM device

// Byte layout of the workspace for capacities.
struct ChunkLayout {
    size_t header, pairs, splits, pair_tmp, bitmaps, stats, partials, total;
    int64_t pair_cap, part_cap;
    int tt, words;

    __host__ __device__ static size_t align(size_t x) { return (x + 255) / 256 * 256; }

    ChunkLayout() = default;

    __host__ __device__ ChunkLayout(int64_t total_q, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t NB,
                                    int64_t n_rows) {
        tt = static_cast<int>(128 / (Hq / Hkv));
        words = static_cast<int>((NB + 31) / 32);
        pair_cap = total_q / (2 * tt) + (B < total_q ? B : total_q);
        part_cap = pair_cap * Hkv * NB;
        if (part_cap > kChunkMaxParts) part_cap = kChunkMaxParts;
        size_t off = 0;
        header = off;   off += align(sizeof(ChunkHeader));
        pairs = off;    off += align(sizeof(ChunkPair) * (size_t)pair_cap);
        splits = off;   off += align(sizeof(ChunkSplit) * (size_t)pair_cap);
        pair_tmp = off; off += align(sizeof(int32_t) * 2 * (size_t)pair_cap);
        bitmaps = off;  off += align(sizeof(uint32_t) * (size_t)Hkv * (size_t)n_rows * (size_t)words);
        stats = off;    off += align(sizeof(float) * 2 * (size_t)part_cap * 256);
        partials = off; off += align(sizeof(float) * (size_t)part_cap * 256 * (size_t)D);
        total = off;
    }
};

struct ChunkPlanArgs {
    ChunkArgs a;
    ChunkLayout lay;
    char *ws;
    int32_t heads_built;  // bitmaps per row: 1 when every kv head shares the selection, else Hkv
    int32_t ctas;         // CTAs of the attention kernel
};

// One launch: CTA 0 cuts the batch into pairs and units; the others turn the
// selection rows into bitmaps of key blocks and zero the output rows of tokens
// that no sequence owns.
cudaError_t launch_chunk_plan(const ChunkPlanArgs &p, cudaStream_t stream);

// Covers bf16 (or, over an E4M3 cache, f16) queries of head dim 64 or 128 with
// 16-byte aligned rows and positive scales; anything else: *used stays false.
cudaError_t launch_chunk_tc(const ChunkArgs &a, void *ws, cudaStream_t stream, bool *used);

}  // namespace spd
