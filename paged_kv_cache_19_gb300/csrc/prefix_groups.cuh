// prefix_groups.cuh -- the groups of sequences that share leading cache blocks, as the two
// kernels of paged_shared_prefix_attention see them: which group a sequence is in, the work
// units of the shared pass, and where its partial results lie.
//
// Group g holds the sequences [off_g, off_g+1) and shares the first blocks_g blocks of each.  Its
// query rows for one kv head are the members' rows one after another (member m's row r is group
// row m * rows + r); they are cut into pairs of 128-row tiles (256 rows).  A run is one
// (group, kv head, pair): PFX_PAD positions for what starting it costs, then its units, the 128-token
// tiles of the prefix.  Positions are numbered in the order (group, kv head, pair, tile); CTA c of G
// takes the positions [P c / G, P (c+1) / G) of all P (G: the grid, or fewer where that keeps ranges
// from being too short).
#pragma once

#include "device_common.cuh"
#include "kernels.h"

namespace kvp {

constexpr int PFX_TILE = 128;              // tokens of a unit, rows of a row tile
constexpr int PFX_PAIR = 2 * PFX_TILE;     // rows of a run

// What starting a run costs (its query rows, its piece), in units.  With 1 / 8 / 16: 32 groups of 8
// sequences 161 / 159 / 159 us, one 8-bit system prompt 86 / 82 / 84, one document 103 / 100 / 102.
constexpr int PFX_PAD = 8;

// a / b for non-negative values; in 32 bits where they fit.
__device__ __forceinline__ long long div_small(long long a, long long b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

struct PrefixGroup {
    int off, n;                            // members
    int blocks;                            // shared blocks; 0: computed without sharing
};

// Whether a group shares anything: its block count is in range, a single sequence has nobody to
// share with, and a run costs more than it saves where few sequences share little (share_least).
__device__ __forceinline__ bool prefix_shares(const PrefixParams& p, int members, int blocks)
{
    return members >= 2 && blocks > 0 && blocks <= p.max_blocks &&
           static_cast<long long>(members - 1) * blocks >= p.share_least;
}

__device__ __forceinline__ PrefixGroup load_prefix_group(const PrefixParams& p, int g)
{
    PrefixGroup gr;
    gr.off = __ldg(p.group_offsets + g);
    gr.n = __ldg(p.group_offsets + g + 1) - gr.off;
    const int blocks = __ldg(p.group_blocks + g);
    gr.blocks = prefix_shares(p, gr.n, blocks) ? blocks : 0;
    return gr;
}

// Whether the offsets of group g are in order and inside the batch.
__device__ __forceinline__ bool prefix_offsets_ok(const PrefixParams& p, int g)
{
    const int a = __ldg(p.group_offsets + g), b = __ldg(p.group_offsets + g + 1);
    return 0 <= a && a <= b && b <= p.batch;
}

__device__ __forceinline__ int prefix_pairs(const PrefixParams& p, const PrefixGroup& gr)
{
    return (gr.n * p.rows + PFX_PAIR - 1) / PFX_PAIR;
}

// Index of a sharing group's first run among all runs, with gaps: it grows by at least the
// group's pairs from one sharing group to the next (two members or more each), so no sum over
// the groups is needed to find it.  Less than prefix_run_slots().
__device__ __forceinline__ int prefix_run_base(const PrefixParams& p, int g, const PrefixGroup& gr)
{
    return p.kv_heads * (gr.off * p.rows / PFX_PAIR + min(gr.off / 2, g));
}

}  // namespace kvp
