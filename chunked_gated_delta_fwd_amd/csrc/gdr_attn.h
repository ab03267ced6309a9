// Internal interface between the host API (gdr_attn_api.cpp) and the kernels
// of softmax attention (gdr_attn.hip, gdr_attn_bwd.hip) and of the paged cache
// (gdr_paged.hip).  Not installed; not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

constexpr int kAttnRows = 128;   // query rows (gradient of keys: key rows) of a block, 32 a wave

struct AttnArgs {
    const void *q, *k, *v;       // rows ldq, ldk, ldv elements apart, heads and channels compact
    const int32_t *cu, *cuk;     // [N + 1] of queries and keys; NULL: n_seq rows of seq_q and seq_k tokens
    void *o;                     // [total_q, hq, d]; backward: input, rows ldo apart
    float *lse;                  // [total_q, hq], NULL: not written
    int64_t ldq, ldk, ldv, ldo;
    int64_t n_seq, seq_q, seq_k, total_q, total_k;
    int32_t hq, hk, d, bf16, causal;
    int64_t window;              // keys that a query sees back from its own place, itself included; 0: all
    float scale;
    // Forward: the keys of the blocks from `whole` (a multiple of 8 team) on are split in `splits` runs at most, each of
    // at least `least` tiles, whose outputs before they are scaled and whose reference and sum are joined by a second
    // kernel.  An XCD takes a split of `team` blocks, which share their keys, then the next one.
    int32_t splits, least, team, run_rows;
    int64_t whole;
    float *run_o, *run_stat;     // [blocks from `whole` on][run_rows][d], .. [2]; splits 1: none
    // backward
    const void *dout;            // rows lddo apart
    int64_t lddo;
    void *dq, *dk, *dv;          // compact
    float *stat;                 // [2][hq][total_q]: lse in powers of two, and do . o
    // Where blocks are few, `parts` of them share a key block: its group's heads, and then `runs` the queries of a
    // head; and runs_q share a query block's keys.
    float *part;                 // [parts][2][total_k][hk][d]: sums of dk and dv; NULL: one part
    float *part_q;               // [runs_q][total_q][hq][d]: sums of dq; NULL: one run
    int32_t parts, runs, runs_q;
};
// How long a launch takes, in us, by a model: blocks go through the chip `slots`
// at a time, and a step of one takes `full` where the CUs are full and `half`
// where a block has one for itself.  Blocks of one length go in rounds, uneven
// ones fill the gaps, and the longest takes its own time.
struct AttnCost {
    double slots, full, half;
};
inline double attn_time(const AttnCost &c, double blocks, double mean_steps, double most_steps) {
    const double rounds = static_cast<double>(static_cast<int64_t>(blocks / c.slots)), rest = blocks - rounds * c.slots;
    const double last = rest > 256 ? c.full : rest > 0.5 ? c.half : 0;
    const bool even = rounds < 1 || mean_steps > 0.9 * most_steps;
    const double all = (even ? rounds * c.full + last : blocks / c.slots * c.full) * mean_steps;
    const double longest = (blocks > 256 ? 0.85 * c.full : c.half) * most_steps;
    return all > longest ? all : longest;
}
// Tiles of kAttnRows rows of all sequences of `rows` rows each, or about so many.
inline double attn_blocks(bool packed, double sequences, double rows) {
    if (packed) return sequences * (rows < kAttnRows / 2 ? 1.0 : rows / kAttnRows + 0.5);
    return sequences * static_cast<double>((static_cast<int64_t>(rows) + kAttnRows - 1) / kAttnRows);
}
// Sets how the keys are split.
void attn_split(AttnArgs &a);
int64_t attn_cut_blocks(const AttnArgs &a);   // blocks whose keys are split
// Blocks (of 256 threads) of the largest launch of a call; more than 2^24 - 1 cannot be launched.
int64_t attn_fwd_grid(const AttnArgs &a);
int64_t attn_bwd_grid(const AttnArgs &a);
hipError_t launch_attn_fwd(const AttnArgs &a, hipStream_t stream);
// Sets how blocks are shared.
void attn_bwd_split(AttnArgs &a);
hipError_t launch_attn_bwd(const AttnArgs &a, hipStream_t stream);

// Keys and values in pages: row r of page p is row p * page + r of [pages * page, hk, d].
struct PagedArgs {
    const void *q;               // [N, hq, d], rows ldq apart
    const void *k, *v;
    const int32_t *table, *lens; // [N, width] pages of each sequence in order; keys of each
    void *o;                     // [N, hq, d]
    int64_t ldq, n_seq, pages, width, window;
    int32_t page, hq, hk, d, bf16;
    float scale;
    uint32_t magic;              // j / page = j * magic >> shift, for 0 <= j < 2^31
    int32_t shift;
    // each sequence's keys are split in chunks of `chunk`, `splits` at most
    int64_t splits;
    int32_t chunk;
    float *part, *stat;          // [N, hq, splits][d] outputs before they are scaled, [N, hq, splits][2] their reference and sum
};
// Sets chunk and splits.
void paged_split(PagedArgs &a);
int64_t paged_grid(const PagedArgs &a);
hipError_t launch_paged_step(const PagedArgs &a, hipStream_t stream);

struct StoreArgs {
    const void *k, *v;           // [tokens] rows of row_bytes, ldk and ldv bytes apart
    const int32_t *slots;        // [tokens]; outside the pages: not stored
    void *kp, *vp;               // [rows] of row_bytes
    int64_t tokens, rows, row_bytes, ldk, ldv;
};
int64_t page_store_grid(const StoreArgs &a);
hipError_t launch_page_store(const StoreArgs &a, hipStream_t stream);

struct PlanArgs {
    const int32_t *past, *fresh, *pool;   // [N], [N], [pool_size]
    int32_t *table;                       // [N, width]
    int32_t *cu, *lens, *positions, *slots, *used;   // [N + 1], [N], [tokens], [tokens], [2]
    int64_t n_seq, pool_size, width, tokens;
    int32_t page;
};
hipError_t launch_page_plan(const PlanArgs &a, hipStream_t stream);

}  // namespace gdr
