// rows.h -- internal interface of the ragged attention over the paged latent cache: chunks of
// new tokens (any number per sequence) and decode with a sliding window and sinks.
//
// The work is a list of items. An item is up to 128 query rows of one sequence: `ntok`
// consecutive tokens of `hq` heads each, the first token at position pos0. The pages that its
// tokens see between them form its list of visible pages: the pages of the first `sinks` rows,
// then the pages of the window (one run when the two meet, or without a window). Two pages of
// that list are one tile.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mla.h"

namespace mla {

// Visible pages of ntok tokens from position pos0 on (positions below 0 see nothing): page v of
// the list is page v of the sequence for v < lead, else page v + gap.
struct VisiblePages {
    int count, lead, gap;
};
__host__ __device__ inline VisiblePages visible_pages(int pos0, int ntok, int window, int sinks) {
    VisiblePages r{0, 0, 0};
    const int end = pos0 + ntok;  // rows [0, end) are cached
    if (end <= 0) return r;
    const int pages = (end - 1) / MLA_BLOCK + 1;
    r.count = r.lead = pages;
    if (window > 0) {
        // the window of the first token that sees anything opens the run of window pages
        const int first = pos0 > 0 ? pos0 : 0;
        const int lo = first >= window ? first - window + 1 : 0;
        const int seen = sinks < end ? sinks : end;  // of the first rows
        const int front = seen / MLA_BLOCK + (seen % MLA_BLOCK != 0);
        if (lo / MLA_BLOCK > front) {
            r.lead = front;
            r.gap = lo / MLA_BLOCK - front;
            r.count = pages - r.gap;
        }
    }
    return r;
}
__host__ __device__ inline int visible_tiles(const VisiblePages &v) { return (v.count + 1) / 2; }
// the most tiles that an item of at most ntok tokens can have, for lengths up to max_seqlen
inline int most_visible_tiles(int max_seqlen, int ntok, int window, int sinks) {
    const long all = ((long)max_seqlen + MLA_BLOCK - 1) / MLA_BLOCK;
    if (window == 0) return (int)((all + 1) / 2);
    const long near = ((long)window + ntok - 2) / MLA_BLOCK + 2;  // at any offset in its page
    const long front = ((long)sinks + MLA_BLOCK - 1) / MLA_BLOCK;
    const long some = near + front < all ? near + front : all;
    return (int)((some + 1) / 2);
}

// One cluster's piece of an item, written by the schedule kernel.
struct RowsSegment {
    int32_t b, tok0, ntok, pos0;  // the item: sequence, first token's row in q, tokens, position
    int32_t t0, t1, part, pad;    // its tiles [t0, t1); fp32 part index, or -1: the whole item
};
static_assert(sizeof(RowsSegment) == 32, "two 16-byte loads");

struct RowsParams {
    const uint16_t *q_lat;   // [tokens][hq][512]
    const uint16_t *q_rope;  // [tokens][hq][64]
    const uint16_t *cache;   // bf16 cache, or null:
    const uint8_t *codes;    // FP8 cache
    const int8_t *exps;
    const int32_t *block_table, *seqlens;
    int num_blocks, max_blocks, B, hq, tokens, max_seqlen;
    int window, sinks;  // window 0: none
    float scale_log2;
    uint16_t *out;  // [tokens][hq][512]
    float *lse;     // [tokens][hq]
    float *o_part;  // [parts][rows][512], rows = rows_per_item
    float *lse_part;
    int rows_per_item;
    bool stream_cache;  // every cached row is read by one item only: let it leave L2 first
    uint32_t *err;
    // fixed split (segs null): each item is cut into num_splits ranges of tiles_per_split tiles,
    // one cluster each. Without q_starts item b is sequence b with s_q tokens; with them the items
    // are the sequences' tokens in groups of s_q (find_item).
    int s_q, num_splits, tiles_per_split;
    const int32_t *q_starts;
    // schedule: cluster c runs segs[seg_range[2c] .. seg_range[2c + 1])
    const RowsSegment *segs;
    const int32_t *seg_range;
};

#ifdef __CUDACC__
// Item `item` of the token ranges q_starts [B + 1], in groups of `group` tokens: (sequence, first
// token's row in q, tokens, tokens of the sequence before it), or tokens 0 if there is none. By a
// converged warp. broken: the ranges do not ascend inside [0, tokens] (then there is no item).
__device__ inline int4 find_item(const int32_t *q_starts, int B, int tokens, int group, int item,
                                 bool *broken) {
    const int lane = threadIdx.x & 31;
    int4 r = make_int4(0, 0, 0, 0);
    int carry = 0;
    bool bad = false;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        int q0 = 0, q1 = 0;
        if (b < B) q0 = q_starts[b], q1 = q_starts[b + 1];
        const bool wrong = q0 < 0 || q1 < q0 || q1 > tokens;
        bad |= wrong;
        const int k = wrong ? 0 : (q1 - q0 + group - 1) / group;
        int inc = k;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const int at = (item - (carry + inc - k)) * group;  // tokens before, if it is this lane's
        const unsigned own =
            __ballot_sync(0xffffffffu, item >= carry + inc - k && item < carry + inc);
        if (own) {
            const int from = __ffs(own) - 1;
            r.x = b0 + from;
            r.w = __shfl_sync(0xffffffffu, at, from);
            r.y = __shfl_sync(0xffffffffu, q0, from) + r.w;
            r.z = min(group, __shfl_sync(0xffffffffu, q1, from) - r.y);
        }
        carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    *broken = __any_sync(0xffffffffu, bad);
    if (*broken) r.z = 0;
    return r;
}
#endif

// grid = `clusters` two-CTA clusters
cudaError_t launch_rows_tc(const RowsParams &p, int clusters, cudaStream_t stream);
int rows_tc_cluster_slots();

// A segment costs about as much to begin and end as this many tiles take (2 to 8 are within 3% of
// each other on 128 sequences of 33 tiles and on two chunks of 300 tokens).
constexpr int ROWS_SEG_COST = 4;

struct RowsSchedule {
    const int32_t *q_starts;  // [B + 1] first token of each sequence; null: s_q tokens each
    const int32_t *seqlens;   // [B]
    int B, s_q, tokens, tokens_per_item, hq, max_seqlen, window, sinks;
    int clusters, max_items;
    int32_t *item_wpos;   // [max_items] weight position of the item's first tile
    int4 *items;          // [max_items] (b, tok0, ntok, pos0)
    RowsSegment *segs;    // [max_items + clusters]
    int32_t *seg_range;   // [2 * clusters]
    int4 *jobs;           // [clusters] merge: (first row of out, rows, first part, parts)
    int32_t *n_items;
    uint32_t *err;
};
cudaError_t launch_rows_schedule(const RowsSchedule &s, cudaStream_t stream);
// The same with fixed ranges: the `splits` parts of each of at most max_items items.
cudaError_t launch_rows_merge_items(const RowsParams &p, int max_items, cudaStream_t stream);
// Merges the jobs' parts and writes the items that see nothing (out = 0, lse = -inf).
cudaError_t launch_rows_merge(const RowsSchedule &s, const float *o_part, const float *lse_part,
                              int rows_per_item, uint16_t *out, float *lse, cudaStream_t stream);

}  // namespace mla
