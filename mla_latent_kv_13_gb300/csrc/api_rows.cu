// api_rows.cu -- the C ABI of the ragged attention over the paged latent cache (declared in
// include/mla.h): chunks of new tokens, and decode with a sliding window and sinks.
#include <limits.h>
#include <math.h>

#include "abi.h"
#include "common.cuh"
#include "rows.h"

using namespace mla;

namespace {

struct RowsPlan {
    int splits;  // fixed ranges per item, or 0: the schedule
    int tiles;   // the most tiles of an item
    int max_items, clusters, rows;
    size_t items, wpos, segs, range, jobs, n_items, o_part, lse_part, total;
};

// Workspace of the schedule over at most max_items items.
bool plan_schedule(RowsPlan &r) {
    // the schedule's weights are 32-bit
    if ((long)r.max_items * (r.tiles + ROWS_SEG_COST) > INT_MAX) return false;
    const long tiles = (long)r.max_items * (r.tiles > 0 ? r.tiles : 1);
    const int slots = rows_tc_cluster_slots();
    const int P = r.clusters = (int)(tiles < slots ? tiles : slots);
    r.items = HDR;
    r.wpos = r.items + align256((size_t)r.max_items * sizeof(int4));
    r.segs = r.wpos + align256((size_t)r.max_items * 4);
    r.range = r.segs + align256(((size_t)r.max_items + P) * sizeof(RowsSegment));
    r.jobs = r.range + align256((size_t)P * 8);
    r.n_items = r.jobs + align256((size_t)P * sizeof(int4));
    r.o_part = r.n_items + 256;
    const size_t parts = 2 * (size_t)P;  // a cluster cuts at most two items
    r.lse_part = r.o_part + align256(parts * r.rows * D_C * sizeof(float));
    r.total = r.lse_part + align256(parts * r.rows * sizeof(float));
    return true;
}

// Ranges of an item with `tiles` tiles while `items` of them fit the GPU at once: each short, one
// tile up to 6 tiles of an item, then two, from 13 on three, as far as clusters are free and at
// most 32 (the parts of a row are merged by one warp, eight at a time). Measured for window decode
// at 128 heads, bf16 (FP8) cache, us: 1 sequence of 5 tiles 14.3 (20.1) whole, 13.2 (15.7) in
// ranges of one; 4 of 9 tiles 19.3 (30.5) whole, 14.4 (17.6) in fives; 1 of 34 tiles 47.0 (82.4)
// whole, 16.3 (20.7) in 12 ranges, 18.7 (21.9) in 32; 1 of 127 tiles 22.8 (32.0) in 16, 20.8 (26.0)
// in 32, 23.7 (26.9) in 64; 16 of 9 tiles 19.5 (31.3) whole, 20.6 (24.6) in four. Over a bf16 cache
// up to 6 tiles of more than 64 rows stay whole, as the parts cost what the ranges gain and the
// merge a launch (12 of 5 tiles 15.0 whole, 17.1 in fives; 1 of 3 tiles 12.3 and 13.3), but for 5 or
// 6 tiles of up to four items (1 of 5 tiles 14.7 and 13.1, 4 of them 14.8 and 13.3, 8 of them 14.8
// and 14.9).
int fixed_ranges(int items, int tiles, int rows, bool fp8) {
    const int slots = rows_tc_cluster_slots();
    const int per = tiles <= 6 ? 1 : tiles <= 12 ? 2 : 3;
    int n = (tiles + per - 1) / per;
    if (n > slots / items) n = slots / items;
    if (n > 32) n = 32;
    const bool whole = !fp8 && tiles <= 6 && rows > 64 && (tiles < 5 || items > 4);
    return n < 1 || whole ? 1 : n;
}
// Workspace of fixed ranges.
void plan_fixed(RowsPlan &r, int items, int splits) {
    r.splits = splits;
    r.clusters = items * splits;
    r.total = HDR;
    if (splits > 1) {
        r.o_part = HDR;
        r.lse_part = r.o_part + align256((size_t)items * splits * r.rows * D_C * sizeof(float));
        r.total = r.lse_part + align256((size_t)items * splits * r.rows * sizeof(float));
    }
}

// Window decode: items are whole sequences. Fixed ranges, which need no schedule launch; with more
// sequences than clusters the schedule.
bool plan_window(int B, int s_q, int H, int max_seqlen, int window, int sinks, int num_splits,
                 bool fp8, RowsPlan &r) {
    r = RowsPlan{};
    r.rows = s_q * H;
    r.max_items = B;
    r.tiles = most_visible_tiles(max_seqlen, s_q, window, sinks);
    int best = num_splits;
    if (num_splits == 0 && B <= rows_tc_cluster_slots()) best = fixed_ranges(B, r.tiles, r.rows, fp8);
    if (best == 0) return plan_schedule(r);
    plan_fixed(r, B, best);
    if (num_splits == 0 && r.tiles > 1) {
        // the size for the most parts that a smaller batch can have, so that a workspace for the
        // largest one serves them all (the schedule's has room for more)
        const int slots = rows_tc_cluster_slots();
        const long parts = (long)B * (r.tiles < 32 ? r.tiles : 32);
        RowsPlan most = r;
        plan_fixed(most, 1, (int)(parts < slots ? parts : slots));
        r.total = most.total;
    }
    return true;
}

// Chunks: the schedule; for few short items fixed ranges (a launch less). They are not balanced, so
// only as long as the longest range that a sequence of max_seqlen can have takes about as long as
// a schedule with its merge at least does: 12 tiles (FP8 8). Measured, us, schedule and fixed
// ranges over a bf16 (FP8) cache: 3 sequences of 9 tokens on 300 rows 17.9 and 12.0 (21.6 and
// 18.8); 8 tokens on 8000 rows 40.7 and 17.1 (44.1 and 21.1); 70 single tokens of 128 heads on 12 tiles
// 41.3 and 29.2; 20 sequences of 8 tokens on 16 tiles 27.0 and 25.0 (32.4 and 34.3).
bool plan_chunk(int B, int tokens, int H, int max_seqlen, int window, int sinks, bool fp8,
                RowsPlan &r) {
    r = RowsPlan{};
    const int per = 128 / H;  // tokens of an item
    r.rows = 128;
    r.max_items = (int)(((long)tokens + (long)B * (per - 1)) / per);
    r.tiles = most_visible_tiles(max_seqlen, per, window, sinks);
    if (!plan_schedule(r)) return false;
    if (r.max_items <= rows_tc_cluster_slots() && B <= rows_tc_cluster_slots()) {
        const int best = fixed_ranges(r.max_items, r.tiles, 128, fp8);
        // (the schedule has room for at least as many parts; with its size in both cases a workspace
        // for longer sequences serves shorter ones too)
        const size_t total = r.total;
        const int range_tiles = fp8 ? 8 : 12;
        if (r.tiles <= range_tiles * best) plan_fixed(r, r.max_items, best);
        r.total = total;
    }
    return true;
}

// Attention of the planned items; q_starts null: s_q tokens in every sequence.
mla_status_t run(const RowsPlan &r, RowsParams p, const int32_t *q_starts, int tokens_per_item,
                 void *workspace, cudaStream_t st) {
    char *w = static_cast<char *>(workspace);
    p.err = err_word(workspace);
    p.rows_per_item = r.rows;
    if (r.o_part) {
        p.o_part = reinterpret_cast<float *>(w + r.o_part);
        p.lse_part = reinterpret_cast<float *>(w + r.lse_part);
    }
    if (r.splits > 0) {
        p.num_splits = r.splits;
        p.tiles_per_split = r.tiles > 0 ? (r.tiles + r.splits - 1) / r.splits : 1;
        p.q_starts = q_starts;
        if (q_starts) p.s_q = tokens_per_item;
        if (launch_rows_tc(p, r.clusters, st) != cudaSuccess) return MLA_ERR_CUDA;
        if (r.splits == 1) return MLA_OK;
        return cuda_status(launch_rows_merge_items(p, r.max_items, st));
    }
    RowsSchedule s{};
    s.q_starts = q_starts; s.seqlens = p.seqlens;
    s.B = p.B; s.s_q = p.s_q; s.tokens = p.tokens; s.tokens_per_item = tokens_per_item; s.hq = p.hq;
    s.max_seqlen = p.max_seqlen; s.window = p.window; s.sinks = p.sinks;
    s.clusters = r.clusters; s.max_items = r.max_items;
    s.items = reinterpret_cast<int4 *>(w + r.items);
    s.item_wpos = reinterpret_cast<int32_t *>(w + r.wpos);
    s.segs = reinterpret_cast<RowsSegment *>(w + r.segs);
    s.seg_range = reinterpret_cast<int32_t *>(w + r.range);
    s.jobs = reinterpret_cast<int4 *>(w + r.jobs);
    s.n_items = reinterpret_cast<int32_t *>(w + r.n_items);
    s.err = p.err;
    p.segs = s.segs;
    p.seg_range = s.seg_range;
    p.num_splits = 1;
    if (launch_rows_schedule(s, st) != cudaSuccess) return MLA_ERR_CUDA;
    if (launch_rows_tc(p, r.clusters, st) != cudaSuccess) return MLA_ERR_CUDA;
    return cuda_status(launch_rows_merge(s, p.o_part, p.lse_part, r.rows, p.out, p.lse, st));
}

// Checks that both calls share, all but the workspace; B, tokens and head limits are theirs.
mla_status_t validate(const void *q_lat, const void *q_rope, const void *cache, const int8_t *exps,
                      bool fp8, int num_blocks, const int32_t *block_table, int max_blocks,
                      const int32_t *seqlens, int max_seqlen, int sinks, float scale,
                      const void *out, const float *lse) {
    if (!q_lat || !q_rope || !cache || !block_table || !seqlens || !out || !lse || (fp8 && !exps))
        return MLA_ERR_INVALID_ARG;
    if (num_blocks < 1 || max_blocks < 1 || max_seqlen < 0 || sinks < 0 ||
        max_seqlen > (long)max_blocks * BLOCK || !(scale > 0.f) || !isfinite(scale))
        return MLA_ERR_INVALID_ARG;
    if (num_blocks > (1 << 24)) return MLA_ERR_UNSUPPORTED;
    if (!aligned(q_lat, 16) || !aligned(q_rope, 16) || !aligned(cache, 16) || !aligned(out, 32) ||
        !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seqlens, 4) ||
        (fp8 && !aligned(exps, 16)))
        return MLA_ERR_INVALID_ARG;
    return MLA_OK;
}

mla_status_t window_run(const mla_bf16_t *q_lat, const mla_bf16_t *q_rope, const mla_bf16_t *cache,
                        const uint8_t *codes, const int8_t *exps, int num_blocks,
                        const int32_t *block_table, int max_blocks, const int32_t *seqlens, int B,
                        int s_q, int H, int max_seqlen, int window, int sinks, float scale,
                        int num_splits, void *workspace, size_t ws_bytes, mla_bf16_t *out,
                        float *lse, mla_stream_t stream) {
    const void *any = codes ? static_cast<const void *>(codes) : cache;
    mla_status_t v = validate(q_lat, q_rope, any, exps, codes != nullptr, num_blocks, block_table,
                              max_blocks, seqlens, max_seqlen, sinks, scale, out, lse);
    if (v != MLA_OK) return v;
    size_t need = 0;
    v = mla_decode_window_workspace_size(B, s_q, H, max_seqlen, window, sinks, num_splits, &need);
    if (v != MLA_OK) return v;
    if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
    if (ws_bytes < need) return MLA_ERR_WORKSPACE;
    RowsPlan r;
    plan_window(B, s_q, H, max_seqlen, window, sinks, num_splits, codes != nullptr, r);
    RowsParams p{};
    p.q_lat = q_lat; p.q_rope = q_rope; p.cache = cache; p.codes = codes; p.exps = exps;
    p.block_table = block_table; p.seqlens = seqlens;
    p.num_blocks = num_blocks; p.max_blocks = max_blocks; p.B = B; p.hq = H; p.tokens = B * s_q;
    p.max_seqlen = max_seqlen; p.window = window; p.sinks = sinks; p.s_q = s_q;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = out; p.lse = lse;
    p.stream_cache = true;
    return run(r, p, nullptr, s_q, workspace, S(stream));
}

mla_status_t chunk_run(const mla_bf16_t *q_lat, const mla_bf16_t *q_rope, const mla_bf16_t *cache,
                       const uint8_t *codes, const int8_t *exps, int num_blocks,
                       const int32_t *block_table, int max_blocks, const int32_t *q_starts,
                       const int32_t *seqlens, int B, int tokens, int H, int max_seqlen,
                       int window, int sinks, float scale, void *workspace, size_t ws_bytes,
                       mla_bf16_t *out, float *lse, mla_stream_t stream) {
    const void *any = codes ? static_cast<const void *>(codes) : cache;
    mla_status_t v = validate(q_lat, q_rope, any, exps, codes != nullptr, num_blocks, block_table,
                              max_blocks, seqlens, max_seqlen, sinks, scale, out, lse);
    if (v != MLA_OK) return v;
    if (!q_starts || !aligned(q_starts, 4)) return MLA_ERR_INVALID_ARG;
    size_t need = 0;
    v = mla_chunk_workspace_size(B, tokens, H, max_seqlen, window, sinks, &need);
    if (v != MLA_OK) return v;
    if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
    if (ws_bytes < need) return MLA_ERR_WORKSPACE;
    RowsPlan r;
    plan_chunk(B, tokens, H, max_seqlen, window, sinks, codes != nullptr, r);
    RowsParams p{};
    p.q_lat = q_lat; p.q_rope = q_rope; p.cache = cache; p.codes = codes; p.exps = exps;
    p.block_table = block_table; p.seqlens = seqlens;
    p.num_blocks = num_blocks; p.max_blocks = max_blocks; p.B = B; p.hq = H; p.tokens = tokens;
    p.max_seqlen = max_seqlen; p.window = window; p.sinks = sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = out; p.lse = lse;
    return run(r, p, q_starts, 128 / H, workspace, S(stream));
}

}  // namespace

extern "C" {

mla_status_t mla_decode_window_workspace_size(int B, int s_q, int H, int max_seqlen, int window,
                                              int sinks, int num_splits, size_t *bytes) {
    if (!bytes || B < 1 || B > 4096 || s_q < 1 || max_seqlen < 0 || window < 1 || sinks < 0 ||
        num_splits < 0 || num_splits > 256)
        return MLA_ERR_INVALID_ARG;
    if (!heads_ok(H) || s_q > 128 / H) return MLA_ERR_UNSUPPORTED;
    size_t most = 0;  // of either cache
    for (int fp8 = 0; fp8 < 2; ++fp8) {
        RowsPlan r;
        if (!plan_window(B, s_q, H, max_seqlen, window, sinks, num_splits, fp8 != 0, r))
            return MLA_ERR_UNSUPPORTED;
        if (r.total > most) most = r.total;
    }
    *bytes = most;
    return MLA_OK;
}

mla_status_t mla_decode_attention_window(const mla_bf16_t *q_lat, const mla_bf16_t *q_rope,
                                         const mla_bf16_t *kv_cache, int num_blocks,
                                         const int32_t *block_table, int max_blocks,
                                         const int32_t *seqlens, int B, int s_q, int H,
                                         int max_seqlen, int window, int sinks, float scale,
                                         int num_splits, void *workspace, size_t ws_bytes,
                                         mla_bf16_t *out, float *lse, mla_stream_t stream) {
    return window_run(q_lat, q_rope, kv_cache, nullptr, nullptr, num_blocks, block_table,
                      max_blocks, seqlens, B, s_q, H, max_seqlen, window, sinks, scale, num_splits,
                      workspace, ws_bytes, out, lse, stream);
}

mla_status_t mla_decode_attention_window_fp8(const mla_bf16_t *q_lat, const mla_bf16_t *q_rope,
                                             const uint8_t *kv_codes, const int8_t *kv_exps,
                                             int num_blocks, const int32_t *block_table,
                                             int max_blocks, const int32_t *seqlens, int B, int s_q,
                                             int H, int max_seqlen, int window, int sinks,
                                             float scale, int num_splits, void *workspace,
                                             size_t ws_bytes, mla_bf16_t *out, float *lse,
                                             mla_stream_t stream) {
    if (!kv_codes) return MLA_ERR_INVALID_ARG;
    return window_run(q_lat, q_rope, nullptr, kv_codes, kv_exps, num_blocks, block_table,
                      max_blocks, seqlens, B, s_q, H, max_seqlen, window, sinks, scale, num_splits,
                      workspace, ws_bytes, out, lse, stream);
}

mla_status_t mla_chunk_workspace_size(int B, int tokens, int H, int max_seqlen, int window,
                                      int sinks, size_t *bytes) {
    if (!bytes || B < 1 || B > 4096 || tokens < 1 || max_seqlen < 0 || window < 0 || sinks < 0)
        return MLA_ERR_INVALID_ARG;
    if (!heads_ok(H) || tokens > (1 << 20)) return MLA_ERR_UNSUPPORTED;
    RowsPlan r;  // (the same for either cache)
    if (!plan_chunk(B, tokens, H, max_seqlen, window, sinks, false, r)) return MLA_ERR_UNSUPPORTED;
    *bytes = r.total;
    return MLA_OK;
}

mla_status_t mla_chunk_attention(const mla_bf16_t *q_lat, const mla_bf16_t *q_rope,
                                 const mla_bf16_t *kv_cache, int num_blocks,
                                 const int32_t *block_table, int max_blocks,
                                 const int32_t *q_starts, const int32_t *seqlens, int B,
                                 int tokens, int H, int max_seqlen, int window, int sinks,
                                 float scale, void *workspace, size_t ws_bytes, mla_bf16_t *out,
                                 float *lse, mla_stream_t stream) {
    return chunk_run(q_lat, q_rope, kv_cache, nullptr, nullptr, num_blocks, block_table, max_blocks,
                     q_starts, seqlens, B, tokens, H, max_seqlen, window, sinks, scale, workspace,
                     ws_bytes, out, lse, stream);
}

mla_status_t mla_chunk_attention_fp8(const mla_bf16_t *q_lat, const mla_bf16_t *q_rope,
                                     const uint8_t *kv_codes, const int8_t *kv_exps,
                                     int num_blocks, const int32_t *block_table, int max_blocks,
                                     const int32_t *q_starts, const int32_t *seqlens, int B,
                                     int tokens, int H, int max_seqlen, int window, int sinks,
                                     float scale, void *workspace, size_t ws_bytes,
                                     mla_bf16_t *out, float *lse, mla_stream_t stream) {
    if (!kv_codes) return MLA_ERR_INVALID_ARG;
    return chunk_run(q_lat, q_rope, nullptr, kv_codes, kv_exps, num_blocks, block_table, max_blocks,
                     q_starts, seqlens, B, tokens, H, max_seqlen, window, sinks, scale, workspace,
                     ws_bytes, out, lse, stream);
}

}  // extern "C"
